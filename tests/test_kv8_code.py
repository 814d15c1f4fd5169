"""The gfx950 code of the 8-bit key/value cache's kernels, read as assembly on
the CPU: memory is written by vector stores only, no packed FP32 arithmetic is
used, and no vector register is spilled."""

import re

import pytest

from cross_core_barrier_amd import build


@pytest.fixture(scope="module", params=["ccb_kv8_cache.hip", "ccb_kv8_attend.hip"])
def asm(request, tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "k.s")
    with open(build.device_assembly(out, request.param)) as f:
        return f.read()


def _instructions(text):
    return [line.split()[0] for line in text.splitlines() if re.match(r"\t[a-z]\w+( |$)", line)]


def _forbidden(op):
    if op.startswith("v_pk_"):
        return op.endswith("_f32") and op[5:8] in ("add", "mul", "fma")
    # the scalar unit's memory instructions: loads and invalidations only
    return op.startswith("s_") and any(w in op for w in ("store", "atomic", "_wb", "discard"))


def test_stores_and_arithmetic(asm):
    ops = _instructions(asm)
    assert len(ops) > 10000
    assert sum(op.startswith("global_store") for op in ops) > 100
    assert sorted({op for op in ops if _forbidden(op)}) == []


def test_no_vector_register_is_spilled(asm):
    """Scalar ones may go to the lanes of a vector register."""
    found = re.findall(r"\.vgpr_spill_count:\s*(\d+)", asm)
    assert len(found) > 20 and set(found) == {"0"}
    assert not any(op.startswith("scratch_") for op in _instructions(asm))


def test_the_check_sees_what_it_forbids():
    for op in ("v_pk_add_f32", "v_pk_fma_f32", "s_" + "store_dword", "s_buffer_" + "atomic_add"):
        assert _forbidden(op)
    for op in ("v_pk_add_f16", "v_pk_add_u16", "global_store_dwordx4", "s_load_dword", "s_waitcnt", "s_dcache_inv"):
        assert not _forbidden(op)
