"""The 8-bit key/value cache on the CPU: its rounding and range checks,
compiled for the host, against exact fractions; the oracle against itself on
tiny inputs; and every refusal of the entry points that precedes device work."""

import ctypes
import math
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from oracle import kv8 as oracle

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
FMT = {"int8": "0", "e4m3": "1"}


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("kv8") / "math_driver")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-I",
                    os.path.join(ROOT, "cross_core_barrier_amd", "csrc"),
                    os.path.join(HERE, "kv8", "math_driver.cpp"), "-o", exe], check=True)

    def run(mode, fmt, data, dtype):
        res = subprocess.run([exe, mode] + ([FMT[fmt]] if fmt else []), input=np.ascontiguousarray(data).tobytes(),
                             capture_output=True, check=True)
        return np.frombuffer(res.stdout, dtype)
    return run


def _exact(x) -> Fraction:
    return Fraction(float(x))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_new_values_round_once(driver, fmt):
    """Codes of bf16-like values over random scales, among them values that
    lie on or next to the border between two codes."""
    rng = np.random.default_rng(1)
    s = (rng.uniform(1, 2, 6000) * 2.0 ** rng.integers(-60, 60, 6000)).astype(np.float32)
    s[:2000] = (2.0 ** rng.integers(-40, 40, 2000)).astype(np.float32)  # exact borders happen
    grid = np.arange(128.0) if fmt == "int8" else oracle._GRID
    i = rng.integers(0, len(grid) - 1, 6000)
    border = (grid[i] + grid[i + 1]) / 2
    x = (border * s.astype(np.float64)).astype(np.float32)
    x[3000:] = (rng.uniform(-1.2, 1.2, 3000) * oracle.Q[fmt] * s[3000:]).astype(np.float32)
    x[::7] = np.nextafter(x[::7], np.float32(0))
    x[1::7] = np.nextafter(x[1::7], np.float32(np.inf))
    x[::2] *= -1
    inv = (np.float32(1) / s).astype(np.float32)
    got = driver("v", fmt, np.stack([x, inv, s], 1), np.uint8)
    want = np.array([oracle.nearest_code(_exact(a) / _exact(b), fmt) for a, b in zip(x, s)], np.uint8)
    assert np.array_equal(oracle.values(got, fmt), oracle.values(want, fmt))
    # a reciprocal that is off by a few units changes nothing
    for ulps in (-3, 3):
        off = inv.copy()
        for _ in range(abs(ulps)):
            off = np.nextafter(off, np.float32(np.inf if ulps > 0 else 0))
        assert np.array_equal(driver("v", fmt, np.stack([x, off, s], 1), np.uint8), got)
    assert np.array_equal(oracle.values(oracle.encode(x.astype(np.float64), s, fmt), fmt), oracle.values(want, fmt))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_old_codes_round_once(driver, fmt):
    """code * s0 / s1 for every code, at random and at simple ratios (ties)."""
    rng = np.random.default_rng(2)
    codes = np.array([c for c in range(256) if c not in ((0x80,) if fmt == "int8" else (0x7F, 0xFF))], np.uint8)
    v = oracle.values(codes, fmt).astype(np.float32)
    for trial in range(40):
        s0 = np.float32(rng.uniform(1, 2) * 2.0 ** int(rng.integers(-40, 40)))
        ratio = [1.0, 2.0, 3.0, 6.0, 5.0, 4.0, 1.5][trial] if trial < 7 else rng.uniform(1, 30)
        s1 = np.float32(s0 * np.float32(ratio))
        hi = (v * s0).astype(np.float32)
        lo = (v.astype(np.float64) * np.float64(s0) - hi).astype(np.float32)
        n = len(v)
        rec = np.stack([hi, lo, np.full(n, np.float32(1) / s1, np.float32), np.full(n, s1, np.float32)], 1)
        got = driver("e", fmt, rec, np.uint8)
        want = np.array([oracle.nearest_code(_exact(a) * _exact(s0) / _exact(s1), fmt) for a in v], np.uint8)
        assert np.array_equal(oracle.values(got, fmt), oracle.values(want, fmt)), (trial, s0, s1)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_special_values(driver, fmt):
    one = np.float32(1)
    x = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-40, 3e38, -3e38], np.float32)
    got = oracle.values(driver("v", fmt, np.stack([x, np.full(8, one), np.full(8, one)], 1), np.uint8), fmt)
    q = oracle.Q[fmt]
    assert np.array_equal(got, [0, q, -q, 0, 0, 0, q, -q])
    # a block of zeros has scale 0 and codes 0
    assert driver("v", fmt, np.array([[np.inf, np.inf, 0], [0, np.inf, 0]], np.float32), np.uint8).tolist() == [0, 0]
    a = np.array([0.0, 1e-30, 127.0, 448.0, 1.0, 3e38], np.float32)
    want = np.array([oracle.block_scale(v, fmt) for v in a], np.float32)
    assert np.array_equal(driver("b", fmt, a, np.float32), want)
    assert want[0] == 0 and want[1] == np.float32(2.0 ** -64)


def test_weight_order(driver):
    w = np.array([-np.inf, -2.0, -1e-40, 0.0, 1e-45, 1e-40, 0.5, 1.0, 3e38, np.inf], np.float32)
    key = driver("w", None, w, np.uint32).astype(np.int64)
    assert np.all(np.diff(key) > 0)
    nan = driver("w", None, np.array([np.nan, -np.nan], np.float32), np.uint32)
    assert nan.tolist() == [0, 0] and key[0] > 0
    assert len(set(driver("w", None, np.array([0.0, -0.0], np.float32), np.uint32).tolist())) == 1


def test_range_checks(driver):
    lens = np.array([[0, 64], [64, 64], [65, 64], [-1, 64], [-2**31, 64], [2**31 - 1, 64]], np.int32)
    assert driver("l", None, lens, np.int32).tolist() == [0, 64, -1, -1, -1, -1]
    pages = np.array([[0, 7], [6, 7], [7, 7], [-1, 7], [-2**31, 7], [2**31 - 1, 7]], np.int32)
    assert driver("p", None, pages, np.int32).tolist() == [0, 6, -1, -1, -1, -1]


def test_oracle_on_worked_values():
    """One page, one head, numbers small enough to follow by hand."""
    c = dict(k=np.zeros((1, 1, 16, 2), np.uint8), v=np.zeros((1, 1, 16, 2), np.uint8), ks=np.ones((1, 1), np.float32),
             vs=np.ones((1, 1), np.float32), table=np.zeros((1, 1), np.int32), lens=np.array([1], np.int32),
             weight=np.full((1, 1, 16), 9, np.float32), fmt="int8")
    oracle.append(c, np.array([[[[127.0, 1.0]]]]), np.array([[[[2.0, 4.0]]]]), [1])
    assert c["k"][0, 0, 0].tolist() == [127, 1] and c["ks"][0, 0] == 1  # s = 127 / 127
    assert c["v"][0, 0, 0].tolist() == [64, 127]  # 2 * 127 / 4 = 63.5: half to even
    assert c["weight"][0, 0, :2].tolist() == [0, 9]
    c["lens"][0] = 2
    oracle.append(c, np.array([[[[254.0, 0.0]]]]), np.array([[[[4.0, 0.0]]]]), [1])
    assert c["k"][0, 0, :2].tolist() == [[64, 0], [127, 0]]  # 63.5 -> 64, 0.5 -> 0
    out, lse, w, _, _ = oracle.attend(c, np.zeros((1, 1, 1, 2)), 1.0, 0)
    assert np.allclose(lse, math.log(2)) and np.allclose(w[0, 0, :2], 0.5)
    assert oracle.kept(np.array([1, 3, 3, math.nan, 0, 5.0]), 6, 3, 1, 0) == [1, 2, 5]
    assert oracle.kept(np.array([1, 3, 3, math.nan, 0, 5.0]), 6, 5, 1, 0) == [0, 1, 2, 4, 5]


# --- refusals --------------------------------------------------------------------------

@pytest.fixture(scope="module")
def ccb():
    from cross_core_barrier_amd import ccb as lib
    return lib


def _cache(ccb, **changes):
    f = dict(k=1 << 20, v=2 << 20, kScale=3 << 20, vScale=4 << 20, pageTable=5 << 20, lens=6 << 20, weight=7 << 20,
             tableStride=4, weightStride=64, format=0, numPages=8, heads=2, pageSize=16, headDim=64, batch=3, maxPages=4,
             reserved=0)
    f.update(changes)
    return ccb.ccbKv8Cache(**f)


def _rows(ccb, **changes):
    f = dict(data=8 << 20, strideBatch=512, strideToken=128, strideHead=64, type=0, reserved=0)
    f.update(changes)
    return ccb.ccbKv8Rows(**f)


BAD_CACHES = [dict(format=2), dict(format=-1), dict(pageSize=8), dict(pageSize=48), dict(pageSize=256),
              dict(headDim=32), dict(headDim=100), dict(headDim=512), dict(numPages=0), dict(heads=0), dict(batch=-1),
              dict(maxPages=0), dict(maxPages=1 << 27, tableStride=1 << 27), dict(tableStride=3), dict(weightStride=63),
              dict(k=(1 << 20) + 8), dict(v=(1 << 20) + 8), dict(kScale=2), dict(vScale=2), dict(pageTable=2),
              dict(lens=2), dict(weight=2), dict(reserved=1)]
NULL_CACHES = [dict(k=0), dict(v=0), dict(kScale=0), dict(vScale=0), dict(pageTable=0), dict(lens=0)]
BAD_ROWS = [dict(type=2), dict(type=3), dict(type=-1), dict(data=(8 << 20) + 2), dict(strideBatch=4),
            dict(strideToken=130), dict(strideHead=1), dict(reserved=1)]


def _calls(ccb, cache, rows):
    big = 1 << 30
    return {
        "append": lambda: ccb.ccb_kv8_append(cache, rows, rows, 2),
        "attend": lambda: ccb.ccb_kv8_attend(cache, rows, rows, None, 4, 1, 0.1, 0, 0, 9 << 20, big),
        "evict": lambda: ccb.ccb_kv8_evict(cache, _cache(ccb, pageTable=10 << 20, lens=11 << 20, weight=12 << 20), 32,
                                           4, 4, None, 9 << 20, big),
        "read": lambda: ccb.ccb_kv8_read(cache, rows, rows, 5),
    }


def test_struct_sizes(ccb):
    assert ctypes.sizeof(ccb.ccbKv8Cache) == 7 * 8 + 2 * 8 + 8 * 4
    assert ctypes.sizeof(ccb.ccbKv8Rows) == 4 * 8 + 2 * 4


@pytest.mark.parametrize("change", BAD_CACHES, ids=str)
def test_refuses_a_bad_cache(ccb, change):
    for name, call in _calls(ccb, _cache(ccb, **change), _rows(ccb)).items():
        assert call() == ccb.CCB_ERR_INVALID_VALUE, name
    assert ccb.ccb_kv8_attend_workspace_bytes(_cache(ccb, **change), 4, 1, 0) == 0
    assert ccb.ccb_kv8_evict_workspace_bytes(_cache(ccb, **change), 32) == 0


@pytest.mark.parametrize("change", NULL_CACHES, ids=str)
def test_refuses_missing_tensors(ccb, change):
    for name, call in _calls(ccb, _cache(ccb, **change), _rows(ccb)).items():
        assert call() == ccb.CCB_ERR_NULL_POINTER, name
    for name, call in _calls(ccb, None, _rows(ccb)).items():
        assert call() == ccb.CCB_ERR_NULL_POINTER, name


@pytest.mark.parametrize("change", BAD_ROWS, ids=str)
def test_refuses_bad_rows(ccb, change):
    calls = _calls(ccb, _cache(ccb), _rows(ccb, **change))
    for name in ("append", "attend"):
        assert calls[name]() == ccb.CCB_ERR_INVALID_VALUE, name
    if change != dict(type=2):  # float rows can be read into
        assert calls["read"]() == ccb.CCB_ERR_INVALID_VALUE


def test_refuses_bad_arguments(ccb):
    c, r = _cache(ccb), _rows(ccb)
    inv, null, ok = ccb.CCB_ERR_INVALID_VALUE, ccb.CCB_ERR_NULL_POINTER, ccb.CCB_OK
    ws, big = 9 << 20, 1 << 30
    # append
    assert ccb.ccb_kv8_append(c, r, r, -1) == inv
    assert ccb.ccb_kv8_append(c, r, r, 65) == inv
    assert ccb.ccb_kv8_append(c, None, r, 1) == null
    assert ccb.ccb_kv8_append(c, r, None, 1) == null
    assert ccb.ccb_kv8_append(c, r, _rows(ccb, data=0), 1) == null
    assert ccb.ccb_kv8_append(c, r, _rows(ccb, type=1), 1) == inv
    assert ccb.ccb_kv8_append(c, r, r, 1, counts=2) == inv
    assert ccb.ccb_kv8_append(c, r, r, 1, err=2) == inv
    assert ccb.ccb_kv8_append(c, None, None, 0) == ok  # nothing to do
    assert ccb.ccb_kv8_append(_cache(ccb, batch=0, k=0), None, None, 1) == ok
    # attend
    def attend(cache=c, q=r, out=r, lse=None, heads=4, n=1, scale=0.1, window=0, acc=0, w=ws, size=big, err=None):
        return ccb.ccb_kv8_attend(cache, q, out, lse, heads, n, scale, window, acc, w, size, err)
    assert attend(heads=3) == inv and attend(heads=0) == inv and attend(n=-1) == inv and attend(window=-1) == inv
    assert attend(scale=math.nan) == inv and attend(scale=math.inf) == inv
    assert attend(q=None) == null and attend(out=None) == null and attend(out=_rows(ccb, type=1)) == inv
    assert attend(lse=2) == inv and attend(err=2) == inv
    assert attend(w=None) == null and attend(w=ws + 64) == inv
    need = ccb.ccb_kv8_attend_workspace_bytes(c, 4, 1, 0)
    assert need > 0 and attend(size=need - 1) == inv
    assert attend(cache=_cache(ccb, weight=0), acc=1) == null
    assert attend(n=0, q=None, out=None, w=None) == ok
    assert attend(cache=_cache(ccb, batch=0, k=0), q=None) == ok
    assert ccb.ccb_kv8_attend_workspace_bytes(c, 3, 1, 0) == 0
    # evict
    to = dict(pageTable=10 << 20, lens=11 << 20, weight=12 << 20)

    def evict(src=c, dst=_cache(ccb, **to), budget=32, recent=4, sinks=4, kept=None, w=ws, size=big, err=None):
        return ccb.ccb_kv8_evict(src, dst, budget, recent, sinks, kept, w, size, err)
    assert evict(budget=0) == inv and evict(recent=-1) == inv and evict(sinks=-1) == inv
    assert evict(recent=30, sinks=3) == inv and evict(budget=65) == inv
    assert evict(dst=None) == null and evict(src=_cache(ccb, weight=0)) == null and evict(w=None) == null
    for change in (dict(format=1), dict(heads=1), dict(headDim=128), dict(pageSize=32, weightStride=128),
                   dict(batch=2), dict(maxPages=1)):
        assert evict(dst=_cache(ccb, **{**to, **change})) == inv, change
    for same in ("pageTable", "lens", "weight"):  # these belong to one cache only
        assert evict(dst=_cache(ccb, **{**to, same: getattr(c, same)})) == inv, same
    assert evict(kept=2) == inv and evict(err=2) == inv and evict(w=ws + 64) == inv
    need = ccb.ccb_kv8_evict_workspace_bytes(c, 32)
    assert need > 0 and evict(size=need - 1) == inv
    assert ccb.ccb_kv8_evict_workspace_bytes(c, 0) == 0
    assert evict(src=_cache(ccb, batch=0), dst=_cache(ccb, batch=0, **to)) == ok
    # read
    assert ccb.ccb_kv8_read(c, r, r, -1) == inv
    assert ccb.ccb_kv8_read(c, None, None, 1) == null
    assert ccb.ccb_kv8_read(c, r, _rows(ccb, type=1), 1) == inv
    assert ccb.ccb_kv8_read(c, r, r, 1, first=2) == inv
    assert ccb.ccb_kv8_read(c, None, None, 0) == ok


def test_workspace_bytes_of_nothing(ccb):
    """No sequence, no query: a size all the same, and calls that do nothing."""
    long = dict(maxPages=4096, tableStride=4096, weightStride=65536)
    for extra in ({}, long):
        c, none = _cache(ccb, **extra), _cache(ccb, batch=0, **extra)
        for acc in (0, 1):
            assert ccb.ccb_kv8_attend_workspace_bytes(none, 4, 1, acc) > 0
            assert ccb.ccb_kv8_attend_workspace_bytes(c, 4, 0, acc) > 0
        assert ccb.ccb_kv8_evict_workspace_bytes(none, 32) > 0
        assert ccb.ccb_kv8_attend(none, None, None, None, 4, 1, 0.1, 0, 0, None, 0) == ccb.CCB_OK
        assert ccb.ccb_kv8_attend(c, None, None, None, 4, 0, 0.1, 0, 0, None, 0) == ccb.CCB_OK


@pytest.mark.parametrize("batch,heads,pages", [(1, 1, 1), (1, 65536, 1), (100000, 8, 2), (1, 8, 1 << 23), (4096, 1, 1 << 20)])
def test_workspace_bytes_of_extremes(ccb, batch, heads, pages):
    """Sizes far from the usual ones: a number, the larger with weights."""
    c = _cache(ccb, batch=batch, heads=heads, maxPages=pages, pageSize=128, tableStride=pages, weightStride=128 * pages)
    for group, queries in ((1, 1), (8, 5), (1, 1 << 20)):
        sizes = [ccb.ccb_kv8_attend_workspace_bytes(c, heads * group, queries, acc) for acc in (0, 1)]
        assert 128 <= sizes[0] <= sizes[1]
    assert ccb.ccb_kv8_evict_workspace_bytes(c, 128 * pages) >= 4 * batch * heads * 128 * pages


def test_class_checks_its_tensors():
    torch = pytest.importorskip("torch")
    from cross_core_barrier_amd import kv8
    f = dict(k=torch.zeros((4, 2, 16, 64), dtype=torch.int8), v=torch.zeros((4, 2, 16, 64), dtype=torch.int8),
             k_scale=torch.zeros((4, 2)), v_scale=torch.zeros((4, 2)), page_table=torch.zeros((3, 2), dtype=torch.int32),
             lens=torch.zeros(3, dtype=torch.int32), weight=torch.zeros((3, 2, 32)))
    c = kv8.Kv8Cache(**f)
    for name, bad in (("k", f["k"].float()), ("v", f["v"][:3]), ("k_scale", f["k_scale"].double()),
                      ("v_scale", f["v_scale"][:, :1]), ("page_table", f["page_table"].long()),
                      ("page_table", torch.zeros((2, 3), dtype=torch.int32).t()), ("lens", f["lens"][:2]),
                      ("weight", f["weight"][:, :, :31]), ("k", f["k"].transpose(1, 2))):
        with pytest.raises(ValueError):
            kv8.Kv8Cache(**{**f, name: bad})
    x = torch.zeros((3, 1, 2, 64), dtype=torch.bfloat16)
    for bad in (x.double(), x[:, :, :1], x[:2], x[..., :32], x[0], torch.zeros((3, 1, 64, 2)).transpose(2, 3)):
        with pytest.raises(ValueError):
            c.append(bad, bad)
    with pytest.raises(ValueError):
        c.append(x, x.half())
    with pytest.raises(ValueError):
        c.append(x, x, counts=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        c.evict(c, 8, kept=torch.zeros((3, 2, 7), dtype=torch.int32))
    with pytest.raises(ValueError):
        c.read(1, dtype=torch.int8)
    with pytest.raises(ValueError):
        c.attend_workspace(3)
    with pytest.raises(ValueError):
        kv8.Kv8Cache.allocate(4, 2, 16, 64, 1, 2, fmt="int4", device="cpu")


# --- codes under another scale, eight at a time ------------------------------------------

@pytest.fixture(scope="module")
def again(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("kv8again") / "again_driver")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-Wno-unknown-pragmas", "-I",
                    os.path.join(ROOT, "cross_core_barrier_amd", "csrc"),
                    os.path.join(HERE, "kv8", "again_driver.cpp"), "-o", exe], check=True)

    def run(fmt, v, s0, s1):
        """Values [n, 8] of codes under the scales s0 [n], as codes under s1 [n]."""
        rec = np.concatenate([v, np.stack([s0, s1], 1)], 1).astype(np.float32)
        res = subprocess.run([exe, FMT[fmt]], input=rec.tobytes(), capture_output=True, check=True)
        return np.frombuffer(res.stdout, np.uint8).reshape(-1, 8)
    return run


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_zero_codes_of_a_loud_block_stay_zero(again, fmt):
    """A token whose codes are all 0 fits every new scale, also one that its
    own block's scale is 2^128 and more times as large as."""
    s0 = 2.0 ** np.array([66, 100, 127, 64, 0, 60])
    s1 = 2.0 ** np.array([-64, -64, -64, -64, -64, 60.0])
    got = again(fmt, np.zeros((6, 8)), s0, s1)
    assert np.array_equal(oracle.values(got, fmt), np.zeros((6, 8)))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_eight_codes_round_once(again, fmt):
    """Every code at random scales and at ratios that put codes on borders."""
    rng = np.random.default_rng(3)
    codes = np.array([c for c in range(256) if c not in ((0x80,) if fmt == "int8" else (0x7F, 0xFF))], np.uint8)
    values = oracle.values(codes, fmt)
    rows, s0, s1 = [], [], []
    for trial in range(40):
        a = np.float32(rng.uniform(1, 2) * 2.0 ** int(rng.integers(-60, 60)))
        b = np.float32(a * np.float32([1.0, 2.0, 3.0, 6.0, 5.0, 4.0, 1.5, 64.0][trial] if trial < 8 else rng.uniform(1, 30)))
        rows.append(np.resize(values, (32, 8)))
        s0 += [a] * 32
        s1 += [b] * 32
    v = np.concatenate(rows)
    got = again(fmt, v, np.array(s0), np.array(s1))
    want = [[oracle.nearest_code(_exact(x) * _exact(a) / _exact(b), fmt) for x in row] for row, a, b in zip(v, s0, s1)]
    assert np.array_equal(oracle.values(got, fmt), oracle.values(np.array(want, np.uint8), fmt))


def test_attend_refuses_to_overwrite_queries_it_needs_again(ccb):
    """Weights whose scores are not kept are computed from the queries after
    the results are written."""
    inv, big = ccb.CCB_ERR_INVALID_VALUE, 1 << 40

    def attend(cache, out, n, acc):
        q = _rows(ccb, strideBatch=1 << 20, strideToken=256)
        return ccb.ccb_kv8_attend(cache, q, out, None, 4, n, 0.1, 0, acc, 9 << 20, big)
    same = _rows(ccb, strideBatch=1 << 20, strideToken=256)
    assert attend(_cache(ccb), same, 33, 1) == inv  # 66 rows
    wide = dict(maxPages=1 << 13, tableStride=1 << 13, weightStride=1 << 17)
    assert attend(_cache(ccb, **wide), same, 10, 1) == inv  # 20 rows, 63 MB of scores
    # rows that begin alike and then part
    for other in (dict(strideBatch=1 << 21, strideToken=256), dict(strideBatch=1 << 20, strideToken=512),
                  dict(strideBatch=1 << 20, strideToken=256, strideHead=128)):
        assert attend(_cache(ccb), _rows(ccb, **other), 2, 0) == inv, other


@pytest.fixture
def cpu_cache(monkeypatch):
    """A whole cache on the CPU, and what reached the library of it: its entry
    points record their names and enqueue nothing."""
    torch = pytest.importorskip("torch")
    from cross_core_barrier_amd import ccb, kv8
    reached = []
    for name in ("append", "attend", "evict", "read"):
        monkeypatch.setattr(ccb, f"ccb_kv8_{name}", lambda *a, _n=name: reached.append(_n) or 0)
    monkeypatch.setattr(kv8, "_current_stream", lambda index: 0)
    make = lambda: kv8.Kv8Cache.allocate(8, 2, 16, 64, 3, 2, "int8", weights=True, device="cpu")  # noqa: E731
    x = torch.zeros((3, 1, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((3, 1, 4, 64), dtype=torch.bfloat16)
    calls = {
        "append": lambda c: c.append(x, x), "attend": lambda c: c.attend(q, accumulate=True),
        "evict": lambda c: c.evict(make(), 8, recent=2), "read": lambda c: c.read(5),
        "attend_workspace": lambda c: c.attend_workspace(4), "evict_workspace": lambda c: c.evict_workspace(8),
    }
    return make, calls, reached


def test_no_call_on_cpu_tensors_reaches_a_kernel(cpu_cache):
    """Well-shaped calls on a cache in host memory are refused before the
    library gets its addresses."""
    make, calls, reached = cpu_cache
    for name, call in calls.items():
        with pytest.raises(ValueError, match="not on a GPU"):
            call(make())
        assert reached == [], name


def test_calls_run_on_the_cache_s_device(cpu_cache, monkeypatch):
    """The entry points act on the current device: the class makes the cache's
    current for the call, and leaves it alone where it is already."""
    import contextlib
    from cross_core_barrier_amd import ccb, kv8
    torch = pytest.importorskip("torch")
    make, calls, reached = cpu_cache
    current = [0]

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before
    where = []
    for name in ("append", "attend", "evict", "read"):
        def entry(*a):
            where.append(current[0])
            return 0
        monkeypatch.setattr(ccb, f"ccb_kv8_{name}", entry)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(kv8, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(kv8.Kv8Cache, "_on_gpu", lambda self: None)  # the CPU's index, -1, plays another GPU's
    for other in (0, -1):
        current[0] = other
        for name in ("append", "attend", "evict", "read"):
            del where[:]
            calls[name](make())
            assert where == [-1] and current[0] == other, name


def test_tensors_of_a_cache_change_in_place_only(cpu_cache):
    """The library holds their addresses: another tensor in their place would
    leave it with freed memory."""
    make, _, _ = cpu_cache
    c = make()
    for name in ("k", "v", "k_scale", "v_scale", "page_table", "lens", "weight", "err", "heads", "head_dim", "batch",
                 "device", "_c", "_index"):
        before = getattr(c, name)
        with pytest.raises(AttributeError):
            setattr(c, name, before + 1 if isinstance(before, int) else None)
        assert getattr(c, name) is before, name
    at = c.lens.data_ptr()
    c.lens += 1
    c.lens[0] = 7
    assert c.lens.tolist() == [7, 1, 1] and c.lens.data_ptr() == at
    assert c._c.lens == at


def test_refuses_more_than_a_launch_holds(ccb):
    """2^32 threads and more: refused with nothing enqueued, not by the launch
    of one of a call's kernels after others."""
    inv, big = ccb.CCB_ERR_INVALID_VALUE, (1 << 63) - 1
    wide = dict(heads=64, batch=4096, maxPages=1 << 16, tableStride=1 << 16, weightStride=1 << 23, pageSize=128)
    c, r = _cache(ccb, **wide), _rows(ccb)
    out = _rows(ccb, data=13 << 20)
    assert ccb.ccb_kv8_append(c, r, r, 1 << 15) == inv  # 2^18 pairs of a sequence and a head, 2^8 pages, 2 sides
    assert ccb.ccb_kv8_read(c, out, out, 1 << 15) == inv
    assert ccb.ccb_kv8_read(c, out, None, 1 << 15) == inv
    to = _cache(ccb, **{**wide, "pageTable": 10 << 20, "lens": 11 << 20, "weight": 12 << 20})
    assert ccb.ccb_kv8_evict(c, to, 1 << 15, 4, 4, None, 9 << 20, big) == inv
    for acc in (0, 1):  # 2^11 rows: 2^7 tiles of them
        assert ccb.ccb_kv8_attend(c, r, out, None, 64, 1 << 11, 0.1, 0, acc, 9 << 20, big) == inv
    # so many pairs that their number passes 31 bits
    far = _cache(ccb, **{**wide, "heads": 65536, "batch": 1 << 30})
    assert ccb.ccb_kv8_append(far, r, r, 1) == inv and ccb.ccb_kv8_read(far, out, out, 1) == inv
    assert ccb.ccb_kv8_attend(far, r, out, None, 65536, 1, 0.1, 0, 0, 9 << 20, big) == inv


def test_refuses_tensors_that_ask_for_a_gradient(cpu_cache, monkeypatch):
    """None is computed: the results would silently have no history."""
    torch = pytest.importorskip("torch")
    from cross_core_barrier_amd import kv8
    make, _, reached = cpu_cache
    monkeypatch.setattr(kv8, "_current_device", lambda: -1)
    monkeypatch.setattr(kv8.Kv8Cache, "_on_gpu", lambda self: None)  # no kernel runs
    c = make()
    x, q = torch.zeros((3, 1, 2, 64)).half(), torch.zeros((3, 1, 4, 64)).half()
    asks_x, asks_q = x.clone().requires_grad_(), q.clone().requires_grad_()
    for call in (lambda: c.append(asks_x, x), lambda: c.append(x, asks_x), lambda: c.attend(asks_q)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    assert reached == []
    with torch.no_grad():
        c.append(asks_x, asks_x)
        c.attend(asks_q)
    c.append(asks_x.detach(), x)
    assert reached == ["append", "attend", "append"]


def test_session_refuses_what_does_not_fit():
    """A cut that leaves no room for the next token, and prompts that pass the
    limit or hold nothing, before any page is taken."""
    torch = pytest.importorskip("torch")
    from cross_core_barrier_amd.kv8_decode import Session
    for budget in (96, 97, 0, -1):
        with pytest.raises(ValueError):
            Session(batch=2, limit=96, budget=budget)
    s = Session.__new__(Session)  # the checks need no device
    s.batch, s.limit = 2, 96
    for lens in ([97, 5], [5, 0], [5], [5, 5, 5]):
        with pytest.raises(ValueError):
            s.prefill([torch.zeros((n, 64)) for n in lens])
