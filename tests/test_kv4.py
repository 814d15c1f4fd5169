"""The 4-bit key/value cache on the CPU: the oracle on worked values, refusals
of the C entry points before anything is enqueued, and the class's checks."""

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import kv4 as oracle


@pytest.fixture(scope="module")
def ccb():
    from cross_core_barrier_amd import ccb as lib
    return lib


def test_oracle_codes():
    assert [oracle.e2m1_value(c) for c in range(8)] == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert [oracle.e2m1_value(c) for c in range(8, 16)] == [0, -0.5, -1, -1.5, -2, -3, -4, -6]
    worked = {0.25: 0, 0.26: 1, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 2.51: 5, 3.5: 6, 5: 6, 5.01: 7, 7: 7, 100: 7}
    for x, code in worked.items():
        assert oracle.nearest_code(Fraction(x)) == code and oracle.nearest_code(Fraction(-x)) == (code | 8 if x else 0)


def test_oracle_scales():
    for a, e in ((7, 0), (7.01, 1), (6, 0), (3.5, -1), (3.6, 0), (0, -64), (2.0 ** -70, -64), (1.75, -2), (1.76, -1),
                 (3.3e38, 125), (7 * 2.0 ** 100, 100)):
        assert oracle.exponent(Fraction(a)) == e, a


def test_oracle_rounds_like_exact_fractions():
    rng = np.random.default_rng(1)
    x = (rng.normal(0, 1, (40, 64)) * 2.0 ** rng.integers(-70, 60, (40, 1))).astype(np.float32)
    x.view(np.uint32)[...] &= 0xFFFF0000  # bf16
    x[3] = 0
    x[4, 5], x[4, 40], x[5, 7] = np.inf, -np.inf, np.nan
    codes, scales = oracle.quantise(x.astype(np.float64))
    for i in range(40):
        for g in range(2):
            row = x[i, 32 * g:32 * g + 32]
            e = oracle.exponent(max((Fraction(abs(float(v))) for v in row if np.isfinite(v)), default=Fraction(0)))
            assert scales[i, g] == e + 127
            for d, v in enumerate(row):
                got = (codes[i, 16 * g + d // 2] >> (4 * (d % 2))) & 15
                if np.isnan(v):
                    assert got == 0
                elif np.isinf(v):
                    assert got == (7 if v > 0 else 15)
                else:
                    assert got & 7 == oracle.nearest_code(Fraction(float(v)) / Fraction(2) ** e) & 7
                    # nothing is off by more than half a step (at the top 1 * 2^e)
                    assert abs(oracle.e2m1_value(int(got)) - float(v) / 2.0 ** e) <= 1


def test_oracle_attention_on_one_token():
    c = dict(k=np.full((2, 1, 16, 16), 0x22, np.uint8), v=np.full((2, 1, 16, 16), 0x75, np.uint8),
             ks=np.full((2, 1, 16, 1), 127, np.uint8), vs=np.full((2, 1, 16, 1), 128, np.uint8),
             table=np.array([[1]], np.int32), lens=np.array([1], np.int32))
    out, lse, _, _ = oracle.attend(c, np.ones((1, 1, 2, 32)), 0.5, 0)
    assert np.array_equal(out[0, 0, 0], [6.0, 12.0] * 16) and lse[0, 0, 0] == 16
    out, lse, _, _ = oracle.attend(c, np.ones((1, 2, 1, 32)), 0.5, 0)
    assert not out[0, 0].any() and lse[0, 0, 0] == -math.inf


def _cache(ccb, **change):
    f = dict(k=1 << 20, v=2 << 20, kScale=3 << 20, vScale=4 << 20, pageTable=5 << 20, lens=6 << 20, tableStride=4,
             numPages=8, heads=2, pageSize=16, headDim=64, batch=3, maxPages=4)
    f.update(change)
    return ccb.ccbKv4Cache(**f)


def _rows(ccb, **change):
    f = dict(data=8 << 20, strideBatch=256, strideToken=128, strideHead=64, type=0, reserved=0)
    f.update(change)
    return ccb.ccbKv8Rows(**f)


def _calls(ccb, cache, rows):
    big = 1 << 30
    return {
        "append": lambda: ccb.ccb_kv4_append(cache, rows, rows, 2, 10 << 20),
        "attend": lambda: ccb.ccb_kv4_attend(cache, rows, rows, None, 4, 1, 0.1, 0, 9 << 20, big),
        "read": lambda: ccb.ccb_kv4_read(cache, rows, rows, 5),
    }


def test_struct_size(ccb):
    assert ctypes.sizeof(ccb.ccbKv4Cache) == 6 * 8 + 8 + 6 * 4


BAD_CACHES = [dict(pageSize=0), dict(pageSize=8), dict(pageSize=24), dict(pageSize=256), dict(headDim=32),
              dict(headDim=80), dict(headDim=512), dict(numPages=0), dict(numPages=1 << 27), dict(heads=0), dict(heads=65537), dict(batch=-1),
              dict(maxPages=0), dict(maxPages=(1 << 26) + 1, tableStride=1 << 27), dict(tableStride=3), dict(k=8),
              dict(v=8), dict(kScale=8), dict(vScale=4), dict(pageTable=2), dict(lens=2)]


@pytest.mark.parametrize("change", BAD_CACHES, ids=str)
def test_refuses_a_bad_cache(ccb, change):
    for name, call in _calls(ccb, _cache(ccb, **change), _rows(ccb)).items():
        assert call() == ccb.CCB_ERR_INVALID_VALUE, name
    assert ccb.ccb_kv4_attend_workspace_bytes(_cache(ccb, **change), 4, 1) == 0


@pytest.mark.parametrize("name", ["k", "v", "kScale", "vScale", "pageTable", "lens"])
def test_refuses_missing_tensors(ccb, name):
    for what, call in _calls(ccb, _cache(ccb, **{name: 0}), _rows(ccb)).items():
        assert call() == ccb.CCB_ERR_NULL_POINTER, what
    for what, call in _calls(ccb, None, _rows(ccb)).items():
        assert call() == ccb.CCB_ERR_NULL_POINTER, what


@pytest.mark.parametrize("change", [dict(data=4), dict(strideBatch=4), dict(strideToken=12), dict(strideHead=63),
                                    dict(type=2), dict(type=-1), dict(type=3), dict(reserved=1)], ids=str)
def test_refuses_bad_rows(ccb, change):
    calls = _calls(ccb, _cache(ccb), _rows(ccb, **change))
    for name in ("append", "attend"):
        assert calls[name]() == ccb.CCB_ERR_INVALID_VALUE, name
    if change != dict(type=2):  # float rows can be read into
        assert calls["read"]() == ccb.CCB_ERR_INVALID_VALUE


def test_refuses_bad_arguments(ccb):
    c, r, slots = _cache(ccb), _rows(ccb), 10 << 20
    inv, null, ok = ccb.CCB_ERR_INVALID_VALUE, ccb.CCB_ERR_NULL_POINTER, ccb.CCB_OK
    # append
    assert ccb.ccb_kv4_append(c, r, r, -1, slots) == inv
    assert ccb.ccb_kv4_append(c, r, r, (1 << 30) + 1, slots) == inv
    assert ccb.ccb_kv4_append(c, None, r, 1, slots) == null and ccb.ccb_kv4_append(c, r, None, 1, slots) == null
    assert ccb.ccb_kv4_append(c, r, r, 1, None) == null and ccb.ccb_kv4_append(c, r, r, 1, 12) == inv
    assert ccb.ccb_kv4_append(c, _rows(ccb, data=0), r, 1, slots) == null
    assert ccb.ccb_kv4_append(c, r, _rows(ccb, type=1), 1, slots) == inv
    assert ccb.ccb_kv4_append(c, r, r, 1, slots, err=2) == inv
    assert ccb.ccb_kv4_append(c, None, None, 0, None) == ok  # nothing to do
    assert ccb.ccb_kv4_append(_cache(ccb, batch=0, k=0), None, None, 1, None) == ok

    # attend
    def attend(cache=c, q=r, out=r, lse=None, heads=4, n=1, scale=0.1, window=0, w=9 << 20, size=1 << 30, err=None):
        return ccb.ccb_kv4_attend(cache, q, out, lse, heads, n, scale, window, w, size, err)
    assert attend(heads=3) == inv and attend(heads=0) == inv and attend(n=-1) == inv and attend(window=-1) == inv
    assert attend(scale=math.nan) == inv and attend(scale=math.inf) == inv and attend(n=1 << 20) == inv
    assert attend(q=None) == null and attend(out=None) == null and attend(out=_rows(ccb, type=1)) == inv
    assert attend(lse=2) == inv and attend(err=2) == inv and attend(w=None) == null and attend(w=(9 << 20) + 64) == inv
    need = ccb.ccb_kv4_attend_workspace_bytes(c, 4, 1)
    assert need > 0 and attend(size=need - 1) == inv
    long = _cache(ccb, maxPages=1 << 20, tableStride=1 << 20)
    need = ccb.ccb_kv4_attend_workspace_bytes(long, 4, 1)
    assert need > 1 << 16 and attend(cache=long, size=need - 1) == inv
    assert attend(n=0, q=None, out=None, w=None) == ok
    assert attend(cache=_cache(ccb, batch=0, k=0), q=None) == ok
    assert ccb.ccb_kv4_attend_workspace_bytes(c, 3, 1) == 0
    # out over q: with the same strides only
    for name, wide in (("strideBatch", dict(n=1)), ("strideToken", dict(n=2)), ("strideHead", dict(n=1))):
        assert attend(out=_rows(ccb, **{name: 512}), **wide) == inv, name
    # read
    assert ccb.ccb_kv4_read(c, r, r, -1) == inv and ccb.ccb_kv4_read(c, None, None, 1) == null
    assert ccb.ccb_kv4_read(c, r, _rows(ccb, type=1), 1) == inv and ccb.ccb_kv4_read(c, r, r, 1, first=2) == inv
    assert ccb.ccb_kv4_read(c, None, None, 0) == ok


def test_refuses_more_than_a_launch_holds(ccb):
    inv, big = ccb.CCB_ERR_INVALID_VALUE, (1 << 63) - 1
    c = _cache(ccb, heads=64, batch=4096, maxPages=1 << 16, tableStride=1 << 16, pageSize=128)
    r, out = _rows(ccb), _rows(ccb, data=13 << 20)
    assert ccb.ccb_kv4_append(c, r, r, 1 << 30, 10 << 20) == inv
    assert ccb.ccb_kv4_read(c, out, out, 1 << 15) == inv
    assert ccb.ccb_kv4_attend(c, r, out, None, 64, 1 << 11, 0.1, 0, 9 << 20, big) == inv  # 2^7 tiles of rows
    far = _cache(ccb, heads=65536, batch=1 << 30)
    assert ccb.ccb_kv4_read(far, out, out, 1) == inv
    assert ccb.ccb_kv4_attend(far, r, out, None, 65536, 1, 0.1, 0, 9 << 20, big) == inv
    ccb.ccb_kv4_attend_workspace_bytes(far, 65536, 1)  # whatever it says, it says it


@pytest.mark.parametrize("queries", [0, 1])
@pytest.mark.parametrize("batch,heads,pages", [(1, 1, 1), (1 << 20, 64, 1 << 26), (1, 65536, 1 << 26), (0, 1, 1)])
def test_workspace_bytes_of_extremes(ccb, batch, heads, pages, queries):
    c = _cache(ccb, batch=batch, heads=heads, maxPages=pages, tableStride=pages)
    n = ccb.ccb_kv4_attend_workspace_bytes(c, heads, queries)
    assert 128 <= n <= 128 + max(4096, batch * heads) * 66 * 4 + 256


torch = pytest.importorskip("torch")


def test_class_checks_its_tensors():
    from cross_core_barrier_amd import kv4
    k, s = torch.zeros((5, 2, 16, 32), dtype=torch.uint8), torch.zeros((5, 2, 16, 2), dtype=torch.uint8)
    table, lens = torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    good = dict(k=k, v=k.clone(), k_scale=s, v_scale=s.clone(), page_table=table, lens=lens)
    assert kv4.Kv4Cache(**good).head_dim == 64
    for change in (dict(k=k.float()), dict(k=k[0]), dict(v=k[:4]), dict(v=k.to(torch.int8)), dict(k_scale=s[:4]),
                   dict(k_scale=s.float()), dict(v_scale=s[..., :1]), dict(page_table=table.long()),
                   dict(page_table=table[0]), dict(page_table=torch.zeros((4, 3), dtype=torch.int32).t()),
                   dict(lens=lens[:2]), dict(lens=lens.long()), dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)),
                   dict(lens=lens.to("meta"))):
        with pytest.raises(ValueError):
            kv4.Kv4Cache(**{**good, **change})
    with pytest.raises(ValueError):
        kv4.Kv4Cache.allocate(5, 2, 16, 80, 3, 4, device="cpu")
    c = kv4.Kv4Cache(**good)
    for name in ("k", "v", "k_scale", "v_scale", "page_table", "lens", "err", "heads", "_c", "_index"):
        with pytest.raises(AttributeError):
            setattr(c, name, None)
    c.lens += 1
    assert c.lens.tolist() == [1, 1, 1]


@pytest.fixture
def cpu_cache(monkeypatch):
    """A whole cache on the CPU, and what reached the library of it: its entry
    points record their names and enqueue nothing."""
    from cross_core_barrier_amd import ccb, kv4, kv8
    reached = []
    for name in ("append", "attend", "read"):
        monkeypatch.setattr(ccb, f"ccb_kv4_{name}", lambda *a, _n=name: reached.append(_n) or 0)
    monkeypatch.setattr(kv8, "_current_stream", lambda index: 0)
    monkeypatch.setattr(kv8, "_current_device", lambda: -1)
    return kv4.Kv4Cache.allocate(8, 2, 16, 64, 3, 2, device="cpu"), reached


def test_no_call_on_cpu_tensors_reaches_a_kernel(cpu_cache):
    c, reached = cpu_cache
    x, q = torch.zeros((3, 2, 64)).half(), torch.zeros((3, 1, 4, 64)).half()
    slots = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: c.append(x, x, slots), lambda: c.attend(q), lambda: c.read(5), lambda: c.attend_workspace(4)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()
    assert reached == []


def test_class_checks_its_rows(cpu_cache, monkeypatch):
    from cross_core_barrier_amd import kv4
    c, reached = cpu_cache
    monkeypatch.setattr(kv4.Kv4Cache, "_on_gpu", lambda self: None)  # the CPU's index, -1, plays a GPU's
    x, q = torch.zeros((3, 2, 64)).half(), torch.zeros((3, 1, 4, 64)).half()
    slots = torch.zeros(3, dtype=torch.int64)
    asks_x, asks_q = x.clone().requires_grad_(), q.clone().requires_grad_()
    bad = [lambda: c.append(x[0], x, slots), lambda: c.append(x, x[:2], slots), lambda: c.append(x, x.bfloat16(), slots),
           lambda: c.append(x.float(), x.float(), slots), lambda: c.append(x, x, slots[:2]),
           lambda: c.append(x, x, slots.int()), lambda: c.append(x, x, torch.zeros(6, dtype=torch.int64)[::2]),
           lambda: c.append(x[:, :1], x[:, :1], slots), lambda: c.append(x[..., :32], x[..., :32], slots),
           lambda: c.attend(q[0]), lambda: c.attend(q[:2]), lambda: c.attend(q[..., ::2]),
           lambda: c.attend(q, out=q.bfloat16()), lambda: c.attend(q, out=torch.zeros((3, 2, 4, 64)).half()),
           lambda: c.attend(q, lse=torch.zeros((3, 1, 4)).double()), lambda: c.attend(q, lse=torch.zeros((3, 1, 5))),
           lambda: c.attend_workspace(3), lambda: c.read(5, first=torch.zeros(2, dtype=torch.int32)),
           lambda: c.read(5, dtype=torch.float64)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.append(asks_x, x, slots), lambda: c.append(x, asks_x, slots), lambda: c.attend(asks_q)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    assert reached == []
    with torch.no_grad():
        c.append(asks_x, x, slots)
        c.attend(asks_q)
    c.append(x, x, slots)
    c.append(x[:0], x[:0], slots[:0])
    c.read(5)
    assert reached == ["append", "attend", "append", "append", "read"]


def test_calls_run_on_their_tensors_device(monkeypatch):
    """The entry points act on the current device: the classes make their own
    current for the call, and leave it alone where it is already."""
    import contextlib
    from cross_core_barrier_amd import ccb, kv4, kv8, pages
    current, where = [0], []

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before
    for name in ("kv4_append", "kv4_attend", "kv4_read", "pages_trim", "pages_grow"):
        def entry(*a):
            where.append(current[0])
            return 0
        monkeypatch.setattr(ccb, f"ccb_{name}", entry)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(kv8, "_current_device", lambda: current[0])
    monkeypatch.setattr(kv8, "_current_stream", lambda index: 0)
    for cls in (kv4.Kv4Cache, pages.PagePool):
        monkeypatch.setattr(cls, "_on_gpu", lambda self: None)  # the CPU's index, -1, plays another GPU's
    c, pool = kv4.Kv4Cache.allocate(8, 2, 16, 64, 3, 2, device="cpu"), pages.PagePool.allocate(8, 16, device="cpu")
    x, q, slots = torch.zeros((3, 2, 64)).half(), torch.zeros((3, 1, 4, 64)).half(), torch.zeros(3, dtype=torch.int64)
    n, maps = torch.zeros(3, dtype=torch.int32), pool.maps(3, 5)
    for other in (0, -1):
        current[0] = other
        for call in (lambda: c.append(x, x, slots), lambda: c.attend(q), lambda: c.read(5),
                     lambda: pool.trim(c.page_table, c.lens, n), lambda: pool.grow(c.page_table, c.lens, n, maps)):
            del where[:]
            call()
            assert where == [-1] and current[0] == other


def test_session_refuses_what_does_not_fit():
    """Before any page is taken."""
    from cross_core_barrier_amd.kv8_decode import PooledSession
    with pytest.raises(ValueError):
        PooledSession(batch=2, limit=100, page_size=16, pages=6)  # 7 for one request
    s = PooledSession.__new__(PooledSession)  # the checks need no device
    s.batch, s.limit = 3, 96
    for seats, lens in (([0], [97]), ([0], [0]), ([0, 1], [5]), ([1, 1], [5, 5])):
        with pytest.raises(ValueError):
            s.sit(seats, [torch.zeros((n, 64)) for n in lens])


def test_session_refuses_seats_that_are_not_free():
    """A prompt in a seat that is taken would go on behind the one that sits there."""
    from cross_core_barrier_amd.kv8_decode import PooledSession
    s = PooledSession.__new__(PooledSession)  # the checks need no device
    s.batch, s.limit, s.taken = 3, 96, {1}
    for seats in ([1], [0, 1], [3], [-1]):
        with pytest.raises(ValueError, match="somebody sits"):
            s.sit(seats, [torch.zeros((5, 64)) for _ in seats])
    for seats in ([0], [0, 1], [-2]):
        with pytest.raises(ValueError, match="somebody sits"):
            s.leave(seats)
    assert s.taken == {1}


@pytest.mark.parametrize("prompt", ["100", "101"])
def test_decode_command_refuses_prompts_at_the_limit(prompt):
    """Such a request would sit, with no step left to it, in a seat taken for free."""
    from cross_core_barrier_amd import kv8_decode
    with pytest.raises(ValueError, match="--prompt"):
        kv8_decode.main(["--format", "mxfp4", "--batch", "2", "--limit", "100", "--prompt", prompt])


@pytest.mark.parametrize("window", [-1, 2 ** 31, 2 ** 32 + 5])
def test_windows_past_32_bits_are_refused(monkeypatch, window):
    """2^32 + 5 tokens would arrive as 5."""
    from cross_core_barrier_amd import kv4
    monkeypatch.setattr(kv4.Kv4Cache, "_on_gpu", lambda self: None)
    c = kv4.Kv4Cache.allocate(8, 2, 16, 64, 3, 2, device="cpu")
    with pytest.raises(ValueError, match="window"):
        c.attend(torch.zeros((3, 1, 4, 64)).half(), window=window)


def test_session_refuses_prompts_before_pages_are_taken():
    """Behind grow a refusal would leave the prompt's tokens in a seat that counts
    as free, and the next one's behind them."""
    from cross_core_barrier_amd.kv8_decode import PooledSession

    class Calls:
        def __getattr__(self, name):
            raise AssertionError(f"reached {name}")
    s = PooledSession.__new__(PooledSession)
    s.batch, s.limit, s.taken = 3, 96, set()
    s.x = torch.zeros((3, 64), dtype=torch.bfloat16)
    s.pool = s.cache = s.layer = Calls()
    good = torch.zeros((5, 64), dtype=torch.bfloat16)
    for bad in (good[:, :32], good.half(), good.to("meta"), good[None], good.clone().requires_grad_()):
        for prompts in ([bad], [good, bad]):
            with pytest.raises(ValueError, match="prompts"):
                s.sit(list(range(len(prompts))), prompts)
    assert s.sit([], []) == [] and s.taken == set()
    with pytest.raises(AssertionError, match="reached maps"):
        s.sit([0], [good])


def test_session_projects_before_pages_are_taken():
    """(which may fail for want of memory)"""
    from cross_core_barrier_amd.kv8_decode import PooledSession

    class Pool:
        def maps(self, batch, tokens):
            return None

        def grow(self, *a):
            raise AssertionError("pages are taken")

    class Layer:
        def project(self, rows):
            raise RuntimeError("no memory")
    s = PooledSession.__new__(PooledSession)
    s.batch, s.limit, s.taken, s.pool, s.layer = 3, 96, set(), Pool(), Layer()
    s.x = torch.zeros((3, 64))
    with pytest.raises(RuntimeError, match="no memory"):
        s.sit([1], [torch.zeros((5, 64))])


@pytest.mark.parametrize("batch,queries", [(1023, 1024), (1024, 1024), (64, 16384), (2048, 512), (2047, 1024)])
def test_accepts_what_a_launch_holds(ccb, batch, queries):
    """Up to 2^27 rows (fewer than 2^23 workgroups of 512 threads, 16 rows each) where
    nothing is cut: the kernel that joins runs, which holds fewer than 2^26, is not
    started then."""
    c = _cache(ccb, heads=8, batch=batch, headDim=128, maxPages=8, tableStride=8, pageSize=128)
    r, out, inv = _rows(ccb), _rows(ccb, data=13 << 20), ccb.CCB_ERR_INVALID_VALUE
    size = ccb.ccb_kv4_attend_workspace_bytes(c, 64, queries)
    assert size == 128
    if torch.cuda.is_available():
        pytest.skip("what is accepted would be enqueued")
    assert ccb.ccb_kv4_attend(c, r, out, None, 64, queries, 0.1, 0, 9 << 20, size) not in (inv, ccb.CCB_OK)
    more = _cache(ccb, heads=8, batch=2048, headDim=128, maxPages=8, tableStride=8, pageSize=128)
    assert ccb.ccb_kv4_attend(more, r, out, None, 64, 1024, 0.1, 0, 9 << 20, size) == inv
    # 2^26 rows of sequences that may be cut into more runs than the last of them joins
    long = _cache(ccb, heads=1, batch=1 << 16, headDim=128, maxPages=1 << 14, tableStride=1 << 14, pageSize=128)
    assert ccb.ccb_kv4_attend(long, r, out, None, 64, 16, 0.1, 0, 9 << 20, 1 << 62) == inv


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """Of 2^32 + 5 the library would get 5."""
    from cross_core_barrier_amd import ccb, kv4, kv8

    def reached(*a):
        raise AssertionError("reached the library")
    for name in ("kv4_append", "kv8_append", "kv4_attend_workspace_bytes", "kv8_attend", "kv8_attend_workspace_bytes",
                 "kv8_evict", "kv8_evict_workspace_bytes", "kv4_read", "kv8_read"):
        monkeypatch.setattr(ccb, f"ccb_{name}", reached)
    monkeypatch.setattr(kv8.OnDevice, "_on_gpu", lambda self: None)
    monkeypatch.setattr(kv8, "_current_stream", lambda index: 0)
    monkeypatch.setattr(kv8, "_current_device", lambda: -1)
    big = 2 ** 32 + 5
    c4 = kv4.Kv4Cache.allocate(8, 2, 16, 64, 3, 2, device="cpu")
    c8, to = (kv8.Kv8Cache.allocate(8, 2, 16, 64, 3, 2, "int8", weights=True, device="cpu") for _ in range(2))
    row, rows = torch.zeros((1, 2, 64)).half(), torch.zeros((3, 1, 2, 64)).half()
    slots, q = torch.zeros(1, dtype=torch.int64), torch.zeros((3, 1, 4, 64)).half()
    for call in (lambda: c4.append(row.expand(big, 2, 64), row.expand(big, 2, 64), slots),
                 lambda: c8.append(rows.expand(3, big, 2, 64), rows.expand(3, big, 2, 64)),
                 lambda: c4.attend_workspace(big), lambda: c4.attend_workspace(4, big),
                 lambda: c8.attend_workspace(big), lambda: c8.attend_workspace(4, big),
                 lambda: c8.attend(q, window=big), lambda: c8.attend(q, window=-big), lambda: c8.evict_workspace(big),
                 lambda: c8.evict(to, big), lambda: c8.evict(to, 5, recent=big), lambda: c8.evict(to, 5, sinks=2 ** 31),
                 lambda: c4.read(big), lambda: c8.read(big)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    with pytest.raises(AssertionError, match="library"):
        c8.append(rows, rows)
