"""The 4-bit key/value cache on the GPU against the oracle in 64 bits
(oracle/kv4.py).  Codes and scales are compared exactly; attention within
bounds counted from its roundings (see _bounds).  Unused pages, and slots past
a sequence's end, hold NaN scales."""

import math

import numpy as np
import pytest

from oracle import kv4 as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _say(msg):
    print(f"[gpu case] {msg}", flush=True)


@pytest.fixture(scope="module")
def kv4():
    from cross_core_barrier_amd import ccb, kv4 as module
    st, _, _, _ = ccb.ccb_device_info()
    assert st == 0, ccb.ccb_status_string(st)
    return module


def _host(rng, lens, heads, P, D, width=None, extra=3, low=124, high=127):
    """A cache on the host: pages in random order, the bytes no token owns all
    ones (NaN scales)."""
    batch = len(lens)
    width = width or max(1, -(-max(lens) // P)) + 1
    pages = batch * width + extra
    c = dict(lens=np.array(lens, np.int32),
             table=rng.permutation(pages)[:batch * width].astype(np.int32).reshape(batch, width))
    for w in ("k", "v"):
        c[w] = np.full((pages, heads, P, D // 2), 255, np.uint8)
        c[w + "s"] = np.full((pages, heads, P, D // 32), 255, np.uint8)
    for b, n in enumerate(lens):
        for number in range(-(-n // P)):
            page = c["table"][b, number]
            slots = min(P, n - number * P)
            for w in ("k", "v"):
                c[w][page, :, :slots] = rng.integers(0, 256, (heads, slots, D // 2))
                c[w + "s"][page, :, :slots] = rng.integers(low, high, (heads, slots, D // 32))
    return c


def _device(kv4, c):
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return kv4.Kv4Cache(up(c["k"]), up(c["v"]), up(c["ks"]), up(c["vs"]), up(c["table"]), up(c["lens"]))


def _spread(x, spare, dim):
    """The same values with strides: a slice of a wider tensor."""
    shape = list(x.shape)
    shape[dim] += spare
    wide = torch.zeros(shape, dtype=x.dtype, device=x.device)
    wide.narrow(dim, 1, x.shape[dim]).copy_(x)
    return wide.narrow(dim, 1, x.shape[dim])


def _bounds(D, tokens, seen_mag, big, lse):
    """What fp32 attention over exact 4-bit products may be off by, u half a
    step.  A score is a sum of D exact products (2 D with a query in two
    pieces), each addition in the matrix cores off by a whole step at most
    (they may cut instead of rounding), then times scale * log2 e (its two
    roundings and one more): off by at most (4 D + 6) u of sum |q k| scale
    (`big`).  Its weight is off, relatively, by that, by as much for the
    maximum it is compared with, by the roundings of the exponent (of at most
    |s - m| <= 2 big, in powers of two) and by the exponential's own error (4);
    in the sum of values it stands as two pieces, 64 u, of which each is
    added in a whole step; sums over the tokens add another `tokens` at worst,
    and the joins of waves and runs a few."""
    u = 2.0 ** -24
    ds = (4 * D + 6) * u * big
    rel = 2 * ds + (8 * big + 80 + 6 * tokens) * u
    return rel, ds + rel + 6 * u * np.abs(np.where(np.isfinite(lse), lse, 0)), rel[..., None] * seen_mag


def _compare(D, dtype, lens, want, lse, mag, big, got, got_lse):
    _, tol_lse, tol = _bounds(D, max(max(lens), 1), mag, big, lse)
    eps = torch.finfo(TYPES[dtype]).eps / 2
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0  # half a step of fp16's subnormals
    y = got.double().cpu().numpy()
    assert np.all(np.abs(y - want) <= tol + eps * (np.abs(want) + tol) + tiny)
    z = got_lse.double().cpu().numpy()
    empty = np.isinf(lse)
    assert np.array_equal(np.isneginf(z), empty)
    assert np.all(y[empty] == 0)
    assert np.all(np.abs(np.where(empty, 0, z) - np.where(empty, 0, lse)) <= tol_lse + 1e-45)


def _attend_case(kv4, seed, dtype, lens, heads, group, D, P, queries=1, window=0, scale=None, q_size=1.0, c=None,
                 strided=False, **kw):
    rng = np.random.default_rng(seed)
    c = c or _host(rng, lens, heads, P, D)
    cache = _device(kv4, c)
    q = torch.from_numpy(rng.normal(0, q_size, (len(lens), queries, heads * group, D))).to(TYPES[dtype])
    scale = 1 / math.sqrt(D) if scale is None else scale
    want = oracle.attend(c, q.double().numpy(), float(np.float32(scale)), window)
    dq, out = q.cuda(), None
    if strided:
        dq = _spread(dq, 3, 2)
        out = _spread(torch.zeros_like(q, device="cuda"), 2, 2)
    got, got_lse = cache.attend(dq, scale=scale, window=window, out=out, **kw)
    torch.cuda.synchronize()
    _compare(D, dtype, lens, *want, got, got_lse)
    cache.check()
    return cache, dq, got, got_lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,P", [(64, 16), (64, 128), (96, 32), (96, 64), (96, 16), (128, 64), (128, 16), (192, 128),
                                 (192, 32), (192, 16), (256, 16), (256, 64)])
def test_attend_sizes(kv4, dtype, D, P):
    lens = [1, P, P + 1, 31, 32, 33, 255, 256, 257, 0, 600]
    _say(f"attend {dtype} D={D} P={P} lens={lens}")
    _attend_case(kv4, D + P, dtype, lens, 2, 3, D, P)


@pytest.mark.parametrize("heads,group,queries", [(1, 1, 1), (3, 1, 2), (2, 5, 1), (1, 16, 1), (2, 7, 3), (1, 17, 1),
                                                 (1, 8, 8), (2, 4, 20), (1, 40, 2)])
@pytest.mark.parametrize("window", [0, 1, 33])
def test_attend_heads_queries_windows(kv4, heads, group, queries, window):
    lens = [0, 1, 2, 19, 70, 300]
    _say(f"attend heads={heads} group={group} queries={queries} window={window}")
    _attend_case(kv4, heads + group, "bf16" if group % 2 else "fp16", lens, heads, group, 64, 16, queries, window,
                 strided=True)


@pytest.mark.parametrize("dtype,group,D", [("bf16", 4, 128), ("fp16", 8, 64), ("bf16", 1, 96), ("fp16", 20, 128),
                                           ("bf16", 2, 192), ("fp16", 3, 256)])
def test_attend_long_among_short(kv4, dtype, group, D):
    lens = [9000, 3, 0, 257, 1200]
    _say(f"attend long among short {dtype} group={group} D={D}")
    _attend_case(kv4, group, dtype, lens, 1, group, D, 64)


@pytest.mark.parametrize("queries,window", [(1, 700), (6, 1000), (3, 0)])
def test_attend_long_windows(kv4, queries, window):
    _say(f"attend windows queries={queries} window={window}")
    _attend_case(kv4, 3, "fp16", [3000, 900, 5, 1000], 2, 2, 128, 32, queries, window)


def test_attend_runs_of_many_pages(kv4):
    """One sequence over all workgroups, the joins of more than 32 runs and a
    segment of a wave's pages after another among them."""
    _say("attend 40000 tokens")
    _attend_case(kv4, 4, "bf16", [40000], 1, 4, 64, 16)
    _say("attend 20000 tokens of 300 pairs")  # one workgroup goes over more than a segment
    rng = np.random.default_rng(5)
    c = _host(rng, [20000, 7], 2, 128, 64)
    c["lens"] = np.array([20000] + [7] * 150 + [0], np.int32)
    c["table"] = np.stack([c["table"][0]] + [c["table"][1]] * 151)
    _attend_case(kv4, 6, "fp16", c["lens"].tolist(), 2, 2, 64, 128, c=c)


def test_attend_many_sequences(kv4):
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 90, 700).tolist()
    _say("attend 700 sequences")
    _attend_case(kv4, 7, "bf16", lens, 2, 2, 64, 16)


@pytest.mark.parametrize("dtype,heads,group,D,P,lens", [
    ("bf16", 2, 4, 128, 64, [4000, 100, 0, 2600, 1, 1281, 1280, 900]),          # joined by the last run
    ("fp16", 4, 4, 256, 64, [5000, 700, 0, 513, 512]),
    ("bf16", 1, 16, 64, 32, [3000, 3000, 2999]),                                # by a kernel, of rows in waves
    ("fp16", 1, 20, 96, 16, [20000, 5]),                                        # by a kernel, of rows in workgroups
    ("fp16", 1, 5, 192, 128, [600 * (i % 7) + i for i in range(64)]),           # as many sequences as a wave has lanes
    ("bf16", 1, 2, 64, 16, [(977 * i) % 2500 for i in range(65)]),              # one more
    ("fp16", 1, 1, 128, 64, [3000] + [(13 * i) % 90 for i in range(200)]),      # many, one of them long
    ("bf16", 2, 3, 256, 128, [9000, 17000] + [3] * 150),                        # more workgroups than CUs
    ("bf16", 3, 2, 128, 64, [2048] * 16),                                       # all alike
    ("fp16", 1, 2, 64, 16, [0] * 70 + [1500] + [0] * 5),                        # nearly all empty
])
def test_attend_cut_sequences(kv4, dtype, heads, group, D, P, lens):
    """Sequences cut into runs by all their lengths: every way to find them, and
    every way to join them."""
    _say(f"attend cut {dtype} heads={heads} group={group} D={D} batch={len(lens)}")
    _attend_case(kv4, D + len(lens), dtype, lens, heads, group, D, P)


@pytest.mark.parametrize("window,queries", [(1500, 1), (3000, 5), (1400, 30)])
def test_attend_cut_windows(kv4, window, queries):
    _say(f"attend cut windows window={window} queries={queries}")
    _attend_case(kv4, window, "fp16", [4000, 1700, 1, 0, 2999], 1, 2, 128, 32, queries, window)


def test_attend_cut_sequences_replayed(kv4):
    """The joins within the kernel in a captured call: replayed with other
    lengths, eagerly called on the same workspace between."""
    rng = np.random.default_rng(25)
    c = _host(rng, [6000, 6000, 6000], 2, 64, 64)
    cache = _device(kv4, c)
    q = torch.from_numpy(rng.normal(0, 1, (3, 1, 8, 64))).half().cuda()
    out, lse = torch.empty_like(q), torch.empty((3, 1, 8), device="cuda")
    ws = cache.attend_workspace(8)
    cache.attend(q, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend(q, out=out, lse=lse, workspace=ws)
    for rep, lens in enumerate(([6000, 6000, 6000], [1, 6000, 0], [5000, 3, 2000], [0, 0, 0], [6000, 5999, 1300])):
        _say(f"attend cut, replay {rep}")
        c["lens"][:] = lens
        cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(torch.from_numpy(rng.normal(0, 1, q.shape)).half())
        torch.cuda.synchronize()
        for _ in range(3):
            out.fill_(7)
            g.replay()
        torch.cuda.synchronize()
        _compare(64, "fp16", lens, *oracle.attend(c, q.double().cpu().numpy(), 0.125, 0), out, lse)
        again = cache.attend(q, workspace=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("q_size,scale", [(30.0, None), (1.0, 0.0), (1e-3, -2.0), (1.0, -0.3), (1.0, 1e-30),
                                          (300.0, 1e-3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attend_score_ranges(kv4, dtype, q_size, scale):
    _say(f"attend {dtype} q_size={q_size} scale={scale}")
    _attend_case(kv4, 8, dtype, [300, 40, 1], 2, 3, 128, 32, 2, q_size=q_size, scale=scale)


@pytest.mark.parametrize("q_size", [1e-30, 1e8, 1e12, 1e30])
@pytest.mark.parametrize("lens", [[300, 2], [2600, 700, 33]])
def test_attend_bf16_range(kv4, q_size, lens):
    """Scores far beyond what a weight's exponent holds, and far below."""
    _say(f"attend q_size={q_size} lens={lens}")
    _attend_case(kv4, 26, "bf16", lens, 1, 2, 64, 16, q_size=q_size)


@pytest.mark.parametrize("low,high", [(63, 64), (64, 190), (127, 160)])
def test_attend_scale_ranges(kv4, low, high):
    """Scales of unlike size side by side: loud and silent groups."""
    rng = np.random.default_rng(9)
    lens = [200, 31]
    c = _host(rng, lens, 2, 16, 96, low=low, high=high)
    if high > 128:  # keys stay where scores are numbers, values may be loud
        c["ks"][c["ks"] != 255] = rng.integers(120, 128, c["ks"].shape)[c["ks"] != 255]
    _say(f"attend scales {low} .. {high - 1}")
    _attend_case(kv4, 10, "bf16", lens, 2, 3, 96, 16, c=c)


def test_attend_without_lse_and_workspaces(kv4):
    from cross_core_barrier_amd import ccb
    rng = np.random.default_rng(11)
    c = _host(rng, [900, 900, 900], 2, 32, 64)
    cache = _device(kv4, c)
    ws = cache.attend_workspace(6, 2)
    for lens in ([900, 900, 900], [0, 0, 0], [1, 900, 33], [64, 2, 0], [0, 0, 850]):
        _say(f"attend, one workspace, lens={lens}")
        c["lens"][:] = lens
        cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q = torch.from_numpy(rng.normal(0, 1, (3, 2, 6, 64))).half()
        want = oracle.attend(c, q.double().numpy(), 0.125, 0)
        ws.random_()  # whatever it holds
        out, lse = cache.attend(q.cuda(), workspace=ws)
        _compare(64, "fp16", lens, *want, out, lse)
        again = torch.empty_like(out)
        qd = q.cuda()
        assert ccb.ccb_kv4_attend(cache._c, cache._rows(qd, 6, "q"), cache._rows(again, 6, "out"), None, 6, 2, 0.125, 0,
                                  ws, ws.numel()) == 0
        torch.cuda.synchronize()
        assert torch.equal(out, again)


def test_attend_in_place(kv4):
    rng = np.random.default_rng(12)
    for lens, group, queries in (([300, 5], 4, 1), ([5000], 3, 9), ([40, 3, 0], 6, 6)):
        c = _host(rng, lens, 2, 32, 64)
        cache = _device(kv4, c)
        q = torch.from_numpy(rng.normal(0, 1, (len(lens), queries, 2 * group, 64))).half().cuda()
        _say(f"attend in place lens={lens}")
        want, lse = cache.attend(q)
        got, again = cache.attend(q, out=q)
        assert got is q and torch.equal(want, q) and torch.equal(lse, again)


def test_attend_nan_and_infinite_queries_stay_in_their_rows(kv4):
    rng = np.random.default_rng(13)
    c = _host(rng, [70, 20], 2, 16, 64)
    cache = _device(kv4, c)
    for dtype in TYPES:
        q = torch.from_numpy(rng.normal(0, 1, (2, 2, 8, 64))).to(TYPES[dtype])
        want, *_ = oracle.attend(c, q.double().numpy(), 0.125, 0)
        q[0, 1, 2, 5] = math.nan
        q[1, 0, 7, 0] = math.inf
        _say(f"attend with NaN and infinity in two queries, {dtype}")
        out, _ = cache.attend(q.cuda())
        y = out.float().cpu().numpy()
        assert np.isnan(y[0, 1, 2]).all() and np.isnan(y[1, 0, 7]).all()
        good = np.ones(y.shape[:3], bool)
        good[0, 1, 2] = good[1, 0, 7] = False
        assert np.all(np.abs(y - want)[good] < 0.02 * np.abs(want[good]) + 0.02)


def test_attend_same_bits_every_time(kv4):
    _say("attend four times")
    rng = np.random.default_rng(14)
    c = _host(rng, [4000, 17, 900], 4, 64, 128)
    cache = _device(kv4, c)
    q = torch.from_numpy(rng.normal(0, 1, (3, 1, 16, 128))).half().cuda()
    ws = cache.attend_workspace(16)
    first = None
    for _ in range(4):
        now = [t.clone() for t in cache.attend(q, workspace=ws)]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def _append_case(kv4, rng, dtype, heads, D, P, rows, special=False, size=1.0, strided=False):
    """Rows to random distinct slots, some of them left out."""
    pages = -(-rows // P) + 4
    c = _host(rng, [0], heads, P, D, width=pages - 3)
    for w in ("k", "v"):
        c[w][...] = rng.integers(0, 256, c[w].shape)
        c[w + "s"][...] = rng.integers(0, 256, c[w + "s"].shape)
    cache = _device(kv4, c)
    slots = rng.permutation(pages * P)[:rows].astype(np.int64)
    slots[rng.random(rows) < 0.1] = -1
    x = []
    for _ in range(2):
        t = torch.from_numpy(rng.normal(0, size, (rows, heads, D)) * 2.0 ** rng.integers(-6, 6, (rows, heads, 1)))
        t = t.to(TYPES[dtype])
        if special:
            flat = t.view(-1)
            at = torch.from_numpy(rng.permutation(flat.numel())[:max(6, flat.numel() // 20)])
            bad = torch.tensor([math.nan, math.inf, -math.inf, -0.0, 0.0, torch.finfo(t.dtype).tiny])
            flat[at] = bad[torch.arange(len(at)) % 6].to(t.dtype)
            t[0, 0] = 0
            t[-1, -1, :32] = math.nan
            t[-1, 0, 32:64] = math.inf
        x.append(t)
    dev = [_spread(t.cuda(), 2, 1) if strided else t.cuda() for t in x]
    cache.append(*dev, torch.from_numpy(slots).cuda())
    oracle.append(c, x[0].double().numpy(), x[1].double().numpy(), slots)
    torch.cuda.synchronize()
    for w, t, s in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        assert np.array_equal(s.cpu().numpy(), c[w + "s"]), w
        assert np.array_equal(t.cpu().numpy(), c[w]), w
    cache.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,P", [(64, 16), (96, 32), (128, 64), (192, 128), (256, 128), (128, 16), (256, 16)])
@pytest.mark.parametrize("rows", [1, 23, 150])
def test_append(kv4, dtype, D, P, rows):
    _say(f"append {dtype} D={D} P={P} rows={rows}")
    rng = np.random.default_rng(D + rows)
    _append_case(kv4, rng, dtype, 3, D, P, rows, strided=rows == 23)
    _append_case(kv4, rng, dtype, 2, D, P, rows, special=True)


@pytest.mark.parametrize("size", [1e-38, 1e-30, 2.0 ** -66, 1e20, 1e37])
def test_append_tiny_and_huge_values(kv4, size):
    _say(f"append values of {size}")
    _append_case(kv4, np.random.default_rng(15), "bf16", 2, 64, 16, 40, size=size)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_every_value(kv4, dtype):
    """All 16-bit numbers beside a largest one: every border of every scale."""
    _say(f"append all values {dtype}")
    all16 = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(TYPES[dtype])
    x = all16.view(-1, 64).clone()
    tops = torch.tensor([7.0, 6.0, 7.03125, 3.5, 448.0, 1e-3, 65504.0, 2.0 ** -14])
    rows = torch.cat([x] + [torch.cat([x[:, :31], t.to(x.dtype).expand(1024, 1), x[:, 32:]], 1) for t in tops])
    rows = rows.view(-1, 1, 64)
    n, P = rows.shape[0], 128
    c = _host(np.random.default_rng(0), [0], 1, P, 64, width=-(-n // P))
    cache = _device(kv4, c)
    slots = np.arange(n, dtype=np.int64)
    cache.append(rows.cuda(), rows.flip(0).contiguous().cuda(), torch.from_numpy(slots).cuda())
    wide = rows.double().numpy()
    oracle.append(c, wide, wide[::-1], slots)
    torch.cuda.synchronize()
    assert np.array_equal(cache.k_scale.cpu().numpy(), c["ks"]) and np.array_equal(cache.k.cpu().numpy(), c["k"])
    assert np.array_equal(cache.v_scale.cpu().numpy(), c["vs"]) and np.array_equal(cache.v.cpu().numpy(), c["v"])


def test_append_bad_slots_are_dropped(kv4):
    from cross_core_barrier_amd import ccb
    rng = np.random.default_rng(16)
    c = _host(rng, [40], 2, 16, 64)
    cache = _device(kv4, c)
    room = cache.k.shape[0] * 16
    x = torch.ones((7, 2, 64), dtype=torch.float16, device="cuda")
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    _say("append to slots that are not there")
    for bad in (room, -2, 1 << 40, -(1 << 62), (1 << 32) + 3, (1 << 63) - 1):
        cache.append(x, x, torch.tensor([-1, bad, -1, bad, -1, -1, -1], device="cuda"))
        with pytest.raises(ccb.CcbError):
            cache.check()
    cache.append(x, x, torch.full((7,), -1, dtype=torch.int64, device="cuda"))
    cache.check()
    for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,P", [(64, 16), (96, 64), (128, 128), (192, 32), (256, 16)])
def test_read(kv4, dtype, D, P):
    rng = np.random.default_rng(D)
    lens = [0, 1, 70, 200]
    c = _host(rng, lens, 2, P, D, low=120, high=132)
    cache = _device(kv4, c)
    for first, count in (([0, 0, 0, 0], 200), ([5, -3, 60, 150], 61), ([-200, 0, 69, 199], 1), ([0, 1, 2 ** 30, -1], 33)):
        _say(f"read {dtype} D={D} first={first} count={count}")
        got = cache.read(count, first=torch.tensor(first, dtype=torch.int32, device="cuda"), dtype=dtype)
        for x, want in zip(got, oracle.read(c, count, first)):
            assert torch.equal(x.cpu(), torch.from_numpy(want).to(dtype))
    assert torch.equal(cache.read(7)[1].cpu(), torch.from_numpy(oracle.read(c, 7, [0] * 4)[1]).float())
    cache.check()


def test_read_one_side_and_every_scale(kv4):
    from cross_core_barrier_amd import ccb
    rng = np.random.default_rng(17)
    c = _host(rng, [254 * 2], 1, 128, 64)
    t = np.arange(508)
    for w in ("ks", "vs"):
        c[w][c["table"][0, t // 128], 0, t % 128] = (t // 2)[:, None]
    cache = _device(kv4, c)
    _say("read keys alone, values alone, all scales")
    want = oracle.read(c, 508, [0])
    for side in (0, 1):
        out = torch.full((1, 508, 1, 64), 7.0, device="cuda")
        rows = cache._rows(out, 1, "out")
        assert ccb.ccb_kv4_read(cache._c, None if side else rows, rows if side else None, 508, None, cache.err) == 0
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), torch.from_numpy(want[side]).float())


def test_bad_pages_and_lengths_are_met(kv4):
    """Page numbers and lengths out of range: reported, unseen, harmless."""
    from cross_core_barrier_amd import ccb
    rng = np.random.default_rng(18)
    lens = [100, 100, 100, 100]
    c = _host(rng, lens, 2, 16, 64)
    q = torch.from_numpy(rng.normal(0, 1, (4, 1, 6, 64))).half()
    good = oracle.attend(c, q.double().numpy(), 0.125, 0)
    pages = c["k"].shape[0]
    for name, bad in (("page", [pages, -1, 2 ** 31 - 1]), ("length", [-1, 8 * 16 + 1, 2 ** 31 - 1])):
        for value in bad:
            cache = _device(kv4, c)
            _say(f"bad {name} {value}")
            if name == "page":
                cache.page_table[1, 2] = value
            else:
                cache.lens[1] = value
            out, lse = cache.attend(q.cuda())
            with pytest.raises(ccb.CcbError):
                cache.check()
            k, _ = cache.read(100)
            with pytest.raises(ccb.CcbError):
                cache.check()
            y = out.double().cpu().numpy()
            for b in (0, 2, 3):
                assert np.allclose(y[b], good[0][b], rtol=2e-3, atol=2e-3)
            if name == "length":
                assert not out[1].any() and torch.all(lse[1] == -math.inf) and not k[1].any()
            else:
                assert not k[1, 32:48].any()
                t = np.r_[0:32, 48:100]
                for j in range(6):
                    s = oracle.dense(c, "k", 1, j // 3, t) @ q[1, 0, j].double().numpy() * 0.125
                    p = np.exp(s - s.max())
                    assert np.allclose(y[1, 0, j], p @ oracle.dense(c, "v", 1, j // 3, t) / p.sum(), rtol=2e-3, atol=2e-3)
    cache = _device(kv4, c)
    cache.page_table[1] = -1  # nothing to see at all
    out, lse = cache.attend(q.cuda())
    assert not out[1].any() and torch.all(lse[1] == -math.inf)


def test_window_does_not_look_at_pages_before_it(kv4):
    _say("window over pages that were given away")
    rng = np.random.default_rng(19)
    c = _host(rng, [300], 2, 16, 64)
    cache = _device(kv4, c)
    q = torch.from_numpy(rng.normal(0, 1, (1, 2, 4, 64))).half()
    want = oracle.attend(c, q.double().numpy(), 0.125, 50)
    first = 300 - 2 + 1 - 50
    cache.page_table[0, :first // 16] = -1
    out, lse = cache.attend(q.cuda(), window=50)
    _compare(64, "fp16", [300], *want, out, lse)
    cache.check()


def test_side_stream(kv4):
    rng = np.random.default_rng(20)
    c = _host(rng, [400, 33, 129], 2, 32, 128)
    a, b = _device(kv4, c), _device(kv4, c)
    x = torch.from_numpy(rng.normal(0, 1, (3, 2, 128))).half().cuda()
    q = torch.from_numpy(rng.normal(0, 1, (3, 1, 8, 128))).half().cuda()
    slots = torch.tensor([int(c["table"][i, (n - 1) // 32]) * 32 + (n - 1) % 32 for i, n in enumerate([400, 33, 129])],
                         device="cuda")
    s = torch.cuda.Stream()
    _say("append + attend + read on a side stream")
    a.append(x, -x, slots)
    want = a.attend(q)
    b.append(x, -x, slots, stream=s)
    got = b.attend(q, stream=s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(i, j) for i, j in zip(b.read(20, stream=s), a.read(20)))


def test_steps_with_a_pool_captured(kv4):
    """A whole decoding step (pages and slots, append, attention) captured once
    and replayed with other tokens, requests that end and others in their
    places, eager work between; against the same calls made eagerly, whose
    attention is held against the oracle."""
    from cross_core_barrier_amd.pages import PagePool
    rng = np.random.default_rng(21)
    batch, heads, D, P, pages, room = 5, 2, 96, 16, 40, 24

    def make():
        cache = kv4.Kv4Cache.allocate(pages, heads, P, D, batch, 12)
        cache.k_scale.fill_(255)
        cache.v_scale.fill_(255)
        return cache, PagePool.allocate(pages, P)
    (cache, pool), (plain, plain_pool) = make(), make()
    keep, counts = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2))
    k, v = (torch.zeros((room, heads, D), dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros((batch, 2, 6, D), dtype=torch.float16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((batch, 2, 6), device="cuda")
    maps, plain_maps = pool.maps(batch, room), plain_pool.maps(batch, room)
    ws = cache.attend_workspace(6, 2)

    def step(cache, pool, maps, **kw):
        pool.trim(cache.page_table, cache.lens, keep)
        pool.grow(cache.page_table, cache.lens, counts, maps)
        cache.append(k, v, maps.slots)
        return cache.attend(q, **kw)
    step(cache, pool, maps, out=out, lse=lse, workspace=ws)  # of nothing
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(cache, pool, maps, out=out, lse=lse, workspace=ws)
    for rep in range(12):
        _say(f"step {rep}")
        keep.copy_(torch.tensor([0 if rng.random() < 0.15 else -1 for _ in range(batch)], dtype=torch.int32))
        counts.copy_(torch.tensor(rng.integers(0, 5, batch) if rep % 4 else [9, 2, 0, 7, 5], dtype=torch.int32))
        for t in (k, v, q):
            t.copy_(torch.from_numpy(rng.normal(0, 1, t.shape)).half())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = step(plain, plain_pool, plain_maps)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), rep
        for a, b in ((cache, plain), (pool, plain_pool), (maps, plain_maps)):
            for name, t in vars(a).items():
                if isinstance(t, torch.Tensor):
                    assert torch.equal(t, getattr(b, name)), (rep, name)
        c = dict(k=cache.k.cpu().numpy(), v=cache.v.cpu().numpy(), ks=cache.k_scale.cpu().numpy(),
                 vs=cache.v_scale.cpu().numpy(), table=cache.page_table.cpu().numpy(), lens=cache.lens.cpu().numpy())
        _compare(D, "fp16", c["lens"].tolist(), *oracle.attend(c, q.double().cpu().numpy(), float(np.float32(D ** -0.5)), 0),
                 out, lse)
    cache.check()
    pool.check()


def test_pages_past_32_bits(kv4):
    """Pages whose bytes lie beyond 2^32, and slots beyond 2^24: every operator
    on the far end of a 5.4 GB pool."""
    heads, P, D = 16, 128, 128
    pages = 41_000  # 41,000 * 16 * 128 * 64 bytes
    k, v = (torch.empty((pages, heads, P, D // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = [torch.full((pages, heads, P, D // 32), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    lens = [300, 129]
    rng = np.random.default_rng(22)
    table = torch.tensor([[pages - 1, pages - 7, pages - 3], [pages - 2, 5, 40_000]], dtype=torch.int32, device="cuda")
    far = kv4.Kv4Cache(k, v, *scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    near = kv4.Kv4Cache.allocate(6, heads, P, D, 2, 3)
    near.page_table.copy_(torch.arange(6, dtype=torch.int32).view(2, 3))
    near.lens.copy_(far.lens)
    x = [torch.from_numpy(rng.normal(0, 1, (429, heads, D))).half().cuda() for _ in range(2)]
    q = torch.from_numpy(rng.normal(0, 1, (2, 1, 32, D))).half().cuda()
    b = torch.tensor([0] * 300 + [1] * 129, device="cuda")
    t = torch.cat([torch.arange(300), torch.arange(129)]).cuda()
    _say("append, attend and read beyond 2^32 bytes")
    results = []
    for c in (far, near):
        c.append(*x, c.page_table.long()[b, t // P] * P + t % P)
        results.append([*c.attend(q), *c.read(300)])
        c.check()
    for a, z in zip(*results):
        assert torch.equal(a, z)


def test_capacity_far_beyond_the_lengths(kv4):
    _say("attend and read in a table of 2^20 tokens")
    rng = np.random.default_rng(23)
    c = _host(rng, [5, 700], 2, 128, 64, width=8192, extra=0)
    _attend_case(kv4, 23, "bf16", [5, 700], 2, 4, 64, 128, c=c)


def test_an_error_left_by_another_call_is_not_reported(kv4):
    from cross_core_barrier_amd import ccb
    rng = np.random.default_rng(24)
    c = _host(rng, [40], 2, 16, 64)
    cache = _device(kv4, c)
    q = torch.zeros((1, 1, 4, 64), dtype=torch.float16, device="cuda")
    assert ccb.ccb_bench_copy(q, q, -1) != 0
    out, _ = cache.attend(q)
    assert torch.isfinite(out).all()


def _session(graph, pages=None, limit=40):
    """A session driven through arrivals, ends and shortages; what it ends in."""
    from cross_core_barrier_amd.kv8_decode import PooledSession
    s = PooledSession(batch=4, heads=2, q_heads=6, head_dim=64, page_size=16, limit=limit, pages=pages, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(7)
    prompt = lambda n: torch.randn((n, s.x.shape[1]), generator=gen, device="cuda").to(s.x.dtype)  # noqa: E731
    log = [s.sit([2, 0, 3], [prompt(20), prompt(1), prompt(33)])]
    for i in range(12):
        s.step(graph)
        if i == 4:
            s.leave([3])
            log.append(s.sit([1, 3], [prompt(30), prompt(17)]))
        if i == 8:
            s.leave([0])
    torch.cuda.synchronize()
    s.cache.check()
    s.pool.check()
    # every page is in the pool, or held once
    held = [p for b, n in enumerate(s.cache.lens.tolist()) for p in s.cache.page_table[b, :-(-n // 16)].tolist()]
    free = s.pool.free[:s.pool.count.item()].tolist()
    assert sorted(held + free) == list(range(s.cache.k.shape[0]))
    return s, log, gen


@pytest.mark.parametrize("pages", [None, 6])
def test_pooled_session(kv4, pages):
    """Requests that come and go, with pages for everybody and with too few:
    replayed from a graph and made eagerly the session ends in the same bits, and
    its attention is the oracle's over what the cache holds."""
    ends = []
    for graph in (True, False):
        _say(f"pooled session pages={pages} graph={graph}")
        s, log, gen = _session(graph, pages)
        ends.append((s.x.clone(), s.cache.lens.clone(), s.pool.free.clone(), *s.cache.read(48)))
        if pages is None:
            assert log == [[0, 2, 3], [1, 3]] and s.cache.lens.tolist() == [0, 37, 32, 24]
        else:  # 1 + 2 + 3 pages, and then 3 of them for the two that come: the second has to wait
            assert log[0] == [0, 2, 3] and log[1] == [1]
    assert all(torch.equal(a, b) for a, b in zip(*ends))
    q = torch.randn((4, 1, 6, 64), generator=gen, device="cuda").half()
    c = dict(lens=s.cache.lens.cpu().numpy(), table=s.cache.page_table.cpu().numpy(), k=s.cache.k.cpu().numpy(),
             v=s.cache.v.cpu().numpy(), ks=s.cache.k_scale.cpu().numpy(), vs=s.cache.v_scale.cpu().numpy())
    want = oracle.attend(c, q.double().cpu().numpy(), 0.125, 0)
    _compare(64, "fp16", c["lens"].tolist(), *want, *s.cache.attend(q))


def test_pooled_session_waits_for_pages(kv4):
    """A request whose next page is not there stays at its token until another
    one leaves."""
    from cross_core_barrier_amd.kv8_decode import PooledSession
    _say("pooled session: a token that waits")
    s = PooledSession(batch=2, heads=1, q_heads=2, head_dim=64, page_size=16, limit=64, pages=4, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(8)
    rows = torch.randn((64, 128), generator=gen, device="cuda").to(s.x.dtype)
    assert s.sit([0, 1], [rows[:31], rows[:30]]) == [0, 1]
    s.step()
    s.step()  # both at the end of their second page, the second in its last place
    assert s.cache.lens.tolist() == [32, 32]
    x = s.x.clone()
    s.step()
    assert s.cache.lens.tolist() == [32, 32] and torch.equal(s.x, x)
    s.leave([1])
    s.step()
    assert s.cache.lens.tolist() == [33, 0] and not torch.equal(s.x[0], x[0])
    s.pool.check()


def test_decode_command_serves_requests(kv4, capsys):
    from cross_core_barrier_amd import kv8_decode
    _say("kv8_decode --format mxfp4")
    kv8_decode.main(["--batch", "3", "--steps", "30", "--prompt", "90", "--limit", "100", "--format", "mxfp4"])
    # prompts of 90, 53, 16, 90, 53, 16 tokens, to 100 each: the first seat's ends after 10 steps, and after 20
    out = capsys.readouterr().out
    assert "3 seats, 30 steps, 2 requests ended" in out and "lengths now 46 to 83" in out


def test_pooled_session_after_a_refused_prompt(kv4):
    """The seat is as free as before."""
    from cross_core_barrier_amd.kv8_decode import PooledSession
    _say("pooled session: a refused prompt")
    s = PooledSession(batch=2, heads=1, q_heads=2, head_dim=64, page_size=16, limit=40, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(9)
    rows = torch.randn((20, 128), generator=gen, device="cuda").to(s.x.dtype)
    for bad in (rows[:, :64], rows.half(), rows.cpu(), rows.clone().requires_grad_()):
        with pytest.raises(ValueError, match="prompts"):
            s.sit([0], [bad])
    assert s.cache.lens.tolist() == [0, 0] and s.pool.count.item() == 6
    assert s.sit([], []) == [] and s.sit([0], [rows]) == [0]
    s.step()
    assert s.cache.lens.tolist() == [21, 0] and s.pool.count.item() == 4
    s.pool.check()


@pytest.mark.parametrize("graph", [True, False])
@pytest.mark.parametrize("limit", [32, 40])
def test_pooled_session_stops_at_the_limit(kv4, limit, graph):
    """A limit that fills its pages, and one that does not: a request at it stays
    as it is, the others go on, and nothing is reported."""
    from cross_core_barrier_amd.kv8_decode import PooledSession
    _say(f"pooled session: limit {limit} graph={graph}")
    ends = []
    for full in (True, False):  # the same neighbour beside a request that ends, and beside none
        s = PooledSession(batch=3, heads=1, q_heads=2, head_dim=64, page_size=16, limit=limit, seed=4)
        gen = torch.Generator(device="cuda").manual_seed(10)
        rows = torch.randn((64, 128), generator=gen, device="cuda").to(s.x.dtype)
        s.sit([1], [rows[:5]])
        if full:
            s.sit([0, 2], [rows[:limit - 2], rows[:limit]])
        at_limit = []
        for i in range(8):
            s.step(graph)
            if i >= 1:
                at_limit.append(s.x[::2].clone())
        lens = [limit, 13, limit] if full else [0, 13, 0]
        assert s.cache.lens.tolist() == lens
        assert s.pool.count.item() == s.cache.k.shape[0] - sum(-(-n // 16) for n in lens)
        assert all(torch.equal(x, at_limit[0]) for x in at_limit)
        if full:
            assert torch.equal(s.x[2], rows[limit - 1])
            s.leave([0, 2])
            assert s.sit([2], [rows[:3]]) == [2]
            s.step(graph)
            assert s.cache.lens.tolist() == [0, 14, 4]
        else:
            s.step(graph)
        s.cache.check()
        s.pool.check()
        ends.append(s.x[1].clone())
    assert torch.equal(*ends)  # (rows of the same products, and a sequence in one run)


@pytest.mark.parametrize("steps,ended,lens", [(1, 1, "26 to 99"), (2, 2, "27 to 64"), (3, 2, "28 to 65")])
def test_decode_command_counts_requests_of_the_first_step(kv4, capsys, steps, ended, lens):
    """Prompts of 99, 62, 25, 99, 62, 25 tokens, to 100 each: the first seat's end with
    the first step and the second."""
    from cross_core_barrier_amd import kv8_decode
    _say(f"kv8_decode --format mxfp4, {steps} steps, prompts one short of the limit")
    kv8_decode.main(["--batch", "3", "--steps", str(steps), "--prompt", "99", "--limit", "100", "--format", "mxfp4"])
    out = capsys.readouterr().out
    assert f"3 seats, {steps} steps, {ended} requests ended" in out and f"lengths now {lens}" in out


def test_attend_of_2_26_rows(kv4):
    """A call of 4.2 million workgroups, more rows than the kernel that joins runs would
    hold: 1024 sequences alike, each as it comes out by itself."""
    rng = np.random.default_rng(27)
    c = _host(rng, [40], 8, 16, 64)
    one = _device(kv4, c)
    many = kv4.Kv4Cache(one.k, one.v, one.k_scale, one.v_scale, one.page_table.repeat(1024, 1), one.lens.repeat(1024))
    q = torch.from_numpy(rng.normal(0, 1, (1, 1024, 64, 64))).bfloat16().cuda()
    _say("attend 1024 sequences, 1024 queries, 64 heads")
    want, want_lse = one.attend(q)
    out, lse = many.attend(q.expand(1024, -1, -1, -1))
    torch.cuda.synchronize()
    assert (want[0, :984] == 0).all() and (want[0, 984:] != 0).any(-1).all()
    assert torch.equal(lse, want_lse.expand_as(lse))
    for b0 in range(0, 1024, 128):  # (8.6 GB)
        assert torch.equal(out[b0:b0 + 128], want.expand(128, -1, -1, -1))
    many.check()


@pytest.mark.parametrize("keys,values,q_size", [(0, 127, 2.0 ** 124), (1, 127, 2.0 ** 123), (2, 127, 2.0 ** 122),
                                                (0, 0, 1.0), (127, 1, 1.0), (120, 2, 3.0), (127, 8, 1.0)])
def test_attend_smallest_scales(kv4, keys, values, q_size):
    """Scales below those that an append writes, whose values are bf16's subnormals
    among them: keys under queries that bring them back, and values as they are
    (there half a step of out is 2^-134)."""
    rng = np.random.default_rng(28)
    lens = [40, 700, 1500]
    c = _host(rng, lens, 1, 16, 64)
    for w, low in (("ks", keys), ("vs", values)):
        c[w][c[w] != 255] = rng.integers(low, low + 3, c[w].shape)[c[w] != 255]
    cache = _device(kv4, c)
    q = torch.from_numpy(rng.normal(0, q_size, (3, 1, 3, 64))).bfloat16()
    _say(f"attend scales from {keys} and {values}")
    want, lse, mag, big = oracle.attend(c, q.double().numpy(), 1.0, 0)
    assert big.max() > 0.5 or keys == values == 0
    out, got = cache.attend(q.cuda(), scale=1.0)
    rel, tol_lse, tol = _bounds(64, max(lens), mag, big, lse)
    y = out.double().cpu().numpy()
    # sums of values are rounded in steps of 2^-149, once for each of two products of 32 tokens and each join
    assert np.all(np.abs(y - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -134 + 2.0 ** -140)
    assert np.all(np.abs(got.double().cpu().numpy() - lse) <= tol_lse)
    # a scale of 0 that counted as nothing would be seen, in keys or in values
    c0 = dict(c, k=np.where(np.repeat(c["ks"] == 0, 16, -1), 0, c["k"]), v=np.where(np.repeat(c["vs"] == 0, 16, -1), 0, c["v"]))
    if keys == 0 or values == 0:
        other, other_lse, _, _ = oracle.attend(c0, q.double().numpy(), 1.0, 0)
        assert np.any(np.abs(other - want) > 2 * (tol + 2.0 ** -8 * np.abs(want) + 2.0 ** -134)) or \
            np.any(np.abs(other_lse - lse) > 2 * tol_lse)
    cache.check()


@pytest.mark.parametrize("graph", [True, False])
def test_pooled_session_waits_just_below_the_limit(kv4, graph):
    """Steps without a token do not count towards the limit, and one that waited for
    its page gets there."""
    from cross_core_barrier_amd.kv8_decode import PooledSession
    _say(f"pooled session: a token that waits below the limit, graph={graph}")
    s = PooledSession(batch=2, heads=1, q_heads=2, head_dim=64, page_size=16, limit=36, pages=4, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(11)
    rows = torch.randn((36, 128), generator=gen, device="cuda").to(s.x.dtype)
    assert s.sit([0, 1], [rows[:30], rows[:20]]) == [0, 1]
    for _ in range(2 + 13):
        s.step(graph)  # to the end of their second pages; seat 0 could be at the limit by its steps
    assert s.cache.lens.tolist() == [32, 32]
    s.leave([1])
    for n in (33, 34, 35, 36, 36, 36):
        s.step(graph)
        assert s.cache.lens.tolist() == [n, 0]
    s.leave([0])
    assert s.sit([1, 0], [rows[:35], rows[:1]]) == [0, 1]
    for n in (36, 36):
        s.step(graph)
        assert s.cache.lens.tolist()[1] == n
    assert s.cache.lens.tolist() == [3, 36]
    s.cache.check()
    s.pool.check()
