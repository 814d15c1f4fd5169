"""The 8-bit key/value cache on the GPU against the oracle in 64 bits
(oracle/kv8.py).  Codes, scales, kept tokens and lengths are compared exactly;
attention within bounds counted from its roundings (see _attend_case).  Unused
pages, and slots past a sequence's end, hold NaN codes and NaN scales."""

import math

import numpy as np
import pytest

from oracle import kv8 as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _say(msg):
    print(f"[gpu case] {msg}", flush=True)


@pytest.fixture(scope="module")
def kv8():
    from cross_core_barrier_amd import ccb, kv8 as module
    st, _, _, _ = ccb.ccb_device_info()
    assert st == 0, ccb.ccb_status_string(st)
    return module


def _host(rng, fmt, lens, heads, P, D, width=None, extra=3, quiet=1.0):
    """A cache on the host: pages in random order, the bytes no token owns all
    0x7F / 0x80 (NaN in e4m3, the out-of-range -128 in int8)."""
    batch = len(lens)
    width = width or max(1, -(-max(lens) // P)) + 1
    pages = batch * width + extra
    junk = 0x7F if fmt == "e4m3" else 0x80
    c = dict(fmt=fmt, lens=np.array(lens, np.int32), table=rng.permutation(pages)[:batch * width].astype(np.int32)
             .reshape(batch, width), weight=None)
    for w in ("k", "v"):
        c[w] = np.full((pages, heads, P, D), junk, np.uint8)
        c[w + "s"] = np.full((pages, heads), np.nan, np.float32)
    for b, n in enumerate(lens):
        for number in range(-(-n // P)):
            page = c["table"][b, number]
            slots = min(P, n - number * P)
            for w in ("k", "v"):
                if fmt == "int8":
                    x = np.clip(np.round(rng.normal(0, 40, (heads, slots, D))), -127, 127).astype(np.int8)
                    c[w][page, :, :slots] = x.view(np.uint8)
                else:
                    x = rng.integers(0, 127, (heads, slots, D)) | (rng.integers(0, 2, (heads, slots, D)) << 7)
                    c[w][page, :, :slots] = x
                top = 40 if fmt == "int8" else 150
                c[w + "s"][page] = (rng.uniform(0.2, 2, heads) / top * quiet).astype(np.float32)
    return c


def _device(kv8, c):
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    code = CODES[c["fmt"]]
    return kv8.Kv8Cache(up(c["k"]).view(code), up(c["v"]).view(code), up(c["ks"]), up(c["vs"]), up(c["table"]),
                        up(c["lens"]), None if c["weight"] is None else up(c["weight"]))


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


def _spread_heads(x, spare):
    """The same values with strides: a slice of a wider tensor."""
    wide = torch.zeros((*x.shape[:2], x.shape[2] + spare, x.shape[3]), dtype=x.dtype, device=x.device)
    wide[:, :, 1:1 + x.shape[2]] = x
    return wide[:, :, 1:1 + x.shape[2]]


def _bounds(D, tokens, seen_mag, big, lse):
    """What fp32 attention over exact 8-bit products may be off by.
    A score is a sum of D exact products in fp32, scaled by two more factors:
    off by at most (D + 4) half steps of sum |q k| scale (`big`).  Its weight
    is off, relatively, by that plus as much for the maximum it is compared
    with, plus the exponential's own error (the argument's rounding, a few
    half steps of the largest |s - m| <= 2 big, and 4 of its value); sums over
    the tokens add `tokens` half steps at worst."""
    u = 2.0 ** -24
    ds = (D + 4) * u * big
    rel = 2 * ds + (4 * big + 8 + 2 * tokens) * u
    return rel, ds + rel + 4 * u * np.abs(np.where(np.isfinite(lse), lse, 0)), rel[..., None] * seen_mag


def _attend_case(kv8, seed, fmt, dtype, lens, heads, group, D, P, queries=1, window=0, accumulate=True, scale=None,
                 q_size=1.0, c=None, strided=False, skip=(), **kw):
    rng = np.random.default_rng(seed)
    c = c or _host(rng, fmt, lens, heads, P, D)
    tokens = c["table"].shape[1] * P
    base = rng.uniform(0, 1, (len(lens), heads, tokens)).astype(np.float32) * 1e-2
    c["weight"] = base.copy()
    cache = _device(kv8, c)
    q = torch.from_numpy(rng.normal(0, q_size, (len(lens), queries, heads * group, D))).to(TYPES[dtype])
    scale = 1 / math.sqrt(D) if scale is None else scale
    want, lse, weight, mag, big = oracle.attend(c, q.double().numpy(), float(np.float32(scale)), window)
    dq = q.cuda()
    out = None
    if strided:
        dq = _spread_heads(dq, 3)
        out = _spread_heads(torch.zeros_like(q, device="cuda"), 2)
    got, got_lse = cache.attend(dq, scale=scale, window=window, accumulate=accumulate, out=out, **kw)
    torch.cuda.synchronize()
    rel, tol_lse, tol = _bounds(D, max(max(lens), 1), mag, big, lse)
    eps = torch.finfo(TYPES[dtype]).eps / 2
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0  # half a step of fp16's subnormals
    y = got.double().cpu().numpy()
    live = [b for b in range(len(lens)) if b not in skip]
    assert np.all(np.abs(y - want)[live] <= (tol + eps * (np.abs(want) + tol) + tiny)[live])
    z = got_lse.double().cpu().numpy()
    empty = np.isinf(lse)
    assert np.array_equal(np.isneginf(z)[live], empty[live])
    assert np.all(y[empty] == 0)
    diff = np.abs(np.where(empty, 0, z) - np.where(empty, 0, lse))
    assert np.all(diff[live] <= tol_lse[live] + 1e-45)
    w = cache.weight.double().cpu().numpy()
    worst = rel.max() if rel.size else 0.0
    if accumulate:
        rows = queries * group
        tol_w = weight * (worst + rows * 2.0 ** -24) + 2.0 ** -24 * (base + weight) + rows * 2.0 ** -120
        assert np.all(np.abs(w - (base.astype(np.float64) + weight))[live] <= tol_w[live])
    else:
        assert np.array_equal(w, base.astype(np.float64))
    return cache, dq, got, got_lse


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,P", [(64, 16), (64, 128), (96, 32), (96, 64), (128, 64), (128, 16), (192, 128), (192, 32),
                                 (256, 64), (256, 128)])
def test_attend_sizes(kv8, fmt, dtype, D, P):
    """Lengths around the borders of pages and tiles, empty ones among them."""
    lens = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 257]
    _say(f"attend {fmt} {dtype} D={D} P={P} lens={lens}")
    _attend_case(kv8, D + P, fmt, dtype, lens, 2, 4, D, P)


@pytest.mark.parametrize("heads,group,queries", [(1, 1, 1), (3, 1, 2), (2, 5, 1), (1, 16, 1), (2, 7, 3), (1, 17, 1),
                                                 (1, 8, 4), (1, 32, 2), (1, 71, 1), (2, 4, 40), (1, 3, 100)])
@pytest.mark.parametrize("window", [0, 1, 33])
def test_attend_heads_queries_windows(kv8, heads, group, queries, window):
    """Rows that see nothing (more queries than tokens), windows that begin
    inside a tile, and more rows than one tile of queries holds."""
    _say(f"attend heads={heads} group={group} queries={queries} window={window}")
    fmt, dtype = ("int8", "bf16") if (heads + group) % 2 else ("e4m3", "fp16")
    _attend_case(kv8, group, fmt, dtype, [0, 1, 2, 39, 150], heads, group, 64, 32, queries, window, strided=True)


@pytest.mark.parametrize("fmt,group,D", [("int8", 4, 128), ("e4m3", 8, 64), ("int8", 1, 96), ("e4m3", 20, 128)])
def test_attend_long_among_short(kv8, fmt, group, D):
    """One long sequence that many workgroups share, short ones beside it."""
    _say(f"attend long {fmt} group={group} D={D}")
    _attend_case(kv8, 5, fmt, "fp16", [7, 9001, 0, 130, 2050], 2, group, D, 64)


@pytest.mark.parametrize("queries,window", [(1, 700), (6, 1000), (3, 0)])
def test_attend_long_windows(kv8, queries, window):
    _say(f"attend long, queries={queries} window={window}")
    _attend_case(kv8, 6, "int8", "bf16", [5003, 64, 1500], 2, 6, 96, 128, queries, window)


def test_attend_many_sequences(kv8):
    _say("attend 150 sequences, 3 heads")
    lens = [(i * 37) % 211 for i in range(150)]
    _attend_case(kv8, 7, "e4m3", "bf16", lens, 3, 2, 64, 16)


@pytest.mark.parametrize("q_size,scale", [(30.0, None), (1.0, 0.0), (1e-3, -2.0), (1.0, 1e-30), (300.0, 1e-3)])
def test_attend_score_ranges(kv8, q_size, scale):
    """One token that takes everything, all tokens alike, a negative scale."""
    _say(f"attend q_size={q_size} scale={scale}")
    _attend_case(kv8, 8, "int8", "fp16", [100, 1, 65], 2, 3, 64, 32, scale=scale, q_size=q_size)


@pytest.mark.parametrize("q_size", [1e-30, 1e30])
def test_attend_bf16_range(kv8, q_size):
    """Queries far outside fp16's range; the scale brings the scores back."""
    _say(f"attend bf16 queries of size {q_size}")
    _attend_case(kv8, 9, "e4m3", "bf16", [90, 300], 2, 4, 128, 64, scale=0.1 / q_size, q_size=q_size)


def test_attend_quiet_and_loud_blocks(kv8):
    """Scales of a sequence's blocks 2^-40 .. 2^20 apart, zero among them: a
    block that is quiet beside its neighbours still counts where the loud ones
    draw no weight."""
    rng = np.random.default_rng(10)
    c = _host(rng, "int8", [256, 130], 2, 16, 64)
    for b in range(2):
        for j in range(c["table"].shape[1]):
            c["vs"][c["table"][b, j]] *= np.float32(2.0 ** rng.integers(-40, 20))
    c["vs"][c["table"][0, 3]] = 0
    c["ks"][c["table"][0, 4]] = 0
    _say("attend with unlike block scales")
    _attend_case(kv8, 10, "int8", "bf16", [256, 130], 2, 4, 64, 16, c=c)


def test_attend_without_weight_and_lse_unasked(kv8):
    from cross_core_barrier_amd import ccb
    rng = np.random.default_rng(11)
    c = _host(rng, "int8", [50, 3], 2, 16, 64)
    cache = _device(kv8, c)
    q = torch.from_numpy(rng.normal(0, 1, (2, 1, 4, 64))).to(torch.bfloat16).cuda()
    _say("attend without weight, and without lse")
    out, lse = cache.attend(q)
    ws = cache.attend_workspace(4)
    again = torch.empty_like(out)
    st = ccb.ccb_kv8_attend(cache._c, cache._rows(q, 4, "q"), cache._rows(again, 4, "out"), None, 4, 1, 0.125, 0, 0,
                            ws, ws.numel())
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    with pytest.raises(ccb.CcbError):
        cache.attend(q, accumulate=True)


def test_attend_nan_and_infinite_queries_stay_in_their_rows(kv8):
    rng = np.random.default_rng(12)
    c = _host(rng, "int8", [70, 20], 2, 16, 64)
    cache = _device(kv8, c)
    q = torch.from_numpy(rng.normal(0, 1, (2, 2, 8, 64))).to(torch.bfloat16)
    want, *_ = oracle.attend(c, q.double().numpy(), 0.125, 0)
    q[0, 1, 2, 5] = math.nan
    q[1, 0, 7, 0] = math.inf
    _say("attend with NaN and infinity in two queries")
    out, _ = cache.attend(q.cuda())
    y = out.float().cpu().numpy()
    assert np.isnan(y[0, 1, 2]).all() and np.isnan(y[1, 0, 7]).all()
    good = np.ones(y.shape[:3], bool)
    good[0, 1, 2] = good[1, 0, 7] = False
    assert np.all(np.abs(y - want)[good] < 0.02 * np.abs(want[good]) + 0.02)


def test_attend_same_bits_every_time(kv8):
    _say("attend twice, with and without another call between")
    rng = np.random.default_rng(13)
    c = _host(rng, "e4m3", [4000, 17, 900], 4, 64, 128)
    c["weight"] = np.zeros((3, 4, c["table"].shape[1] * 64), np.float32)
    cache = _device(kv8, c)
    q = torch.from_numpy(rng.normal(0, 1, (3, 1, 16, 128))).half().cuda()
    ws = cache.attend_workspace(16, 1, True)
    first = None
    for _ in range(4):
        cache.weight.zero_()
        out, lse = cache.attend(q, accumulate=True, workspace=ws)
        now = [t.clone() for t in (out, lse, cache.weight)]
        torch.cuda.synchronize()
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_attend_workspace_serves_other_lengths(kv8):
    """One workspace over calls with other lengths: nothing stays behind."""
    rng = np.random.default_rng(14)
    c = _host(rng, "int8", [900, 900, 900], 2, 32, 64)
    c["weight"] = np.zeros((3, 2, c["table"].shape[1] * 32), np.float32)
    cache = _device(kv8, c)
    ws = cache.attend_workspace(6, 2, True)
    for lens in ([900, 900, 900], [0, 0, 0], [1, 900, 33], [64, 2, 0], [0, 0, 850]):
        _say(f"attend, one workspace, lens={lens}")
        c["lens"][:] = lens
        c["weight"][:] = 0
        cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        cache.weight.zero_()
        q = torch.from_numpy(rng.normal(0, 1, (3, 2, 6, 64))).half()
        want, lse, weight, *_ = oracle.attend(c, q.double().numpy(), 0.125, 0)
        out, got = cache.attend(q.cuda(), accumulate=True, workspace=ws)
        assert np.allclose(out.double().cpu().numpy(), want, rtol=2e-3, atol=2e-3)
        assert np.allclose(got.double().cpu().numpy(), lse, rtol=1e-4, atol=1e-4)
        assert np.allclose(cache.weight.cpu().numpy(), weight, rtol=1e-3, atol=1e-6)


def test_bad_pages_and_lengths_are_met(kv8):
    """Page numbers and lengths out of range: reported, unseen, harmless."""
    from cross_core_barrier_amd import ccb
    rng = np.random.default_rng(15)
    lens = [100, 100, 100, 100]
    c = _host(rng, "int8", lens, 2, 16, 64)
    want_c = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in c.items()}
    c["weight"] = np.zeros((4, 2, c["table"].shape[1] * 16), np.float32)
    cache = _device(kv8, c)
    cache.page_table[0, 2] = -1
    cache.page_table[1, 0] = c["k"].shape[0]
    cache.page_table[1, 6] = 2**31 - 1
    cache.lens[2] = c["table"].shape[1] * 16 + 1
    q = torch.from_numpy(rng.normal(0, 1, (4, 1, 4, 64))).half()
    _say("attend with bad pages and a bad length")
    out, lse = cache.attend(q.cuda(), accumulate=True)
    with pytest.raises(ccb.CcbError):
        cache.check()
    cache.check()  # cleared
    # the oracle without the tokens of the bad pages
    for b, gone in ((0, range(32, 48)), (1, list(range(16)) + list(range(96, 100)))):
        stay = np.array([t for t in range(100) if t not in gone])
        for h in range(2):
            k, v = oracle.dense(want_c, "k", b, h, stay), oracle.dense(want_c, "v", b, h, stay)
            for j in (2 * h, 2 * h + 1):
                s = k @ q[b, 0, j].double().numpy() * 0.125
                p = np.exp(s - s.max())
                assert np.allclose(out[b, 0, j].double().cpu().numpy(), p @ v / p.sum(), rtol=2e-3, atol=2e-3)
        assert float(cache.weight[b, :, list(gone)].abs().max()) == 0
    assert float(out[2].abs().max()) == 0 and torch.isneginf(lse[2]).all()
    want, *_ = oracle.attend(want_c, q.double().numpy(), 0.125, 0)
    assert np.allclose(out[3].double().cpu().numpy(), want[3], rtol=2e-3, atol=2e-3)
    # append, evict and read meet them too
    before = (cache.k.clone(), cache.v.clone())
    x = torch.ones((4, 5, 2, 64), dtype=torch.bfloat16, device="cuda")
    counts = torch.tensor([0, 2, 3, 6], dtype=torch.int32, device="cuda")  # 2: page 2^31 - 1; 6 > 5
    _say("append with bad pages, lengths and counts")
    cache.append(x, x, counts)
    assert torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1])
    with pytest.raises(ccb.CcbError):
        cache.check()
    _say("read with bad pages and lengths")
    k, _ = cache.read(100)
    assert float(k[0, 32:48].abs().max()) == 0 and float(k[2].abs().max()) == 0
    assert np.array_equal(k[3].double().cpu().numpy(), np.float32(oracle.read(want_c, 100, [0] * 4)[0][3]).astype(float))
    with pytest.raises(ccb.CcbError):
        cache.check()
    to = kv8.Kv8Cache.allocate(20, 2, 16, 64, 4, 4, "int8", weights=True)
    to.page_table.copy_(torch.arange(16, dtype=torch.int32).view(4, 4))
    to.page_table[3, 1] = -5
    _say("evict with bad pages and lengths")
    cache.evict(to, 40, recent=10)
    with pytest.raises(ccb.CcbError):
        cache.check()
    assert to.lens.tolist() == [40, 40, 0, 40]


# --- append ---------------------------------------------------------------------------

def _append_case(kv8, seed, fmt, dtype, lens, counts, n, heads, P, D, strided=False, special=False, quiet=1.0,
                 null_counts=False):
    rng = np.random.default_rng(seed)
    c = _host(rng, fmt, lens, heads, P, D, quiet=quiet)
    c["weight"] = rng.uniform(0, 1, (len(lens), heads, c["table"].shape[1] * P)).astype(np.float32)
    cache = _device(kv8, c)
    xs = []
    for _ in range(2):
        x = rng.normal(0, 1, (len(lens), n, heads, D)) * rng.choice([0.01, 1, 8], (len(lens), n, heads, 1))
        if special:
            pick = rng.random(x.shape)
            x[pick < 0.02] = np.nan
            x[(pick > 0.02) & (pick < 0.03)] = np.inf
            x[(pick > 0.03) & (pick < 0.04)] = -np.inf
            x[:, :, 0] = 0
            x[0, :, 1] = np.nan
        xs.append(torch.from_numpy(x).to(TYPES[dtype]))
    oracle.append(c, xs[0].double().numpy(), xs[1].double().numpy(), counts)
    dx = [x.cuda() for x in xs]
    if strided:
        dx = [_spread_heads(x, 3) for x in dx]
    dc = None if null_counts else torch.tensor(counts, dtype=torch.int32, device="cuda")
    for again in range(2):  # a second call changes nothing
        cache.append(dx[0], dx[1], dc)
        for which, codes, scales in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
            got = _codes(codes)
            s = scales.cpu().numpy()
            assert np.array_equal(s, c[which + "s"], equal_nan=True), (which, again)
            junk = 0x7F if fmt == "e4m3" else 0x80
            # -0 and 0 are one value
            same = (got == c[which]) | (((got | c[which]) == 0x80) & (fmt == "e4m3") & (junk != 0x80))
            assert same.all(), (which, again, np.argwhere(~same)[:5])
        assert np.array_equal(cache.weight.cpu().numpy(), c["weight"])
    cache.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,P", [(64, 16), (96, 32), (128, 64), (192, 128), (256, 128), (128, 128), (256, 16)])
def test_append_one_token(kv8, fmt, dtype, D, P):
    _say(f"append one token {fmt} {dtype} D={D} P={P}")
    lens = [1, 2, P - 1, P, P + 1, 2 * P, 3 * P + 5]
    _append_case(kv8, D + P, fmt, dtype, lens, [1] * 7, 1, 3, P, D, null_counts=True, quiet=0.3)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,P", [(64, 16), (96, 64), (128, 128), (256, 32)])
@pytest.mark.parametrize("special", [False, True])
def test_append_many_tokens(kv8, fmt, D, P, special):
    _say(f"append many {fmt} D={D} P={P} special={special}")
    _append_case(kv8, P, fmt, "bf16", [300, 77, 5, 200, 0], [300, 70, 0, 129, 0], 300, 2, P, D, strided=True,
                 special=special, quiet=0.1)


def test_append_whole_pages(kv8):
    """Counts and starts that fall on page borders."""
    _say("append whole pages")
    _append_case(kv8, 3, "int8", "fp16", [64, 128, 96, 33], [64, 64, 32, 32], 64, 2, 32, 64)


def test_append_tiny_and_huge_values(kv8):
    """Subnormal values and the largest bf16 values."""
    from cross_core_barrier_amd import ccb  # noqa: F401
    for fmt in ("int8", "e4m3"):
        c = _host(np.random.default_rng(4), fmt, [3, 2], 1, 16, 64)
        cache = _device(kv8, c)
        x = torch.zeros((2, 2, 1, 64), dtype=torch.bfloat16)
        x[0, 0] = torch.linspace(-3.3e38, 3.3e38, 64)
        x[0, 1] = 1e30
        x[1, 0] = 2.0 ** -130
        x[1, 1] = torch.linspace(-1, 1, 64) * 2.0 ** -66
        _say(f"append tiny and huge values {fmt}")
        oracle.append(c, x.double().numpy(), x.double().numpy(), [2, 2])
        cache.append(x.cuda(), x.cuda())
        assert np.array_equal(cache.k_scale.cpu().numpy(), c["ks"], equal_nan=True)
        got = oracle.values(_codes(cache.k), fmt)
        assert np.array_equal(got, oracle.values(c["k"], fmt), equal_nan=True)


# --- evict and read -------------------------------------------------------------------

def _evict_case(kv8, seed, fmt, lens, budget, recent, sinks, heads, P, D, ties=False, shared=True):
    rng = np.random.default_rng(seed)
    batch, out_width = len(lens), -(-budget // P)
    c = _host(rng, fmt, lens, heads, P, D, extra=batch * out_width + 2)
    room = c["table"].shape[1] * P
    w = rng.exponential(1, (batch, heads, room)).astype(np.float32)
    if ties:
        w = np.round(w * 2) / 2
        w[rng.random(w.shape) < 0.05] = np.nan
        w[rng.random(w.shape) < 0.02] = np.inf
        w[rng.random(w.shape) < 0.1] *= -1
    c["weight"] = w.astype(np.float32)
    free = np.setdiff1d(np.arange(c["k"].shape[0]), c["table"])
    to = dict(c, table=rng.permutation(free)[:batch * out_width].astype(np.int32).reshape(batch, out_width),
              lens=np.full(batch, -7, np.int32), weight=np.full((batch, heads, out_width * P), 5, np.float32))
    cache = _device(kv8, c)
    dst = kv8.Kv8Cache(cache.k, cache.v, cache.k_scale, cache.v_scale, torch.from_numpy(to["table"]).cuda(),
                       torch.from_numpy(to["lens"]).cuda(), torch.from_numpy(to["weight"]).cuda())
    index = oracle.evict(c, to, budget, recent, sinks)
    ws = cache.evict_workspace(budget)
    kept = torch.zeros((batch, heads, budget), dtype=torch.int32, device="cuda")
    for again in range(3):  # the workspace is ready for the next call
        kept.zero_()
        dst.weight.fill_(5)
        cache.evict(dst, budget, recent, sinks, kept=kept, workspace=ws)
        assert np.array_equal(kept.cpu().numpy(), index), again
        assert np.array_equal(dst.lens.cpu().numpy(), to["lens"])
        assert np.array_equal(dst.weight.cpu().numpy(), to["weight"], equal_nan=True)
        k, v = dst.read(budget)
        for got, which in ((k, "k"), (v, "v")):
            x = got.double().cpu().numpy()
            for b in range(batch):
                n = to["lens"][b]
                assert np.all(x[b, n:] == 0)
                for h in range(heads):
                    want = oracle.dense(to, which, b, h, np.arange(n)).astype(np.float32).astype(np.float64)
                    assert np.array_equal(x[b, :n, h], want), (again, which, b, h)
    cache.check()
    dst.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,P", [(64, 16), (96, 32), (128, 64), (192, 128), (256, 128)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict(kv8, fmt, D, P, ties):
    _say(f"evict {fmt} D={D} P={P} ties={ties}")
    _evict_case(kv8, D, fmt, [0, 1, 60, 61, 100, 333], 60, 13, 4, 2, P, D, ties)


@pytest.mark.parametrize("budget,recent,sinks", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (700, 0, 0), (700, 696, 4),
                                                 (700, 0, 700), (129, 64, 1), (1025, 100, 4)])
def test_evict_budgets(kv8, budget, recent, sinks):
    _say(f"evict budget={budget} recent={recent} sinks={sinks}")
    _evict_case(kv8, budget, "int8", [2500, 1024, 1025, 3], budget, recent, sinks, 2, 32, 64, ties=True)


@pytest.mark.parametrize("same", [0.0, 1.0, math.nan, -math.inf])
def test_evict_all_alike(kv8, same):
    """Equal weights: the lowest tokens stay."""
    rng = np.random.default_rng(1)
    c = _host(rng, "int8", [3000, 40], 1, 64, 64)
    c["weight"] = np.full((2, 1, c["table"].shape[1] * 64), same, np.float32)
    cache = _device(kv8, c)
    to = kv8.Kv8Cache.allocate(16, 1, 64, 64, 2, 8, "int8", weights=False)
    to.page_table.copy_(torch.arange(16, dtype=torch.int32).view(2, 8))
    kept = torch.zeros((2, 1, 500), dtype=torch.int32, device="cuda")
    _say(f"evict with every weight {same}")
    cache.evict(to, 500, recent=7, sinks=2, kept=kept)
    want = list(range(493)) + list(range(2993, 3000))
    assert kept[0, 0].tolist() == want
    assert kept[1, 0].tolist() == list(range(40)) + [-1] * 460


def test_evict_long(kv8):
    """A long row, many heads: selection over several workgroups' worth."""
    _say("evict 40001 tokens")
    _evict_case(kv8, 2, "int8", [40001, 9000], 2000, 64, 4, 3, 128, 64, ties=True)

@pytest.mark.parametrize("kind", ["ties", "alike", "few", "spread"])
@pytest.mark.parametrize("budget,recent,sinks", [(1, 0, 0), (900, 100, 4), (19000, 0, 0), (5000, 5000, 0)])
def test_evict_rows_in_segments(kv8, kind, budget, recent, sinks):
    """Rows that several workgroups share, beside short and empty ones: the
    kept tokens of a segment start where the ones before it end."""
    rng = np.random.default_rng(budget)
    lens = [30011, 0, 700, 17000, 20480]
    heads, P, D, width = 2, 128, 64, 240
    w = rng.random((5, heads, width * P)).astype(np.float32) ** 8
    if kind == "ties":
        w = np.round(w * 8) / 8
    elif kind == "alike":
        w[:] = 0.25
    elif kind == "few":  # most tokens never drew any weight
        w[rng.random(w.shape) < 0.98] = 0
    pages = torch.from_numpy(rng.permutation(5 * width).astype(np.int32).reshape(5, width)).cuda()
    k = torch.zeros((5 * width, heads, P, D), dtype=torch.int8, device="cuda")
    scales = [torch.ones((5 * width, heads), device="cuda") for _ in range(2)]
    cache = kv8.Kv8Cache(k, k.clone(), *scales, pages, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                         torch.from_numpy(w).cuda())
    rows = -(-budget // P)
    to = kv8.Kv8Cache.allocate(5 * rows, heads, P, D, 5, rows, "int8", weights=True)
    to.page_table.copy_(torch.arange(5 * rows, dtype=torch.int32).view(5, rows))
    _say(f"evict rows in segments, {kind}, budget={budget} recent={recent} sinks={sinks}")
    kept = torch.zeros((5, heads, budget), dtype=torch.int32, device="cuda")
    cache.evict(to, budget, recent, sinks, kept=kept)
    got, gw = kept.cpu().numpy(), to.weight.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(heads):
            want = oracle.kept(w[b, h], n, budget, recent, sinks)
            assert got[b, h].tolist() == want + [-1] * (budget - len(want)), (b, h)
            assert np.array_equal(gw[b, h, :budget], np.r_[w[b, h, want], np.zeros(budget - len(want), np.float32)])
    assert to.lens.tolist() == [min(n, budget) for n in lens]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_on_borders(kv8, fmt, dtype):
    """Values on the border between two codes, and a step to either side: with
    a largest value of Q times a power of two the scale is that power, and
    every border is a value of the type."""
    D, P, n = 256, 16, 16
    q = oracle.Q[fmt]
    grid = np.arange(128.0) if fmt == "int8" else oracle._GRID
    border = (grid[1:] + grid[:-1]) / 2
    c = _host(np.random.default_rng(5), fmt, [n, n, n], 1, P, D)
    cache = _device(kv8, c)
    x = torch.zeros((3, n, 1, D), dtype=TYPES[dtype])
    place = torch.from_numpy(border).to(TYPES[dtype])
    assert torch.equal(place.double(), torch.from_numpy(border))  # exact
    step = torch.finfo(TYPES[dtype]).eps
    for i, scale in enumerate((1.0, 2.0 ** -5, 2.0 ** 4)):
        for j, by in enumerate((1.0, 1 + step, 1 - step / 2, -1.0, -1 - step, -1 + step / 2)):
            x[i, j, 0, :len(border)] = (place.double() * by * scale).to(TYPES[dtype])
        x[i, 6, 0, 0] = q * scale
    _say(f"append on borders {fmt} {dtype}")
    oracle.append(c, x.double().numpy(), -x.double().numpy(), [n] * 3)
    cache.append(x.cuda(), -x.cuda())
    for which, codes in (("k", cache.k), ("v", cache.v)):
        pages = c["table"][:, 0]
        assert np.array_equal(oracle.values(_codes(codes)[pages], fmt), oracle.values(c[which][pages], fmt))
    assert np.array_equal(cache.k_scale.cpu().numpy(), c["ks"], equal_nan=True)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("ratio", [1.5, 2.0, 3.0, 4.0, 6.0, 64.0])
def test_append_rescales_older_codes_on_borders(kv8, fmt, ratio):
    """Every code of an older token under a scale that grows by a simple
    ratio: many land exactly between two codes."""
    D, P = 256, 16
    c = _host(np.random.default_rng(6), fmt, [P], 1, P, D)
    page = c["table"][0, 0]
    ok = [x for x in range(256) if x not in ((0x80,) if fmt == "int8" else (0x7F, 0xFF))]
    for w in ("k", "v"):
        c[w][page, 0, :P - 1] = np.resize(np.array(ok, np.uint8), (P - 1, D))
        c[w + "s"][page] = 0.375
    cache = _device(kv8, c)
    x = torch.zeros((1, 1, 1, D), dtype=torch.bfloat16)
    x[0, 0, 0, 0] = oracle.Q[fmt] * 0.375 * ratio
    _say(f"append rescales on borders {fmt} {ratio}")
    oracle.append(c, x.double().numpy(), x.double().numpy(), [1])
    cache.append(x.cuda(), x.cuda())
    for which, codes, scales in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        assert np.array_equal(scales.cpu().numpy(), c[which + "s"], equal_nan=True)
        assert np.array_equal(oracle.values(_codes(codes)[page], fmt), oracle.values(c[which][page], fmt))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_read(kv8, fmt, dtype):
    rng = np.random.default_rng(3)
    c = _host(rng, fmt, [0, 5, 64, 130], 3, 32, 96)
    cache = _device(kv8, c)
    first = [0, -3, 60, 100]
    _say(f"read {fmt} {dtype}")
    t = {**TYPES, "fp32": torch.float32}[dtype]
    got = cache.read(70, torch.tensor(first, dtype=torch.int32, device="cuda"), dtype=t)
    for x, want in zip(got, oracle.read(c, 70, first)):
        # code * scale as float, then rounded once to the type
        exact = torch.from_numpy(want.astype(np.float32)).to(t)
        assert torch.equal(x.cpu(), exact)
    cache.check()


# --- streams, graphs, far pages --------------------------------------------------------

def _step(cache, k, v, q, ws):
    cache.append(k, v)
    return cache.attend(q, accumulate=True, workspace=ws)


def test_side_stream(kv8):
    rng = np.random.default_rng(20)
    c = _host(rng, "e4m3", [400, 33, 129], 2, 32, 128)
    c["weight"] = np.zeros((3, 2, c["table"].shape[1] * 32), np.float32)
    k, v = (torch.from_numpy(rng.normal(0, 1, (3, 1, 2, 128))).half().cuda() for _ in range(2))
    q = torch.from_numpy(rng.normal(0, 1, (3, 1, 8, 128))).half().cuda()
    a, b = _device(kv8, c), _device(kv8, c)
    s = torch.cuda.Stream()
    _say("append + attend + read on a side stream")
    want = _step(a, k, v, q, None)
    b.append(k, v, stream=s)
    got = b.attend(q, accumulate=True, stream=s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(a.weight, b.weight)
    with torch.cuda.stream(s):
        again = b.read(20)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(again, a.read(20)))


def test_graph_replays(kv8):
    """A whole step and an eviction captured once, replayed with other inputs,
    lengths and pages, with eager work between."""
    rng = np.random.default_rng(21)
    c = _host(rng, "int8", [500, 120, 64], 2, 32, 64, width=20)
    c["weight"] = np.zeros((3, 2, 20 * 32), np.float32)
    cache, plain = _device(kv8, c), _device(kv8, c)
    k, v = (torch.zeros((3, 1, 2, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros((3, 1, 8, 64), dtype=torch.float16, device="cuda")
    to, to_plain = (kv8.Kv8Cache.allocate(9, 2, 32, 64, 3, 3, "int8", weights=True) for _ in range(2))
    for t in (to, to_plain):
        t.page_table.copy_(torch.arange(9, dtype=torch.int32).view(3, 3))
    kept, kept_plain = (torch.zeros((3, 2, 90), dtype=torch.int32, device="cuda") for _ in range(2))
    ws, ews = cache.attend_workspace(8, 1, True), cache.evict_workspace(90)
    out, lse = torch.empty_like(q), torch.empty((3, 1, 8), device="cuda")
    _step(cache, k, v, q, ws)  # once outside the capture
    cache.evict(to, 90, 20, 2, kept=kept, workspace=ews)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.lens.add_(1)
        cache.append(k, v)
        cache.attend(q, accumulate=True, out=out, lse=lse, workspace=ws)
        cache.evict(to, 90, 20, 2, kept=kept, workspace=ews)
    for t in ("k", "v", "k_scale", "v_scale", "weight", "lens"):
        getattr(cache, t).copy_(getattr(plain, t))
    for rep in range(5):
        _say(f"graph replay {rep}")
        for t in (k, v, q):
            t.copy_(torch.from_numpy(rng.normal(0, 1, t.shape)).half())
        if rep == 3:  # other lengths, eagerly (of tokens that were written)
            for x in (cache, plain):
                x.lens.copy_(torch.tensor([3, 119, 40], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        plain.lens.add_(1)
        plain.append(k, v)
        want = plain.attend(q, accumulate=True)
        plain.evict(to_plain, 90, 20, 2, kept=kept_plain)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), rep
        assert torch.equal(cache.weight, plain.weight) and torch.equal(kept, kept_plain), rep
        assert torch.equal(to.lens, to_plain.lens) and torch.equal(to.weight, to_plain.weight), rep
        assert all(torch.equal(x, y) for x, y in zip(to.read(90), to_plain.read(90))), rep


def test_pages_past_32_bits(kv8):
    """Pages whose bytes lie beyond 2^32: every operator on the far end of a
    5.4 GB pool."""
    heads, P, D = 8, 128, 128
    pages = 41_000  # 41,000 * 8 * 128 * 128 bytes
    k, v = (torch.empty((pages, heads, P, D), dtype=torch.int8, device="cuda") for _ in range(2))
    scales = [torch.full((pages, heads), math.nan, device="cuda") for _ in range(2)]
    lens = [300, 129]
    rng = np.random.default_rng(22)
    table = torch.tensor([[pages - 1, pages - 7, pages - 3], [pages - 2, 5, 40_000]], dtype=torch.int32, device="cuda")
    far = kv8.Kv8Cache(k, v, *scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       torch.zeros((2, heads, 3 * P), device="cuda"))
    near = kv8.Kv8Cache.allocate(6, heads, P, D, 2, 3, "int8", weights=True)
    near.page_table.copy_(torch.arange(6, dtype=torch.int32).view(2, 3))
    near.lens.copy_(far.lens)
    x = [torch.from_numpy(rng.normal(0, 1, (2, 300, heads, D))).half().cuda() for _ in range(2)]
    q = torch.from_numpy(rng.normal(0, 1, (2, 1, 16, D))).half().cuda()
    counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    _say("append, attend, evict and read beyond 2^32 bytes")
    results = []
    for c, out_pages in ((far, [[pages - 10], [pages - 9]]), (near, None)):
        c.append(*x, counts)
        got = [*c.attend(q, accumulate=True), c.weight]
        if out_pages is None:
            dst = kv8.Kv8Cache.allocate(2, heads, P, D, 2, 1, "int8", weights=True)
            dst.page_table.copy_(torch.tensor([[0], [1]], dtype=torch.int32))
        else:
            dst = kv8.Kv8Cache(k, v, *scales, torch.tensor(out_pages, dtype=torch.int32, device="cuda"),
                               torch.zeros(2, dtype=torch.int32, device="cuda"),
                               torch.zeros((2, heads, P), device="cuda"))
        kept = torch.zeros((2, heads, 100), dtype=torch.int32, device="cuda")
        c.evict(dst, 100, 10, 2, kept=kept)
        results.append([*got, kept, dst.weight, *dst.read(100), *c.read(300)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_decoding_session(kv8, fmt):
    """Prompts, steps and evictions together (the example's session): replayed
    from a graph and made eagerly they end in the same bits, and a step's
    attention is the oracle's over what the cache holds."""
    from cross_core_barrier_amd.kv8_decode import Session
    ends = []
    for graph in (True, False):
        s = Session(batch=3, heads=2, q_heads=6, head_dim=64, page_size=16, limit=96, budget=40, fmt=fmt, seed=3)
        gen = torch.Generator(device="cuda").manual_seed(7)
        s.prefill([torch.randn((n, s.x.shape[1]), generator=gen, device="cuda").to(s.x.dtype) for n in (70, 5, 33)])
        _say(f"decoding session {fmt} graph={graph}")
        for _ in range(100):
            s.step(graph)
        s.cache.check()
        s.cut.check()
        assert s.evictions == 2 and s.cache.lens.tolist() == s.lens
        used = [p for pages in s.held for p in pages]
        assert len(set(used + s.pages.free)) == len(used) + len(s.pages.free) == s.cache.k.shape[0]
        ends.append((s.x.clone(), s.cache.lens.clone(), s.cache.weight.clone(), *s.cache.read(96)))
    # weights past a sequence's end are whatever was there
    for b, n in enumerate(ends[0][1].tolist()):
        assert torch.equal(ends[0][2][b, :, :n], ends[1][2][b, :, :n])
    for i in (0, 1, 3, 4):
        assert torch.equal(ends[0][i], ends[1][i]), i
    q = torch.randn((3, 1, 6, 64), generator=gen, device="cuda").half()
    c = dict(fmt=fmt, lens=s.cache.lens.cpu().numpy(), table=s.cache.page_table.cpu().numpy(), k=_codes(s.cache.k),
             v=_codes(s.cache.v), ks=s.cache.k_scale.cpu().numpy(), vs=s.cache.v_scale.cpu().numpy())
    want, lse, _, mag, big = oracle.attend(c, q.double().cpu().numpy(), 0.125, 0)
    out, got = s.cache.attend(q, accumulate=True, workspace=None)
    _, tol_lse, tol = _bounds(64, 96, mag, big, lse)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25)
    assert np.all(np.abs(got.double().cpu().numpy() - lse) <= tol_lse)


@pytest.mark.parametrize("D,group,queries", [(64, 5, 4), (96, 11, 3), (96, 3, 16), (128, 5, 4)])
@pytest.mark.parametrize("window", [0, 40])
def test_attend_rows_in_pairs_of_tiles(kv8, D, group, queries, window):
    """More rows than one tile holds in a batch large enough for a workgroup
    to take two tiles of them."""
    _say(f"attend 80 sequences, {group * queries} rows, D={D} window={window}")
    lens = [(i * 29) % 130 for i in range(80)]
    _attend_case(kv8, D + group, "e4m3" if D == 96 else "int8", "bf16", lens, 2, group, D, 32, queries, window)


@pytest.mark.parametrize("window", [0, 2000])
@pytest.mark.parametrize("fmt,dtype", [("int8", "fp16"), ("e4m3", "bf16")])
def test_attend_weights_of_many_rows(kv8, fmt, dtype, window):
    """Rows whose scores are not kept, over several runs of a sequence."""
    _say(f"attend 96 rows, long, {fmt} window={window}")
    _attend_case(kv8, 40, fmt, dtype, [3001, 0, 50, 700], 1, 8, 128, 64, 12, window)


def test_attend_one_run_of_many_pages(kv8):
    """A run longer than the pages a wave can hold at once: many sequences,
    one of them long."""
    _say("attend 130 sequences, one of 12000 tokens")
    _attend_case(kv8, 41, "int8", "bf16", [12000] + [(i * 7) % 90 for i in range(129)], 1, 2, 64, 64)


def test_evict_many_rows_of_few_segments(kv8):
    """So many rows that each has two segments of several steps."""
    rng = np.random.default_rng(42)
    batch, heads, P, D, width = 128, 2, 128, 64, 160
    lens = [20000, 17001, 0, 5, 16385] + [int(x) for x in rng.integers(0, 300, batch - 5)]
    w = rng.random((batch, heads, width * P)).astype(np.float32)
    w[1] = np.round(w[1] * 4)
    k = torch.zeros((50, heads, P, D), dtype=torch.int8, device="cuda")
    scales = [torch.ones((50, heads), device="cuda") for _ in range(2)]
    table = torch.from_numpy(rng.integers(0, 50, (batch, width)).astype(np.int32)).cuda()
    cache = kv8.Kv8Cache(k, k.clone(), *scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                         torch.from_numpy(w).cuda())
    to = kv8.Kv8Cache.allocate(batch * 2, heads, P, D, batch, 2, "int8", weights=True)
    to.page_table.copy_(torch.arange(batch * 2, dtype=torch.int32).view(batch, 2))
    kept = torch.zeros((batch, heads, 200), dtype=torch.int32, device="cuda")
    _say("evict 256 rows, a few of them long")
    cache.evict(to, 200, 20, 4, kept=kept)
    got = kept.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(heads):
            want = oracle.kept(w[b, h], n, 200, 20, 4)
            assert got[b, h].tolist() == want + [-1] * (200 - len(want)), (b, h)
    assert to.lens.tolist() == [min(n, 200) for n in lens]


def test_capacity_far_beyond_the_lengths(kv8):
    """Short sequences in a cache with room for long ones: their runs are as
    short as they are, and the workspace serves any window."""
    rng = np.random.default_rng(30)
    lens = [700, 0, 33, 4100]
    for window in (0, 64, 3000):
        c = _host(rng, "int8", lens, 2, 128, 64, width=200, extra=0)
        _say(f"attend {lens} of 25600, window={window}")
        _attend_case(kv8, 31, "int8", "fp16", lens, 2, 4, 64, 128, queries=2, window=window, c=c)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("P,D", [(16, 64), (128, 256)])
def test_evict_zero_codes_of_a_loud_block(kv8, fmt, P, D):
    """A token of zeros out of a block whose scale is 2^130 times the one its
    new block gets: it stays zeros beside the quiet tokens."""
    rng = np.random.default_rng(50)
    lens = [2 * P, 2 * P]
    c = _host(rng, fmt, lens, 2, P, D, extra=8)
    for b in range(2):
        for w in ("k", "v"):
            c[w + "s"][c["table"][b, 0]] = np.float32(2.0 ** 66)
            c[w + "s"][c["table"][b, 1]] = np.float32(2.0 ** -64)
            c[w][c["table"][b, 0], :, 3] = 0
    c["weight"] = np.zeros((2, 2, c["table"].shape[1] * P), np.float32)
    c["weight"][:, :, [3, P + 5, P + 6]] = 1
    free = np.setdiff1d(np.arange(c["k"].shape[0]), c["table"])[:2].astype(np.int32).reshape(2, 1)
    cache = _device(kv8, c)
    to = kv8.Kv8Cache(cache.k, cache.v, cache.k_scale, cache.v_scale, torch.from_numpy(free).cuda(),
                      torch.zeros(2, dtype=torch.int32, device="cuda"))
    kept = torch.zeros((2, 2, 3), dtype=torch.int32, device="cuda")
    _say(f"evict zero codes of a loud block {fmt} P={P} D={D}")
    cache.evict(to, 3, kept=kept)
    assert kept.tolist() == [[[3, P + 5, P + 6]] * 2] * 2
    dst = dict(c, table=free, lens=np.zeros(2, np.int32), weight=None)
    oracle.evict(c, dst, 3, 0, 0)
    for got, which in zip(to.read(3), ("k", "v")):
        for b in range(2):
            assert np.all(got[b, 0].cpu().numpy() == 0)
            for h in range(2):
                want = oracle.dense(dst, which, b, h, np.arange(3)).astype(np.float32)
                assert np.array_equal(got[b, :, h].cpu().numpy(), want)


@pytest.mark.parametrize("queries,accumulate", [(1, True), (6, True), (33, False), (33, True)])
def test_attend_in_place(kv8, queries, accumulate):
    """out = q gives what a separate out does, or is refused (weights over more
    rows than keep their scores) and changes nothing."""
    from cross_core_barrier_amd import ccb
    rng = np.random.default_rng(51)
    c = _host(rng, "int8", [700, 0, 33], 2, 32, 64)
    c["weight"] = np.zeros((3, 2, c["table"].shape[1] * 32), np.float32)
    a, b = _device(kv8, c), _device(kv8, c)
    q = torch.from_numpy(rng.normal(0, 1, (3, queries, 6, 64))).half().cuda()
    want, lse = a.attend(q, accumulate=accumulate)
    mine = q.clone()
    _say(f"attend in place, {queries} queries, accumulate={accumulate}")
    if accumulate and 3 * queries > 64:
        with pytest.raises(ccb.CcbError):
            b.attend(mine, accumulate=True, out=mine)
        assert torch.equal(mine, q) and float(b.weight.abs().max()) == 0
        return
    got, got_lse = b.attend(mine, accumulate=accumulate, out=mine)
    assert got is mine and torch.equal(got, want) and torch.equal(got_lse, lse)
    assert torch.equal(a.weight, b.weight)


@pytest.mark.parametrize("fmt,dtype,D,P,heads,group", [("int8", "bf16", 128, 64, 4, 4), ("e4m3", "fp16", 192, 128, 1, 3),
                                                       ("int8", "fp16", 96, 32, 2, 5), ("e4m3", "bf16", 256, 16, 1, 8),
                                                       ("int8", "bf16", 64, 128, 1, 16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_attend_joins_many_runs(kv8, fmt, dtype, D, P, heads, group, accumulate):
    """More runs of one sequence than a wave joins: a workgroup for each row."""
    _say(f"attend 17011 tokens, {heads} heads {fmt} {dtype} D={D} P={P} accumulate={accumulate}")
    _attend_case(kv8, 60, fmt, dtype, [17011], heads, group, D, P, accumulate=accumulate)


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "fp16"), ("int8", "fp16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("D,P,window", [(96, 16, 0), (192, 64, 77), (256, 128, 0)])
def test_attend_weights_computed_again(kv8, fmt, dtype, D, P, window):
    """More rows than scores are kept for, in every head size."""
    _say(f"attend 70 rows {fmt} {dtype} D={D} P={P} window={window}")
    _attend_case(kv8, 61, fmt, dtype, [300, 0, 13, 700], 2, 5, D, P, 14, window)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("P,budget", [(128, 128), (128, 129), (128, 256), (128, 257), (64, 128), (64, 129), (32, 128),
                                      (32, 97), (16, 128), (16, 129), (16, 113)])
def test_evict_in_one_kernel_and_in_two(kv8, fmt, P, budget):
    """Budgets at the largest that the selection's own workgroup moves, and one more."""
    _say(f"evict {fmt} P={P} budget={budget}")
    _evict_case(kv8, P, fmt, [600, 128, 256, 257, 0, 129], budget, 11, 3, 2, P, 96, ties=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("side", ["k", "v"])
def test_read_one_side(kv8, side, dtype):
    """Keys alone or values alone, through the C entry point."""
    from cross_core_barrier_amd import ccb
    rng = np.random.default_rng(62)
    c = _host(rng, "e4m3", [0, 5, 64, 130], 3, 32, 96)
    cache = _device(kv8, c)
    kind = {"bf16": ccb.CCB_KV8_BF16, "fp16": ccb.CCB_KV8_FP16, "fp32": ccb.CCB_KV8_FP32}[dtype]
    t = {**TYPES, "fp32": torch.float32}[dtype]
    out = torch.full((4, 150, 3, 96), 7, dtype=t, device="cuda")
    rows = ccb.ccbKv8Rows(out.data_ptr(), *out.stride()[:3], kind, 0)
    _say(f"read {side} alone as {dtype}")
    assert ccb.ccb_kv8_read(cache._c, rows if side == "k" else None, rows if side == "v" else None, 150) == 0
    want = torch.from_numpy(oracle.read(c, 150, [0] * 4)["kv".index(side)].astype(np.float32)).to(t)
    assert torch.equal(out.cpu(), want)


def test_an_error_left_by_another_call_is_not_reported(kv8):
    """A HIP call that failed before, in the caller's own code, says nothing
    of the cache's calls: they run and return OK, and leave that error be."""
    import ctypes
    from cross_core_barrier_amd import ccb
    with open("/proc/self/maps") as f:  # the runtime that is loaded
        hip = ctypes.CDLL(next(line.split()[-1] for line in f if "libamdhip64" in line))
    rng = np.random.default_rng(63)
    c = _host(rng, "int8", [60, 5], 2, 16, 64)
    c["weight"] = np.zeros((2, 2, c["table"].shape[1] * 16), np.float32)
    cache = _device(kv8, c)
    x = torch.from_numpy(rng.normal(0, 1, (2, 1, 2, 64))).half().cuda()
    q = torch.from_numpy(rng.normal(0, 1, (2, 1, 4, 64))).half().cuda()
    out, lse, ws = torch.empty_like(q), torch.empty((2, 1, 4), device="cuda"), cache.attend_workspace(4, 1, True)
    to = kv8.Kv8Cache.allocate(4, 2, 16, 64, 2, 2, "int8", weights=True)
    to.page_table.copy_(torch.arange(4, dtype=torch.int32).view(2, 2))
    kept, ews = torch.zeros((2, 2, 20), dtype=torch.int32, device="cuda"), cache.evict_workspace(20)
    dense = torch.empty((2, 20, 2, 64), device="cuda")
    rows = ccb.ccbKv8Rows(dense.data_ptr(), *dense.stride()[:3], ccb.CCB_KV8_FP32, 0)
    calls = {"append": lambda: cache.append(x, x),
             "attend": lambda: cache.attend(q, accumulate=True, out=out, lse=lse, workspace=ws),
             "evict": lambda: cache.evict(to, 20, 4, 2, kept=kept, workspace=ews),
             "read": lambda: ccb.check(ccb.ccb_kv8_read(cache._c, rows, None, 20))}
    torch.cuda.synchronize()
    for name, call in calls.items():
        _say(f"{name} behind another call's error")
        hip.hipGetLastError()
        assert hip.hipSetDevice(1 << 20) != 0  # refused by the host: no such device
        try:
            call()
        finally:
            left = hip.hipGetLastError()
        assert left != 0, name
    torch.cuda.synchronize()
    cache.check()
