"""Attention over the 4-bit cache at scores far beyond what a weight's exponent
holds, against the oracle in 64 bits, on inputs whose results are exact: every
score is a power of two, so that its product with scale * log2 e is exact in 32
bits, tokens at a row's maximum tie, and all others are further behind than any
weight reaches.  A row's output is then the mean of its tied tokens' values,
whose sum is exact in 32 bits too (multiples of a half, below 2^18)."""

import numpy as np
import pytest

from oracle import kv4 as oracle

torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
D, P, DIM = 64, 16, 5  # DIM: the one dimension where queries are not zero
U = 2.0 ** -24

# Queries are +-2^r there.  The last row's sign is turned: its maximum is the others' minimum.
ROWS = {"bf16": [(1, 0), (1, 9), (1, 40), (-1, 12)], "fp16": [(1, 0), (1, 9), (1, 15), (-1, 12)]}


def _cache(rng, lens, level):
    """level(b, n): the signs and exponents of a sequence's keys at DIM, two arrays."""
    width = -(-max(lens) // P) + 1
    pages = len(lens) * width + 2
    c = dict(lens=np.array(lens, np.int32),
             table=rng.permutation(pages)[:len(lens) * width].astype(np.int32).reshape(len(lens), width),
             k=rng.integers(0, 256, (pages, 1, P, D // 2)).astype(np.uint8),
             v=rng.integers(0, 256, (pages, 1, P, D // 2)).astype(np.uint8),
             ks=rng.integers(100, 150, (pages, 1, P, D // 32)).astype(np.uint8),
             vs=np.full((pages, 1, P, D // 32), 127, np.uint8))
    for b, n in enumerate(lens):
        sign, x = level(b, n)
        t = np.arange(n)
        at = (c["table"][b, t // P], 0, t % P)
        old = c["k"][at + (DIM // 2,)]
        code = np.where(sign > 0, 2, 10)  # +-1
        c["k"][at + (DIM // 2,)] = (old & 0x0f) | (code << 4) if DIM % 2 else (old & 0xf0) | code
        c["ks"][at + (DIM // 32,)] = 127 + x
    return c


def _levels(place, base, top):
    """Tokens at `top` among others at `base`; a pair is a sign and an exponent."""
    def level(b, n):
        sign, x = np.full(n, base[0]), np.full(n, base[1])
        for t in PLACES[place](n):
            sign[t], x[t] = top
        return sign, x
    return level


def _steps(up):
    """A higher (or lower) level in every tile of wave 0, across the border of 2^20 for every row."""
    def level(b, n):
        x = np.full(n, -2)
        steps = [4, 7, 10, 13, 16, 18, 19, 20, 21, 24, 30, 50]
        for i, t in enumerate(range(1, n, 256)):
            x[t] = steps[i % 12 if up else -1 - i % 12]
        return np.ones(n, np.int64), x
    return level


PLACES = {
    "first tile": lambda n: [3, 17],
    "later tiles": lambda n: [t for t in (3 + 256, 30 + 512, 7 + 768) if t < n],
    "another wave": lambda n: [40, 101, 255],
    "the end": lambda n: [n - 1, max(0, n - 33)],
    "everywhere": lambda n: [t for t in (0, 31, 32, 200, 256, 777, 1500, n - 1) if t < n],
}
# lengths: one workgroup; runs joined within the kernel, of one tile a wave and of two; joined by a kernel of their own
LENS = {"whole": [1280, 300], "cut": [3000, 259], "cut in twos": [2600] * 24, "many runs": [20000]}
LEVELS = [((1, 3), (1, 10)), ((1, 12), (1, 40)), ((-1, 40), (-1, 10)), ((-1, 30), (1, 11)), ((-1, 18), (-1, 13))]
CASES = [(lens, place, *pair) for lens in LENS for place in PLACES for pair in LEVELS] + \
        [(lens, "up" if up else "down", None, None) for lens in LENS for up in (True, False)]


def _make(dtype, lens, place, base, top):
    rng = np.random.default_rng([len(place), len(lens), LENS[lens][0]])
    level = _steps(place == "up") if base is None else _levels(place, base, top)
    c = _cache(rng, LENS[lens], level)
    q = np.zeros((len(c["lens"]), 1, 4, D))
    for j, (sign, r) in enumerate(ROWS[dtype]):
        q[:, 0, j, DIM] = sign * 2.0 ** r
    return c, q


def _holds(dtype, want, lse, y, z):
    """out: its rounding (half a step of fp16's subnormals is 2^-25; below 2^-120 are
    the oracle's weights of tokens far behind), and a division's in 32 bits (3 ulps
    at most).  lse: the
    constants log2 e and ln 2, and the sum's and the product's rounding (5 u in
    all), and two ulps of a logarithm below 16."""
    eps, tiny = torch.finfo(TYPES[dtype]).eps / 2, 2.0 ** -25 if dtype == "fp16" else 2.0 ** -120
    return bool(np.all(np.abs(y - want) <= (eps * (1 + 2.0 ** -10) + 6 * U) * np.abs(want) + tiny)
                and np.all(np.abs(z - lse) <= 5 * U * np.abs(lse) + 32 * U))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,place,base,top", CASES[:25] + CASES[-2:], ids=str)
def test_wrong_results_are_seen(dtype, lens, place, base, top):
    """The bound on results that are wrong: planted in the oracle's."""
    c, q = _make(dtype, "whole", place, base, top)
    want, lse, _, _ = oracle.attend(c, q, 1.0, 0)
    rounded = torch.from_numpy(want).to(TYPES[dtype]).double().numpy()
    good = lse.astype(np.float32).astype(np.float64)
    assert _holds(dtype, want, lse, rounded, good)
    assert np.abs(want).max() > 0.1 and np.isfinite(lse).all()
    for wrong in (rounded * 0, -rounded, rounded * 100, rounded * 1.01):
        assert not _holds(dtype, want, lse, wrong, good)
    assert not _holds(dtype, want, lse, rounded, good * (1 + 2.0 ** -20))
    # one of a row's tied tokens left out, and one with half its weight more
    for b, n in enumerate(c["lens"]):
        k, v = (oracle.dense(c, w, b, 0, np.arange(n)) for w in ("k", "v"))
        for j in range(4):
            s = k @ q[b, 0, j]
            tied = np.flatnonzero(s == s.max())
            if not 2 <= len(tied) <= 8:
                continue
            assert np.array_equal(want[b, 0, j], v[tied].mean(0)) or np.allclose(want[b, 0, j], v[tied].mean(0), rtol=1e-9)
            for weights in (np.r_[0, np.ones(len(tied) - 1)], np.r_[1.5, np.ones(len(tied) - 1)]):
                other = rounded.copy()
                other[b, 0, j] = weights @ v[tied] / weights.sum()
                assert not _holds(dtype, want, lse, other, good)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,place,base,top", CASES, ids=str)
def test_attend_loud(dtype, lens, place, base, top):
    from cross_core_barrier_amd import kv4
    print(f"[gpu case] attend loud {dtype} {lens} {place} {base} {top}", flush=True)
    c, q = _make(dtype, lens, place, base, top)
    want, lse, _, _ = oracle.attend(c, q, 1.0, 0)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cache = kv4.Kv4Cache(up(c["k"]), up(c["v"]), up(c["ks"]), up(c["vs"]), up(c["table"]), up(c["lens"]))
    out, got = cache.attend(torch.from_numpy(q).to(TYPES[dtype]).cuda(), scale=1.0)
    assert _holds(dtype, want, lse, out.double().cpu().numpy(), got.double().cpu().numpy())
    cache.check()
