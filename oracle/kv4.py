"""Oracle of the 4-bit key/value cache (include/ccb_kv4.h): append, attention
and read from their definitions, in 64-bit numpy on the CPU, one sequence and
head at a time.  Shares no code with the library.

A cache is a dict of numpy arrays: k, v uint8 [pages, heads, P, D / 2] (two
codes to a byte), ks, vs uint8 [pages, heads, P, D / 32] (e8m0), table int32
[batch, n], lens int32 [batch].
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

GROUP = 32


def e2m1_value(code: int) -> float:
    e, m = (code >> 1) & 3, code & 1
    x = m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
    return -x if code & 8 else x


_E2M1 = np.array([e2m1_value(c) for c in range(16)])
GRID = [Fraction(x) for x in _E2M1[:8]]  # ascending


def nearest_code(x: Fraction) -> int:
    """The code next to an exact number, ties to the even code, saturated."""
    size = abs(x)
    best = min(range(8), key=lambda i: (abs(size - GRID[i]), i % 2))
    return best | (8 if x < 0 else 0)


def exponent(a: Fraction) -> int:
    """The exponent of the scale for numbers up to a in size."""
    e = -64
    while e < 125 and a > 7 * Fraction(2) ** e:
        e += 1
    return e


def quantise(x: np.ndarray):
    """x float64 [..., D] as (codes [..., D / 2], scales [..., D / 32])."""
    flat = x.reshape(-1, GROUP)
    codes = np.zeros(flat.shape, np.uint8)
    scales = np.zeros(flat.shape[0], np.uint8)
    grid = _E2M1[:8]
    for i, row in enumerate(flat):
        fine = np.abs(row[np.isfinite(row)])
        e = exponent(Fraction(float(fine.max()))) if fine.size else -64
        scales[i] = e + 127
        # 64 bits hold a 16-bit number over a power of two, and the borders, exactly
        y = np.where(np.isnan(row), 0.0, np.clip(np.abs(row) * 2.0 ** -e, 0, 6))
        hi = np.clip(np.searchsorted(grid, y), 1, 7)
        low, high = y - grid[hi - 1], grid[hi] - y
        code = np.where((high < low) | ((high == low) & (hi % 2 == 0)), hi, hi - 1)
        codes[i] = code | np.where(np.signbit(row) & ~np.isnan(row), 8, 0)
    codes = codes.reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return codes[..., 0] | (codes[..., 1] << 4), scales.reshape(*x.shape[:-1], x.shape[-1] // GROUP)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 [..., D]."""
    both = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    with np.errstate(over="ignore"):
        return _E2M1[both] * np.repeat(2.0 ** (scales.astype(np.float64) - 127), GROUP, -1)


def append(c: dict, k_new: np.ndarray, v_new: np.ndarray, slots) -> None:
    """In place; k_new, v_new float64 [n, heads, D]."""
    P = c["k"].shape[2]
    for w, x in (("k", k_new), ("v", v_new)):
        codes, scales = quantise(x)
        for i, s in enumerate(slots):
            if s >= 0:
                c[w][s // P, :, s % P] = codes[i]
                c[w + "s"][s // P, :, s % P] = scales[i]


def dense(c: dict, which: str, b: int, h: int, tokens) -> np.ndarray:
    """Sequence b's values of head h at the given tokens, float64 [n, D]."""
    P = c["k"].shape[2]
    t = np.asarray(tokens, dtype=np.int64)
    page = c["table"][b, t // P]
    return values(c[which][page, h, t % P], c[which + "s"][page, h, t % P])


def attend(c: dict, q: np.ndarray, scale: float, window: int):
    """q float64 [batch, queries, q_heads, D].  Returns out, lse, and what an
    error bound needs: sum p |v| like out, and per query the largest sum
    |q k| * |scale|."""
    batch, queries, q_heads, D = q.shape
    heads = c["k"].shape[1]
    group = q_heads // heads
    out, mag = np.zeros_like(q), np.zeros_like(q)
    lse = np.full(q.shape[:3], -math.inf)
    big = np.zeros(q.shape[:3])
    for b in range(batch):
        n = int(c["lens"][b])
        for h in range(heads):
            k, v = (dense(c, w, b, h, np.arange(n)) for w in ("k", "v"))
            for i in range(queries):
                end = n - queries + i + 1
                begin = max(0, end - window) if window else 0
                if end <= begin:
                    continue
                for j in range(h * group, (h + 1) * group):
                    s = (k[begin:end] @ q[b, i, j]) * scale
                    big[b, i, j] = (np.abs(k[begin:end]) @ np.abs(q[b, i, j])).max() * abs(scale)
                    m = s.max()
                    p = np.exp(s - m)
                    out[b, i, j] = p @ v[begin:end] / p.sum()
                    mag[b, i, j] = p @ np.abs(v[begin:end]) / p.sum()
                    lse[b, i, j] = m + math.log(p.sum())
    return out, lse, mag, big


def read(c: dict, count: int, first):
    """(k, v) float64 [batch, count, heads, D]; zeros where no token is."""
    heads, P, half = c["k"].shape[1:]
    got = []
    for w in ("k", "v"):
        x = np.zeros((len(c["lens"]), count, heads, 2 * half))
        for b, n in enumerate(c["lens"]):
            t = np.arange(first[b], first[b] + count)
            ok = (t >= 0) & (t < n)
            for h in range(heads):
                x[b, ok, h] = dense(c, w, b, h, t[ok])
        got.append(x)
    return got
