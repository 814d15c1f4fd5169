"""Oracle of the 8-bit key/value cache (include/ccb_kv8.h): append, attention,
eviction and read from their definitions, in 64-bit numpy on the CPU, one
sequence and head at a time.  Shares no code with the library.

A cache is a dict of numpy arrays: k, v uint8 [pages, heads, P, D] (the codes'
bytes), ks, vs float32 [pages, heads], table int32 [batch, n], lens int32
[batch], weight float32 [batch, heads, tokens] or None; and fmt "int8" or
"e4m3".
"""

from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

Q = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -64


def e4m3_value(code: int) -> float:
    sign, e, m = code >> 7, (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -x if sign else x


_E4M3 = np.array([e4m3_value(c) for c in range(256)])
_GRID = _E4M3[:127]  # values of the non-negative codes, ascending


def values(codes: np.ndarray, fmt: str) -> np.ndarray:
    return codes.view(np.int8).astype(np.float64) if fmt == "int8" else _E4M3[codes]


def nearest_code(x: Fraction, fmt: str) -> int:
    """The code next to an exact number, ties to the even code, saturated."""
    size, sign = abs(x), x < 0
    if fmt == "int8":
        n = min(round(size), 127)  # Fraction rounds half to even
        return (-n if sign else n) & 255
    top = len(_GRID) - 1
    i = int(np.searchsorted(_GRID, float(min(size, Fraction(500))), side="right")) - 1
    i = max(0, min(i, top))
    while i > 0 and Fraction(_GRID[i]) > size:
        i -= 1
    while i < top and Fraction(_GRID[i + 1]) <= size:
        i += 1
    if i < top:
        low, high = size - Fraction(_GRID[i]), Fraction(_GRID[i + 1]) - size
        if high < low or (high == low and i % 2 == 1):
            i += 1
    return i | (128 if sign else 0)


def encode(x: np.ndarray, s: np.ndarray, fmt: str) -> np.ndarray:
    """Codes of x / s, rounded once.  x and s are float64 that hold at most 32
    and 24 significant bits: the 64-bit quotient of two such numbers is at
    least 2^-35 away (relatively) from any border it does not lie on."""
    x, s = np.broadcast_arrays(np.asarray(x, np.float64), np.asarray(s, np.float64))
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(s > 0, x / s, 0.0)
    r = np.where(np.isnan(r), 0.0, np.clip(r, -Q[fmt], Q[fmt]))
    if fmt == "int8":
        return np.round(r).astype(np.int8).view(np.uint8)
    size = np.abs(r)
    hi = np.clip(np.searchsorted(_GRID, size), 1, len(_GRID) - 1)
    low, high = size - _GRID[hi - 1], _GRID[hi] - size
    code = np.where((high < low) | ((high == low) & (hi % 2 == 0)), hi, hi - 1)
    return (code | np.where((r < 0) | ((r == 0) & np.signbit(x)), 128, 0)).astype(np.uint8)


def block_scale(a: float, fmt: str) -> np.float32:
    if not a > 0:
        return np.float32(0)
    return np.maximum(np.float32(np.float64(np.float32(a)) / Q[fmt]), np.float32(TINY))


def append(c: dict, k_new: np.ndarray, v_new: np.ndarray, counts) -> None:
    """In place; k_new, v_new float64 [batch, n, heads, D]."""
    P = c["k"].shape[2]
    for b, (n, cnt) in enumerate(zip(c["lens"], counts)):
        start = n - cnt
        for number in range(start // P, -(-n // P) if cnt else 0):
            page = c["table"][b, number]
            lo, hi = max(start - number * P, 0), min(n - number * P, P)
            if lo >= hi:
                continue
            for codes, scales, x in ((c["k"], c["ks"], k_new), (c["v"], c["vs"], v_new)):
                for h in range(codes.shape[1]):
                    new = x[b, number * P + lo - start:number * P + hi - start, h]
                    fine = np.abs(new[np.isfinite(new)])
                    s1 = block_scale(fine.max() if fine.size else 0.0, c["fmt"])
                    s0 = scales[page, h] if lo > 0 else np.float32(0)
                    s = max(s0, s1)
                    if lo > 0 and s > s0:
                        old = values(codes[page, h, :lo], c["fmt"]) * np.float64(s0)
                        codes[page, h, :lo] = encode(old, np.float64(s), c["fmt"])
                    codes[page, h, lo:hi] = encode(new, np.float64(s), c["fmt"])
                    scales[page, h] = s
        if c["weight"] is not None:
            c["weight"][b, :, start:n] = 0


def dense(c: dict, which: str, b: int, h: int, tokens) -> np.ndarray:
    """Sequence b's values of head h at the given tokens, float64 [n, D]."""
    P = c["k"].shape[2]
    t = np.asarray(tokens, dtype=np.int64)
    page = c["table"][b, t // P]
    return values(c[which][page, h, t % P], c["fmt"]) * c[which + "s"][page, h].astype(np.float64)[:, None]


def attend(c: dict, q: np.ndarray, scale: float, window: int):
    """q float64 [batch, queries, q_heads, D].  Returns out, lse, the weight
    each token draws [batch, heads, tokens], and what an error bound needs:
    sum p |v| like out, and per query the largest sum |q k| * scale."""
    batch, queries, q_heads, D = q.shape
    heads = c["k"].shape[1]
    group = q_heads // heads
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    big = np.zeros(q.shape[:3])
    room = c["table"].shape[1] * c["k"].shape[2]
    weight = np.zeros((batch, heads, room))
    for b, n in enumerate(c["lens"]):
        for i in range(queries):
            end = n - queries + i + 1
            begin = max(0, end - window) if window else 0
            if end <= begin:
                continue
            t = np.arange(begin, end)
            for h in range(heads):
                k, v = dense(c, "k", b, h, t), dense(c, "v", b, h, t)
                for j in range(h * group, (h + 1) * group):
                    s = k @ q[b, i, j] * scale
                    m = s.max()
                    e = np.exp(s - m)
                    p = e / e.sum()
                    out[b, i, j] = p @ v
                    mag[b, i, j] = p @ np.abs(v)
                    lse[b, i, j] = m + np.log(e.sum())
                    big[b, i, j] = (np.abs(k) @ np.abs(q[b, i, j])).max() * abs(scale)
                    weight[b, h, begin:end] += p
    return out, lse, weight, mag, big


def kept(weight: np.ndarray, n: int, budget: int, recent: int, sinks: int) -> list:
    """The tokens of one sequence and head that stay, ascending."""
    if n <= budget:
        return list(range(n))
    middle = list(range(sinks, n - recent))
    # a NaN ranks below every number; equal weights: the lower token first
    middle.sort(key=lambda t: (1, 0.0, t) if math.isnan(weight[t]) else (0, -float(weight[t]), t))
    return sorted(list(range(sinks)) + middle[:budget - recent - sinks] + list(range(n - recent, n)))


def evict(c: dict, to: dict, budget: int, recent: int, sinks: int):
    """Fills `to` (its table given) from c; returns kept [batch, heads, budget]."""
    P, heads = c["k"].shape[2], c["k"].shape[1]
    index = np.full((len(c["lens"]), heads, budget), -1, np.int32)
    for b, n in enumerate(c["lens"]):
        to["lens"][b] = min(n, budget)
        for h in range(heads):
            stay = np.array(kept(c["weight"][b, h], n, budget, recent, sinks), dtype=np.int64)
            index[b, h, :len(stay)] = stay
            if to["weight"] is not None:
                to["weight"][b, h, :budget] = 0
                to["weight"][b, h, :len(stay)] = c["weight"][b, h, stay]
            for number in range(-(-len(stay) // P)):
                part = stay[number * P:(number + 1) * P]
                page = to["table"][b, number]
                for which in ("k", "v"):
                    src = c["table"][b, part // P]
                    code = values(c[which][src, h, part % P], c["fmt"])
                    s = c[which + "s"][src, h]
                    size = (np.abs(code).max(1).astype(np.float32) * s).max()
                    s1 = block_scale(size, c["fmt"])
                    to[which][page, h, :len(part)] = encode(code * s.astype(np.float64)[:, None], np.float64(s1),
                                                            c["fmt"])
                    to[which + "s"][page, h] = s1
    return index


def read(c: dict, count: int, first):
    batch, heads, D = len(c["lens"]), c["k"].shape[1], c["k"].shape[3]
    outs = []
    for which in ("k", "v"):
        o = np.zeros((batch, count, heads, D))
        for b, n in enumerate(c["lens"]):
            t = np.arange(first[b], first[b] + count)
            there = (t >= 0) & (t < n)
            for h in range(heads):
                o[b, there, h] = dense(c, which, b, h, t[there])
        outs.append(o)
    return outs
