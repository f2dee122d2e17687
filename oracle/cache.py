"""Paged K / V cache and the attention of new tokens over it, in float64.

Test infrastructure only (see the package docstring); numpy, no code of the
library.  The definitions are those of include/dynrad.h: token i of the n that
cu_seq gives sequence s stands at position kv_len[s] - n + i; 8-bit pages carry
one scale 2^(byte - 127) for every 32 channels.
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 32
LEAST_EXPONENT = -117
LIMIT = {"fp8": 448.0, "int8": 127.0}
LARGEST = {"fp8": 240.0 * 2.0 ** 120, "int8": 127.0 * 2.0 ** 121}   # stored magnitude that bf16 still holds


def e4m3_grid() -> np.ndarray:
    """Values of the 127 finite non-negative e4m3 codes, ascending by code."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


def round_e4m3(y: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 numbers (ties to the even code), |y| <= 448."""
    grid = e4m3_grid()
    a = np.abs(y)
    hi = np.minimum(np.searchsorted(grid, a, side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == grid[hi], hi, code)
    return (code + 128 * np.signbit(y)).astype(np.uint8)


def quantise(x: np.ndarray, fmt: str):
    """float64 [..., D] -> (codes uint8 [..., D], exponent bytes uint8 [..., D / 32])."""
    g = x.reshape(x.shape[:-1] + (-1, GROUP))
    bad = ~np.isfinite(g).all(-1)
    g = np.clip(np.where(bad[..., None], 0.0, g), -LARGEST[fmt], LARGEST[fmt])
    a = np.abs(g).max(-1)
    e = np.full(a.shape, LEAST_EXPONENT)
    while True:     # least e >= LEAST_EXPONENT with a <= limit * 2^e
        short = a > LIMIT[fmt] * np.exp2(e.astype(np.float64))
        if not short.any():
            break
        e = e + short
    y = g / np.exp2(e.astype(np.float64))[..., None]
    code = round_e4m3(y) if fmt == "fp8" else np.rint(y).astype(np.int8).view(np.uint8)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    return code.reshape(x.shape), np.where(bad, 255, e + 127).astype(np.uint8)


def stands_for(code: np.ndarray, scale: np.ndarray, fmt: str) -> np.ndarray:
    """What codes [..., D] with exponent bytes [..., D / 32] stand for (float64)."""
    if fmt == "fp8":
        grid = np.concatenate([e4m3_grid(), [480.0]])
        v = grid[code & 127] * np.where(code & 128, -1.0, 1.0)
    else:
        v = code.view(np.int8).astype(np.float64)
    s = np.where(scale == 255, math.nan, np.exp2(scale.astype(np.float64) - 127))
    return (v.reshape(v.shape[:-1] + (-1, GROUP)) * s[..., None]).reshape(v.shape)


def place(table: np.ndarray, page: int, s: int, pos: int):
    return int(table[s, pos // page]), pos % page


def seen(frame: int, window: int, x: int, length: int):
    """Positions [lo, hi) that position x sees."""
    if frame == 0:
        return 0, length
    if x < 0:
        return 0, 0
    f = x // frame
    return (max(0, (f - window + 1) * frame) if window else 0), min(length, (f + 1) * frame)


def attend(q, keys, values, length, frame, window, scale):
    """One sequence and one K / V head.  q [n, g, D] float64 (the n tokens end at
    position length - 1), keys / values [length, D].  Returns o, lse and, for
    error bounds, sum softmax |v| per channel and max sum |q k| scale per row."""
    n, g, d = q.shape
    o, lse = np.zeros((n, g, d)), np.full((n, g), -math.inf)
    absv, absqk = np.zeros((n, g, d)), np.zeros((n, g))
    for i in range(n):
        lo, hi = seen(frame, window, length - n + i, length)
        if hi <= lo:
            continue
        k, v = keys[lo:hi], values[lo:hi]
        a = (q[i] @ k.T) * scale
        m = a.max(1, keepdims=True)
        p = np.exp(a - m)
        total = p.sum(1, keepdims=True)
        w = p / total
        o[i], lse[i] = w @ v, (m + np.log(total))[:, 0]
        absv[i] = w @ np.abs(v)
        absqk[i] = (np.abs(q[i]) @ np.abs(k).T).max(1) * scale
    return o, lse, absv, absqk
