"""The paged cache's operators written out plainly in float64 (test infrastructure only).

Sequence by sequence, head by head, from the formulas in include/cp.h: the
rotary angle is pos * base^(-2j/D), the e4m3 scale the least power of two
2^e (e >= -110) with max |x| <= 448 * 2^e, attention a softmax over the visible
positions. Next to the attention's values stand the two sums that bound what
rounding may do to them.
"""
from __future__ import annotations

import numpy as np

MIN_EXP = -110


def e4m3_table() -> np.ndarray:
    """The value of each e4m3 byte (0x7f and 0xff are NaN)."""
    b = np.arange(256)
    ex, man = (b >> 3) & 15, b & 7
    v = np.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * 2.0 ** (ex - 7.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b > 127, -v, v)


def scale_exp(x: np.ndarray) -> np.ndarray:
    """Exponent of each row's scale (the last axis is the row)."""
    a = np.where(np.isfinite(x), np.abs(x), 0).max(-1)
    e = np.full(a.shape, MIN_EXP, np.int64)
    while True:
        up = a > 448.0 * np.exp2(e.astype(np.float64))
        if not up.any():
            return e
        e[up] += 1


def quantise(x: np.ndarray):
    """(bytes, exponents) of rows x[..., D], nearest, ties to the even byte."""
    table = e4m3_table()[:127]
    e = scale_exp(x)
    z = x / np.exp2(e.astype(np.float64))[..., None]
    a = np.where(np.isfinite(z), np.abs(z), 0)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    below, above = a - table[lo], table[hi] - a
    byte = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    byte = np.where(np.signbit(z), byte + 128, byte)
    return np.where(np.isfinite(x), byte, 127).astype(np.uint8), e


def dequantise(byte: np.ndarray, e: np.ndarray) -> np.ndarray:
    return e4m3_table()[byte] * np.exp2(e.astype(np.float64))[..., None]


def norm_rope(x: np.ndarray, pos: np.ndarray, gain, eps: float, base: float) -> np.ndarray:
    """x [n][heads][D] at positions pos [n]."""
    d = x.shape[-1]
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain
    if base:
        ang = pos[:, None] * float(base) ** (-2.0 * np.arange(d // 2) / d)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = x[..., :d // 2], x[..., d // 2:]
        x = np.concatenate([a * c - b * s, b * c + a * s], -1)
    return x


def attend(q, k, v, first: int, scale: float, causal: bool, window: int):
    """q [n][Hq][D] at positions first.., k and v [T][Hkv][D]. Returns the output [n][Hq][D], the weighted sum of
    |v| of the same shape, and the largest sum |q_i k_i| * scale over the row's visible positions [n][Hq]."""
    n, hq, d = q.shape
    t = np.arange(k.shape[0])
    out, size, reach = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq))
    for i in range(n):
        p = first + i
        see = np.ones(len(t), bool)
        if causal:
            see &= t <= p
        if window:
            see &= t > p - window
        if not see.any():
            continue
        for h in range(hq):
            g = h // (hq // k.shape[1])
            ks, vs = k[see, g], v[see, g]
            a = ks @ q[i, h] * scale
            w = np.exp(a - a.max())
            w /= w.sum()
            out[i, h], size[i, h] = w @ vs, w @ np.abs(vs)
            reach[i, h] = (np.abs(ks) @ np.abs(q[i, h])).max() * scale
    return out, size, reach
