"""Projections with 4-bit weights in float64 (test infrastructure only)."""
from __future__ import annotations

import numpy as np


def bf16(x: np.ndarray) -> np.ndarray:
    """float64 numbers to the nearest bfloat16, ties to even, as float64 (of normal size)."""
    with np.errstate(invalid="ignore", over="ignore"):
        m, e = np.frexp(x)
        return np.ldexp(np.round(m * 256) / 256, e)


def nibbles(q: np.ndarray) -> np.ndarray:
    """uint8 [n][k / 2] to whole numbers [n][k]."""
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1).astype(np.int64)


def weights(q: np.ndarray, scale: np.ndarray, zero=None) -> np.ndarray:
    """The bf16 number that each weight is nearest to."""
    n = nibbles(q)
    group = n.shape[1] // scale.shape[1]
    z = np.full(scale.shape, 8) if zero is None else zero.astype(np.int64)
    return bf16((n - np.repeat(z, group, 1)) * np.repeat(scale, group, 1))


def apply(x: np.ndarray, w: np.ndarray, gated: bool, add=None):
    """The result, and a bound for what fp32 sums may be off (before the result's own rounding).

    A sum of K products has at most K roundings, each of at most 2^-23 of the sum of magnitudes (twice fp32's half
    step: tensor cores may cut off where they align)."""
    y, size = x @ w.T, np.abs(x) @ np.abs(w).T
    off = x.shape[1] * 2.0 ** -23 * size
    if gated:
        h = w.shape[0] // 2
        g, u, dg, du = y[:, :h], y[:, h:], off[:, :h], off[:, h:]
        s = 1 / (1 + np.exp(-g))
        y = g * s * u
        # |silu'| <= 1.1; the functions and products themselves: 16 half steps
        off = 1.1 * dg * (np.abs(u) + du) + np.abs(g * s) * du + 16 * 2.0 ** -24 * np.abs(y)
    if add is not None:
        y = y + add
        off = off + 2.0 ** -24 * (np.abs(y) + off)
    return y, off
