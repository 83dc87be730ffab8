"""Matrices in 8-bit integers with one scale a row, in float64, from the definition.

A row x has the scale s = max|x| / 127 rounded to float32, and an element becomes the whole number
nearest x / s, ties to the even one, at most 127 either way.  A row of zeros has scale 0 and codes 0, a
row with an infinity or a NaN a NaN scale and codes 0.
"""
from __future__ import annotations

import numpy as np

from .fp4_oracle import to_f64


def quantise(x):
    """x [rows, cols] -> (codes int8 [rows, cols], scales float32 [rows])."""
    x = to_f64(x)
    with np.errstate(all="ignore"):
        top = np.abs(x).max(1)
        s = (top / 127.0).astype(np.float32)
        bad = ~np.isfinite(x).all(1)
        live = (s > 0) & ~bad
        q = np.where(live[:, None], x / np.where(live, s, 1).astype(np.float64)[:, None], 0.0)
    # float64 tells x / s from the border of two codes: x and s have at most 24 bits each, so a quotient
    # that is no border is at least 2^-26 of itself away from one
    c = np.clip(np.rint(q), -127, 127).astype(np.int8)
    return c, np.where(bad, np.float32("nan"), s).astype(np.float32)


def values(codes, scales) -> np.ndarray:
    return codes.astype(np.float64) * scales.astype(np.float64)[:, None]


def fake(x) -> np.ndarray:
    """What the stored form of x stands for."""
    return values(*quantise(x))


def rmsnorm(h, weight, eps) -> np.ndarray:
    """float64 rows h / sqrt(mean h^2 + eps) * weight."""
    h = to_f64(h)
    with np.errstate(all="ignore"):
        return h / np.sqrt((h * h).mean(1, keepdims=True) + np.float64(np.float32(eps))) * to_f64(weight)


def sums(cx, cw) -> np.ndarray:
    """int64 sums of code products."""
    return cx.astype(np.int64) @ cw.astype(np.int64).T
