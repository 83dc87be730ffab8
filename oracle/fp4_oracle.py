"""Microscaled 4-bit matrices in float64, from the definition of the format.

A block of 32 consecutive elements of a row shares the scale 2^e with
e = max(floor(log2 max|x|) - 2, -127); an element becomes the nearest of
+-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times the scale, of two equally near the one with the even index.
A block with an infinity or a NaN has the NaN scale and zero codes.
"""
from __future__ import annotations

import numpy as np

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([MAGS, -MAGS])  # by code


def to_f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy() if hasattr(t, "detach") else np.asarray(t, np.float64)


def quantise(x):
    """x [rows, cols] -> (codes uint8 [rows, 32 * blocks], scale bytes uint8 [rows, blocks])."""
    x = to_f64(x)
    rows, cols = x.shape
    nb = (cols + 31) // 32
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    _, ex = np.frexp(top)  # top = m 2^ex, m in [0.5, 1)
    e = np.where(top > 0, np.maximum(ex - 1 - 2, -127), -127)
    ratio = np.abs(b) / np.exp2(e.astype(np.float64))[..., None]
    d = np.abs(np.minimum(ratio, 6.0)[..., None] - MAGS)  # distance to every magnitude
    best = d.min(-1, keepdims=True)
    tied = d == best
    idx = np.argmax(tied, -1)  # the lower of two
    two = tied.sum(-1) == 2
    idx = np.where(two & (idx % 2 == 1), idx + 1, idx)
    codes = (idx + 8 * np.signbit(b)).astype(np.uint8)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes.reshape(rows, -1), scales


def values(codes, scales, cols) -> np.ndarray:
    """float64 values of codes and scale bytes."""
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    v = VALUES[codes].reshape(codes.shape[0], -1, 32) * s[..., None]
    return v.reshape(codes.shape[0], -1)[:, :cols]


def fake(x) -> np.ndarray:
    """What the stored form of x stands for."""
    c, s = quantise(x)
    return values(c, s, np.shape(x)[1])


def pack_codes(codes) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).reshape(-1)


def scale_offset(r, b, cols):
    """Byte offset of row r, block b in the tiled scale buffer."""
    kt = 2 * ((cols + 255) // 256)
    return ((r // 128) * kt + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def pack_scales(scales, cols) -> np.ndarray:
    rows, nb = scales.shape
    out = np.zeros((rows + 127) // 128 * 2 * ((cols + 255) // 256) * 512, np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[scale_offset(r, b, cols)] = scales
    return out
