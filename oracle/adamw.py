"""AdamW, as the fp32 operation sequence the library promises, and in fp64.

TEST INFRASTRUCTURE ONLY (see the package header).

numpy's float32 add, multiply, divide and square root each round once, so
step() is the promised sequence itself and the GPU has to match it bit for bit:
    g' = g * scale
    m = m b1 + g' (1 - b1),   v = v b2 + (g' g') (1 - b2),   r = sqrt(v)
    w = w (1 - lr wd) - (m / (r rbc2 + eps)) (lr / (1 - b1^t)),  rbc2 = 1/sqrt(1 - b2^t)
with the factors formed in fp64 and rounded to fp32.  8-bit states hold m and r
as e4m3 codes, one scale per 128 elements: the smallest power of two (at least
2^-100; 1 for a tile of zeros) with amax <= 448 scale over the tile's finite
values; a non-finite value gets the NaN code.

Pins (tests/test_oracle_training.py): step() against exact() (fp64, from the
formulas in their textbook form), a first step from zero states by hand, the
tile scale against a search over powers of two.
"""
from __future__ import annotations

import math

import numpy as np

from . import fp8

TILE = 128
f32 = np.float32


def tile_scale(amax) -> np.float32:
    """Smallest 2^j, j >= -100, with amax <= 448 * 2^j; 1 for amax = 0."""
    if amax == 0:
        return f32(1.0)
    j = -100
    while float(amax) > 448.0 * 2.0 ** j:
        j += 1
    return f32(2.0 ** j)


def encode(x):
    """fp32 [n] -> (codes uint8 [n], scales fp32 [ceil(n/128)])."""
    x = np.asarray(x, dtype=np.float32).reshape(-1)
    n = x.size
    tiles = -(-n // TILE)
    codes = np.zeros(n, dtype=np.uint8)
    scales = np.ones(tiles, dtype=np.float32)
    for i in range(tiles):
        t = x[i * TILE:(i + 1) * TILE]
        fin = np.isfinite(t)
        scales[i] = tile_scale(np.abs(t[fin]).max() if fin.any() else 0.0)
        q = fp8.to_e4m3((np.where(fin, t, 0) / scales[i]).astype(np.float32))
        codes[i * TILE:(i + 1) * TILE] = np.where(fin, q, 0x7F)
    return codes, scales


def decode(codes, scales):
    codes = np.asarray(codes, dtype=np.uint8)
    val = np.where((codes & 0x7F) == 0x7F, f32("nan"), fp8.from_e4m3(codes)).astype(np.float32)
    return (val * np.repeat(np.asarray(scales, dtype=np.float32), TILE)[:codes.size]).astype(np.float32)


def step(w, g, m, v, *, lr, b1, b2, eps, wd, t, scale=None):
    """One step in the promised fp32 sequence: (w, m, v, r)."""
    w, g, m, v = (np.asarray(a, dtype=np.float32) for a in (w, g, m, v))
    with np.errstate(all="ignore"):
        if scale is not None:
            g = g * f32(scale)
        m = m * f32(b1) + g * f32(1 - b1)
        v = v * f32(b2) + (g * g) * f32(1 - b2)
        r = np.sqrt(v)
        rbc2 = f32(1 / math.sqrt(1 - b2 ** t))
        w = w * f32(1 - lr * wd) - (m / (r * rbc2 + f32(eps))) * f32(lr / (1 - b1 ** t))
    return w, m, v, r


def exact(w, g, m, v, *, lr, b1, b2, eps, wd, t, scale=None):
    """One step in fp64, textbook form: (w, m, v)."""
    w, g, m, v = (np.asarray(a, dtype=np.float64) for a in (w, g, m, v))
    g = g * (1.0 if scale is None else float(scale))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    mh, vh = m / (1 - b1 ** t), v / (1 - b2 ** t)
    return w - lr * (mh / (np.sqrt(vh) + eps) + wd * w), m, v
