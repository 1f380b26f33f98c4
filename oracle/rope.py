"""Rotary position embedding, oracle side (test infrastructure; shares no code
with the CUDA-side library).

The pages leave the models' position embedding to the model. Reading taken: the
first R elements of a query or key row at position p turn in pairs (a, b) by the
angles of the position's table row,
    a' = a cos - b sin,  b' = b cos + a sin,
pairs (x[i], x[i + R/2]), or (x[2i], x[2i + 1]) when interleaved; every product,
sum and difference is one float32 operation rounded to nearest.
"""

import math

import numpy as np


def table(num_positions, rotary_dim, theta):
    """cos_i(p), i < R/2, then sin_i(p), of the angles p theta^(-2i/R)."""
    half = rotary_dim // 2
    out = np.empty((num_positions, rotary_dim), np.float32)
    for p in range(num_positions):
        for i in range(half):
            a = p * theta ** (-2.0 * i / rotary_dim)
            out[p, i], out[p, half + i] = math.cos(a), math.sin(a)
    return out


def rotate(x, cos_sin, positions, interleaved):
    """x float32 [T, H, d] -> float32 [T, H, d]."""
    x = np.asarray(x, np.float32)
    half = cos_sin.shape[1] // 2
    out = x.copy()
    for t, p in enumerate(positions):
        for i in range(half):
            lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = cos_sin[p, i], cos_sin[p, half + i]
            a, b = x[t, :, lo], x[t, :, hi]
            out[t, :, lo] = a * c - b * s
            out[t, :, hi] = b * c + a * s
    return out
