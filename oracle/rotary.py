"""Rotary positions in float64 (test oracle).

TEST INFRASTRUCTURE ONLY.  Pair i of a head at position p turns by the angle
p * inv_freq[i]; the pair is the elements (i, i + R/2) (half layout) or
(2i, 2i + 1) (interleaved) of the head's first R dims, the other dims are
copied.  The angle is reduced modulo one turn in exact rational arithmetic, so
positions of any size keep full accuracy.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

# pi to 60 digits, as a fraction: 1 / 2 pi of a double times a 64-bit position
# needs about 40 of them
_TWO_PI = 2 * Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


def angle(position: int, inv_freq: float) -> float:
    """position * inv_freq modulo 2 pi, in [0, 2 pi)."""
    turns = Fraction(int(position)) * Fraction(float(inv_freq)) / _TWO_PI
    turns -= math.floor(turns)
    return float(turns * _TWO_PI)


def pairs(i: int, rotary_dim: int, interleaved: bool):
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)


def rotate(x: np.ndarray, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0) -> np.ndarray:
    """x [T, H, D] float64 -> rotated copy."""
    y = np.array(x, dtype=np.float64)
    R = 2 * len(inv_freq)
    for t, p in enumerate(positions):
        for i, f in enumerate(inv_freq):
            a = angle(p, f)
            c, s = mscale * math.cos(a), mscale * math.sin(a)
            i1, i2 = pairs(i, R, interleaved)
            y[t, :, i1] = x[t, :, i1] * c - x[t, :, i2] * s
            y[t, :, i2] = x[t, :, i2] * c + x[t, :, i1] * s
    return y


def error_bound(x: np.ndarray, y: np.ndarray, rotary_dim: int, interleaved: bool, mscale: float,
                eps: float, tiny: float) -> np.ndarray:
    """How far fp32 arithmetic rounded once to a type of machine epsilon `eps`
    may be from y = rotate(x).  cos and sin: 2 ulp below 1 (2^-23), the
    reduced angle (2^-24 of an eighth of a turn), a step off by 2^-65 turns
    times a position of up to 2^40 (1.9e-7 rad) and the product with mscale
    (2^-24) make under 2^-21 in all, times |x1| + |x2|; two products and a sum
    add 3 * 2^-24.  The last rounding is eps / 2 of the value or half the
    smallest subnormal."""
    R = rotary_dim
    mag = np.zeros_like(y)
    for i in range(R // 2):
        i1, i2 = pairs(i, R, interleaved)
        m = np.abs(x[..., i1]) + np.abs(x[..., i2])
        mag[..., i1] = m
        mag[..., i2] = m
    near = mag * abs(mscale) * (2.0 ** -21 + 3 * 2.0 ** -24)
    out = near + (np.abs(y) + near) * eps / 2 + tiny / 2
    copied = np.ones(y.shape[-1], dtype=bool)
    copied[:R] = False
    out[..., copied] = 0.0
    return out
