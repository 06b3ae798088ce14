"""Attention with modified scores in float64 (test oracle).

TEST INFRASTRUCTURE ONLY.  For a query at position p of its sequence, query
head h, key position j of the same sequence:
    s_j = scale * <q, K_j>
    s_j <- cap * tanh(s_j / cap)            with a cap > 0
    s_j <- s_j - slope_h * |p - j|          with slopes
visible: j < prefix, or max(0, p + 1 - window) <= j <= p (window <= 0: none).
    out = sum_j softmax(s)_j V_j over the visible keys, zeros when there are none.

With every output comes a bound on how far fp32 arithmetic may be from it,
counted from the roundings:
    weights   u_p each (half a step of the type they are rounded to, 0 for fp32)
    scores    an error of e in s_j is a relative error of e in its weight:
              the dot product (D + 2 roundings of 2^-24 of sum |q||k| scale;
              `dot_rounds` of them where a test's products and sums are exact),
              the cap (`cap_error` of the value, see CAP_ERROR), the bias and the exponent's
              argument (4 roundings of 2^-24 of the largest |s|), 2^-22 of the
              exponential
    sums      one rounding of 2^-24 per key in the numerator and denominator
so |out - exact| <= 2 (u_p + e + n 2^-24) sum_j softmax_j |V_j|, and the last
rounding adds half a step of the output.
"""
from __future__ import annotations

import numpy as np

# How far a capped score may be off, relative to itself.  fp32 caches: the
# argument and the factor behind (4 roundings of 2^-24) and tanh itself, 2 ulp
# of at most 2^-23.  16-bit caches: the same roundings and tanh to 1e-6; by
# tcgen05 a polynomial off by 7.2e-6.
CAP_ERROR = {"f32": 8 * 2.0 ** -24, "16-bit": 1e-6 + 4 * 2.0 ** -24, "tcgen05": 7.2e-6 + 4 * 2.0 ** -24}


def visible_keys(p: int, klen: int, window: int = 0, prefix: int = 0) -> np.ndarray:
    j = np.arange(klen)
    first = max(0, p + 1 - window) if window > 0 else 0
    return ((j >= first) & (j <= p)) | (j < prefix)


def attend(q, K, V, p: int, scale: float, cap: float = 0.0, slope: float = 0.0, window: int = 0, prefix: int = 0,
           u_p: float = 0.0, eps: float = 2.0 ** -23, tiny: float = 0.0, cap_error: float = CAP_ERROR["tcgen05"],
           dot_rounds: int | None = None):
    """(output [D], bound [D]) of one query over its sequence's keys K [klen, D]."""
    seen = visible_keys(p, K.shape[0], window, prefix)
    j = np.nonzero(seen)[0]
    if j.size == 0:
        z = np.zeros(V.shape[-1])
        return z, z
    k, v = K[j].astype(np.float64), V[j].astype(np.float64)
    s = scale * (k @ q)
    dot = abs(scale) * (np.abs(k) @ np.abs(q)) * 2.0 ** -24
    dot *= q.shape[0] + 2 if dot_rounds is None else dot_rounds
    if cap > 0:
        s = cap * np.tanh(s / cap)
        dot = dot + np.abs(s) * cap_error
    s = s - slope * np.abs(p - j)
    w = np.exp(s - s.max())
    w = w / w.sum()
    out = w @ v
    # a key far below the maximum has a large score but no weight: errors count by weight
    e = dot + (np.abs(s) + abs(s.max()) + abs(slope) * np.abs(p - j)) * 4 * 2.0 ** -24 + 2.0 ** -22
    mass = np.minimum(1.0, u_p + e + j.size * 2.0 ** -24) * w
    near = mass @ np.abs(v) + mass.sum() * (w @ np.abs(v))
    return out, near + (np.abs(out) + near) * eps / 2 + tiny / 2
