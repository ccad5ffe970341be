"""Float64 CPU oracle of the RMS norm with the residual's addition, its
backward pass, and the 8-bit block form.

TEST INFRASTRUCTURE ONLY (see the package docstring).

  r = x + residual (rounded to the layer's type by ``round_r``)
  rstd = 1 / sqrt(mean(r^2) + eps),  y = r * rstd * weight

Block form: for 32 consecutive elements of a row, S is the smallest power of
two (at least 2^-127) with max|v| <= 448 S, and the elements are v / S rounded
to the nearest e4m3 number: 3 fraction bits, smallest normal exponent -6,
ties to even.
"""
from __future__ import annotations

import numpy as np

__all__ = ["rmsnorm_fwd", "rmsnorm_bwd", "mx8_quantize", "mx8_round"]


def rmsnorm_fwd(x, weight, eps, residual=None, round_r=lambda v: v):
    """(r, rstd, y) in float64; r is x without a residual."""
    x = np.asarray(x, dtype=np.float64)
    r = x if residual is None else round_r(x + np.asarray(residual, dtype=np.float64))
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1) + eps)
    return r, rstd, r * rstd[:, None] * np.asarray(weight, dtype=np.float64)


def rmsnorm_bwd(dy, r, weight, rstd, dres=None):
    """(dx, dw) for the given rstd."""
    dy, r, w = (np.asarray(v, dtype=np.float64) for v in (dy, r, weight))
    rs = np.asarray(rstd, dtype=np.float64)[:, None]
    n = r * rs
    g = dy * w
    dx = rs * (g - n * np.mean(g * n, axis=1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, dtype=np.float64)
    return dx, np.sum(dy * n, axis=0)


def mx8_round(v):
    """The nearest e4m3 number of |v| <= 448 (ties to even)."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))  # |v| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, e - 1 - 3)
    return np.round(v / step) * step


def mx8_quantize(v):
    """(q values, S) of finite rows [n, m], m a multiple of 32."""
    v = np.asarray(v, dtype=np.float64)
    b = v.reshape(v.shape[0], -1, 32)
    top = np.max(np.abs(b), axis=2)
    S = np.full(top.shape, 2.0 ** -127)
    pos = top > 0
    m, e = np.frexp(top[pos] / 448.0)  # top / 448 = m 2^e, m in [0.5, 1): S = 2^e, or 2^(e-1) at m = 0.5
    S[pos] = np.maximum(np.ldexp(1.0, np.where(m == 0.5, e - 1, e)), 2.0 ** -127)
    # the division by 448 rounds in float64; settle borders by exact products
    low = pos & (448.0 * (S / 2) >= top) & (S > 2.0 ** -127)
    S[low] /= 2
    S[pos & (448.0 * S < top)] *= 2
    return mx8_round(b / S[:, :, None]).reshape(v.shape), S
