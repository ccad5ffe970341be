"""Float64 CPU oracle of the dense gated feed-forward block and its gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring).

  h = x W_gu^T, a = silu(h_gate) * h_up, y = a W_down^T + add
"""
from __future__ import annotations

import numpy as np

__all__ = ["dense_ffn_fwd", "dense_ffn_dgrad", "dense_ffn_wgrad"]


def _sig(z):
    return 0.5 * (1.0 + np.tanh(0.5 * z))


def dense_ffn_fwd(x, w_gu, w_down, add=None, round_a=lambda v: v):
    """(h, a, y); round_a: how a is held between the two products."""
    h = np.asarray(x, np.float64) @ np.asarray(w_gu, np.float64).T
    F = h.shape[1] // 2
    a = h[:, :F] * _sig(h[:, :F]) * h[:, F:]
    y = round_a(a) @ np.asarray(w_down, np.float64).T
    return h, a, y if add is None else y + np.asarray(add, np.float64)


def dense_ffn_dgrad(dy, h, w_gu, w_down, add=None):
    """(da, dh, dx)."""
    h = np.asarray(h, np.float64)
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    da = np.asarray(dy, np.float64) @ np.asarray(w_down, np.float64)
    s = _sig(g)
    dh = np.concatenate([da * u * s * (1.0 + g * (1.0 - s)), da * g * s], axis=1)
    dx = dh @ np.asarray(w_gu, np.float64)
    return da, dh, dx if add is None else dx + np.asarray(add, np.float64)


def dense_ffn_wgrad(dy, x, a, dh):
    """(dw_gu, dw_down)."""
    dy, x, a, dh = (np.asarray(v, np.float64) for v in (dy, x, a, dh))
    return dh.T @ x, dy.T @ a
