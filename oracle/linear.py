"""Float64 CPU oracle of the layer norm and of the dense product with bias,
activation and residual, with their gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring).

  r = x + residual (rounded by ``round_r``), n = (r - mean) rstd,  y = n weight + bias
  z = x w^T + bias,  y = act(z) + residual
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["layernorm_fwd", "layernorm_bwd", "act", "act_slope", "linear_fwd", "linear_dgrad", "linear_wgrad", "ACTS"]

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")  # in the order of MOE_ACT_*

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def layernorm_fwd(x, weight, bias, eps, residual=None, round_r=lambda v: v):
    """(r, mean, rstd, n, y); bias may be None."""
    x = np.asarray(x, np.float64)
    r = x if residual is None else round_r(x + np.asarray(residual, np.float64))
    mean = np.mean(r, axis=1)
    c = r - mean[:, None]
    rstd = 1.0 / np.sqrt(np.mean(c * c, axis=1) + eps)
    n = c * rstd[:, None]
    y = n * np.asarray(weight, np.float64)
    return r, mean, rstd, n, y if bias is None else y + np.asarray(bias, np.float64)


def layernorm_bwd(dy, r, weight, mean, rstd, dres=None):
    """(dx, dw, db) for the given mean and rstd."""
    dy, r, w = (np.asarray(v, np.float64) for v in (dy, r, weight))
    rs = np.asarray(rstd, np.float64)[:, None]
    n = (r - np.asarray(mean, np.float64)[:, None]) * rs
    g = dy * w
    dx = rs * (g - np.mean(g, axis=1, keepdims=True) - n * np.mean(g * n, axis=1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, np.sum(dy * n, axis=0), np.sum(dy, axis=0)


def _phi(z):
    return 0.5 * _erfc(-z / math.sqrt(2.0))


def act(name, z):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "gelu":
        return z * _phi(z) if z.size else z
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * 0.5 * (1 + np.tanh(0.5 * z))
    return z


def act_slope(name, z):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return _phi(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 0.5 * (1 + np.tanh(0.5 * z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def linear_fwd(x, w, bias=None, residual=None, activation="none"):
    """(z, y)."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = act(activation, z)
    return z, y if residual is None else y + np.asarray(residual, np.float64)


def linear_dgrad(dz, w, z_in=None, act_in="none", add=None):
    """dx: the gradient of x, times the slope of the activation that made x."""
    dx = np.asarray(dz, np.float64) @ np.asarray(w, np.float64)
    if act_in != "none":
        dx = dx * act_slope(act_in, z_in)
    return dx if add is None else dx + np.asarray(add, np.float64)


def linear_wgrad(dz, x):
    """(dw, db)."""
    dz = np.asarray(dz, np.float64)
    return dz.T @ np.asarray(x, np.float64), np.sum(dz, axis=0)
