"""Float64 CPU oracle of the Newton-Schulz orthogonalisation and of the Muon
step around it.

TEST INFRASTRUCTURE ONLY (see the package docstring).

  X = U / (|U| + eps);  X = a X + (b A + c A A) X with A = X X^T, `steps` times
  momentum = mu momentum + G;  U = G + mu momentum (Nesterov) or momentum
  param = param (1 - lr wd) - lr scale X

(Jordan et al., "Muon: an optimizer for hidden layers in neural networks", with
its coefficients.) ``orthogonalize_halves`` is the same iteration with its
tensors held as the kernels hold them where the short side is long, fp16 times
2^12 with X in two halves (in the last step the high one) and the diagonals of A
and b A + c A A apart, and sums without rounding: what that choice of types
alone costs on a given matrix. ``orthogonalize_both_halves``: where it is short,
every tensor in two halves in every place. ``orthogonalize_f32``: everything in
fp32, sums and all.
"""
from __future__ import annotations

import numpy as np

__all__ = ["ORTH_COEF", "orthogonalize", "orthogonalize_halves", "orthogonalize_both_halves", "orthogonalize_f32", "muon_step"]

ORTH_COEF = (3.4445, -4.7750, 2.0315)
_SCALE = 4096.0


def orthogonalize(u, steps=5, coef=ORTH_COEF, eps=1e-7):
    """One matrix [rows, cols]."""
    a, b, c = coef
    x = np.asarray(u, np.float64)
    x = x / (np.sqrt(np.sum(x * x)) + eps)
    for _ in range(steps):
        if x.shape[0] <= x.shape[1]:
            A = x @ x.T
            x = a * x + (b * A + c * (A @ A)) @ x
        else:
            A = x.T @ x
            x = a * x + x @ (b * A + c * (A @ A))
    return x


def _half(v):
    return (v * _SCALE).astype(np.float16).astype(np.float64) / _SCALE


def orthogonalize_halves(u, steps=5, coef=ORTH_COEF, eps=1e-7):
    a, b, c = coef
    x = np.asarray(u, np.float64)
    if x.shape[0] > x.shape[1]:
        return orthogonalize_halves(x.T, steps, coef, eps).T
    x = x / (np.sqrt(np.sum(x * x)) + eps)
    for k in range(steps):
        hi = _half(x)
        lo = _half(x - hi) if k + 1 < steps else 0.0
        A = hi @ hi.T
        d = np.diag(A).copy()
        np.fill_diagonal(A, 0.0)
        A = _half(A)
        AA = A @ A + (d[:, None] + d[None, :]) * A
        B = b * A + c * AA
        db = np.diag(B) + b * d + c * d * d
        np.fill_diagonal(B, 0.0)
        x = (a + db)[:, None] * (hi + lo) + _half(B) @ hi
    return x


def orthogonalize_both_halves(u, steps=5, coef=ORTH_COEF, eps=1e-7):
    a, b, c = coef
    x = np.asarray(u, np.float64)
    if x.shape[0] > x.shape[1]:
        return orthogonalize_both_halves(x.T, steps, coef, eps).T

    def two(v):
        hi = _half(v)
        return hi + _half(v - hi)

    x = x / (np.sqrt(np.sum(x * x)) + eps)
    for _ in range(steps):
        x = two(x)
        A = x @ x.T
        d = np.diag(A).copy()
        np.fill_diagonal(A, 0.0)
        A = two(A)
        AA = A @ A + (d[:, None] + d[None, :]) * A
        B = b * A + c * AA
        db = np.diag(B) + b * d + c * d * d
        np.fill_diagonal(B, 0.0)
        x = (a + db)[:, None] * x + two(B) @ x
    return x


def orthogonalize_f32(u, steps=5, coef=ORTH_COEF, eps=1e-7):
    a, b, c = (np.float32(v) for v in coef)
    x = np.asarray(u, np.float64)
    if x.shape[0] > x.shape[1]:
        return orthogonalize_f32(x.T, steps, coef, eps).T
    x = (x / (np.sqrt(np.sum(x * x)) + eps)).astype(np.float32)
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.astype(np.float64)


def muon_step(param, grad, momentum, lr, mu=0.95, weight_decay=0.0, scale=1.0, grad_scale=1.0, nesterov=True,
              orth=orthogonalize, **kw):
    """(param, momentum, o) after one step on one matrix."""
    p, g, m = (np.asarray(v, np.float64) for v in (param, grad, momentum))
    g = grad_scale * g
    m = mu * m + g
    o = orth(g + mu * m if nesterov else m, **kw)
    return p * (1 - lr * weight_decay) - lr * scale * o, m, o
