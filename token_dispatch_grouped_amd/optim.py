"""AdamW (``moe_adamw_step``) and Muon (``moe_muon_step``,
``moe_orthogonalize``) for expert and dense weights over the C ABI.

``ExpertAdamW``:

Keeps fp32 master weights and both moments for each expert weight tensor
(w_gu [E,2F,d] and w_down [E,d,F]); each ``step`` runs one fused pass per
tensor that updates master and moments, writes the bf16 working copy the
grouped GEMMs read (in place, in the layer's weight tensor) and zeroes the
fp32 gradient the backward accumulated into. PyTorch only allocates.

``ExpertMuon`` keeps fp32 masters and one momentum; each ``step`` replaces the
update of every matrix by an orthogonalised one. ``Orthogonalizer`` is that
part alone.
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence

import torch

from . import _lib as L
from .block import _TORCH, _check, _check_T, _device, _on


class ExpertAdamW:
    def __init__(self, weights: Sequence[torch.Tensor], lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01):
        """``weights``: the working tensors the layer reads. A bf16 weight
        gets an fp32 master that starts as its exact widening; an fp32
        weight is its own master (updated in place)."""
        self.weights: List[torch.Tensor] = list(weights)
        for w in self.weights:
            if not w.is_contiguous() or w.dtype not in (torch.bfloat16, torch.float32):
                raise ValueError("expert weights must be contiguous bf16 or fp32 tensors")
        self.master = [w.detach().float().clone() if w.dtype == torch.bfloat16 else w for w in self.weights]
        self.exp_avg = [torch.zeros_like(m) for m in self.master]
        self.exp_avg_sq = [torch.zeros_like(m) for m in self.master]
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.t = 0

    def step(self, grads: Sequence[torch.Tensor], grad_scale: float = 1.0, zero_grad: bool = True, stream=None):
        """One update from fp32 gradients (same shapes as the weights)."""
        self.t += 1
        cfg = L.make_adamw_config(self.lr, self.betas[0], self.betas[1], self.eps, self.weight_decay, grad_scale,
                                  self.t, zero_grad)
        for w, mst, g, m, v in zip(self.weights, self.master, grads, self.exp_avg, self.exp_avg_sq):
            if g.dtype != torch.float32 or g.shape != mst.shape or not g.is_contiguous():
                raise ValueError("gradients must be contiguous fp32 tensors shaped like the weights")
            L.moe_adamw_step(cfg, mst.numel(), mst, g, m, v, w if w.dtype == torch.bfloat16 else None, stream)


class Orthogonalizer:
    def __init__(self, batch_max: int, rows: int, cols: int, dtype: int = L.MOE_DTYPE_F32, steps: int = 5,
                 coef=L.ORTH_COEF, eps: float = 1e-7, device: str = "cuda"):
        """Newton-Schulz orthogonalisation of up to ``batch_max`` matrices
        [rows, cols] at a time, to bf16."""
        self.batch_max, self.rows, self.cols, self.dtype = batch_max, rows, cols, dtype
        self.steps, self.coef, self.eps = steps, tuple(coef), eps
        ws = L.moe_orthogonalize_workspace_size(self.shape(batch_max))
        self.device = dev = _device(device)
        self.ws = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
        self.o = torch.empty(batch_max, rows, cols, dtype=torch.bfloat16, device=dev)

    def shape(self, batch: int) -> L.moe_orth_shape:
        return L.make_orth_shape(batch, self.rows, self.cols, self.dtype, self.steps, self.coef, self.eps)

    def check_forward(self, batch: int, x, out=None) -> None:
        _check_T(batch, self.batch_max)
        _check("x", x, batch, (self.rows, self.cols), _TORCH[self.dtype], self.device)
        if out is not None:
            _check("out", out, batch, (self.rows, self.cols), torch.bfloat16, self.device)

    def forward(self, batch: int, x, out=None, stream=None):
        """The first ``batch`` matrices of x, into ``out`` (which may be a bf16
        x) or the object's buffer."""
        self.check_forward(batch, x, out)
        out = self.o if out is None else out
        with _on(self.device):
            L.moe_orthogonalize(self.shape(batch), x, out, self.ws, self.ws.numel(), stream)
        return out[:batch]


class ExpertMuon:
    def __init__(self, weights: Sequence[torch.Tensor], lr: float, momentum: float = 0.95, weight_decay: float = 0.0,
                 nesterov: bool = True, parts: Optional[Sequence[int]] = None, match_rms: Optional[float] = None,
                 steps: int = 5, coef=L.ORTH_COEF, eps: float = 1e-7):
        """``weights``: the working tensors the layers read, [rows, cols] or
        [E, rows, cols], each expert's matrix on its own. ``parts[i]``: how many
        matrices weight i stacks along its rows (2 for w_gu: gate and up),
        default 1. The update is scaled by sqrt(max(1, rows / cols)), or with
        ``match_rms`` by match_rms * sqrt(max(rows, cols)), which gives its
        elements about that root mean square (0.2: as AdamW's). Masters as in
        ``ExpertAdamW``."""
        self.weights: List[torch.Tensor] = list(weights)
        parts = [1] * len(self.weights) if parts is None else list(parts)
        if len(parts) != len(self.weights):
            raise ValueError("parts: one number for each weight")
        self.lr, self.momentum, self.weight_decay, self.nesterov = lr, momentum, weight_decay, nesterov
        self.shapes, self.scales, need = [], [], {}
        for w, p in zip(self.weights, parts):
            if not w.is_contiguous() or w.dtype not in (torch.bfloat16, torch.float32) or w.dim() not in (2, 3):
                raise ValueError("weights must be contiguous bf16 or fp32 tensors of 2 or 3 dimensions")
            if not w.shape[-2] or not w.shape[-1]:
                raise ValueError("weights must have rows and columns")
            if p < 1 or w.shape[-2] % p:
                raise ValueError(f"a weight of {w.shape[-2]} rows does not stack {p} matrices")
            rows, cols = w.shape[-2] // p, w.shape[-1]
            s = L.make_orth_shape(w.numel() // (rows * cols), rows, cols, L.MOE_DTYPE_F32, steps, coef, eps)
            self.shapes.append(s)
            self.scales.append(math.sqrt(max(1.0, rows / cols)) if match_rms is None else
                               match_rms * math.sqrt(max(rows, cols)))
            need[w.device] = max(need.get(w.device, 256), L.moe_orthogonalize_workspace_size(s))
        self.master = [w.detach().float().clone() if w.dtype == torch.bfloat16 else w for w in self.weights]
        self.momenta = [torch.zeros_like(m) for m in self.master]
        self.ws = {d: torch.empty(n, dtype=torch.uint8, device=d) for d, n in need.items()}

    def step(self, grads: Sequence[torch.Tensor], grad_scale: float = 1.0, zero_grad: bool = True, stream=None):
        """One update from fp32 gradients (same shapes as the weights)."""
        grads = list(grads)
        if len(grads) != len(self.weights):
            raise ValueError("one gradient for each weight")
        for g, m in zip(grads, self.master):
            if g.dtype != torch.float32 or g.shape != m.shape or not g.is_contiguous() or g.device != m.device:
                raise ValueError("gradients must be contiguous fp32 tensors shaped like the weights, on their device")
        for w, mst, g, m, s, scale in zip(self.weights, self.master, grads, self.momenta, self.shapes, self.scales):
            cfg = L.make_muon_config(self.lr, self.momentum, self.weight_decay, scale, grad_scale, self.nesterov, zero_grad)
            ws = self.ws[mst.device]
            with _on(mst.device):
                L.moe_muon_step(cfg, s, mst, g, m, w if w.dtype == torch.bfloat16 else None, ws, ws.numel(), stream)
