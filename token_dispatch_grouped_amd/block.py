"""What stands in front of and beside the expert layer, over the C ABI:
``RmsNorm`` (``moe_rmsnorm_*``), ``LayerNorm`` (``moe_layernorm_*``),
``GatedFfn`` (``moe_ffn_*``), ``Linear`` (``moe_linear_*``) and the 8-bit block
form of a matrix (``moe_mx8_quantize``).

As in ``layer.py``, PyTorch only allocates and provides the stream; buffers
and workspaces are made once for the largest microbatch (``T_max``) and serve
any smaller one, the empty one included. Weight gradients are fp32 and
accumulate unless ``overwrite`` is asked for. Tensors are checked (type, shape,
contiguity, device) before anything is called: each call's check is a method of
its own (``check_*``), which ``MoeLayer`` makes before its first launch.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional, Tuple

import torch

from . import _lib as L

_TORCH = {L.MOE_DTYPE_BF16: torch.bfloat16, L.MOE_DTYPE_F32: torch.float32}


@dataclasses.dataclass
class Mx8:
    """A matrix in the 8-bit block form: values q * scale, one scale for 32
    consecutive elements of a row."""
    q: torch.Tensor      # [rows, cols] float8_e4m3fn
    scale: torch.Tensor  # [rows, cols / 32] float8_e8m0fnu

    def rows(self, n: int) -> "Mx8":
        return Mx8(self.q[:n], self.scale[:n])

    def values(self) -> torch.Tensor:
        """The values in fp32 (for inspection: plain torch)."""
        s = self.scale.float().repeat_interleave(32, dim=1)
        return self.q.float() * s


def _check(name: str, t, rows: Optional[int], tail: Tuple[int, ...], dtype, device) -> None:
    """``rows``: at least that many in front of ``tail``; None: exactly ``tail``."""
    ok = isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.is_contiguous()
    if ok:
        s = tuple(t.shape)
        ok = s == tail if rows is None else len(s) == 1 + len(tail) and s[0] >= rows and s[1:] == tail
    if not ok:
        want = f"{'' if rows is None else f'at least {rows} rows of '}{tail}"
        got = f"{tuple(t.shape)} {t.dtype} on {t.device}" if isinstance(t, torch.Tensor) else repr(type(t))
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of {want} on {device}, got {got}")


def _check_mx8(name: str, m, rows: Optional[int], shape: Tuple[int, ...], device) -> None:
    if not isinstance(m, Mx8):
        raise ValueError(f"{name}: expected Mx8, got {type(m)!r}")
    tail = shape[:-1] + (shape[-1] // 32,)
    _check(name + ".q", m.q, rows, shape, torch.float8_e4m3fn, device)
    _check(name + ".scale", m.scale, rows, tail, torch.float8_e8m0fnu, device)


def _check_apart(name: str, t: torch.Tensor, T: int, written: torch.Tensor, what: str) -> None:
    """The first T rows of two contiguous tensors share no memory."""
    def span(v):
        return v.data_ptr(), v.data_ptr() + T * v.stride(0) * v.element_size()
    (a, a_end), (b, b_end) = span(t), span(written)
    if a < b_end and b < a_end:
        raise ValueError(f"{name} lies in {what}, which is written before the last read of {name}: give a copy")


def _device(device) -> torch.device:
    d = torch.device(device)
    return torch.device("cuda", torch.cuda.current_device()) if d.type == "cuda" and d.index is None else d


def _on(device: torch.device):
    """The device as the current one for a call, if it is not already."""
    if torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _made_on(device: torch.device, stream):
    """Memory made for a call on another stream than the current one belongs to
    that stream: the current one may still be writing what was freed there."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device))


def _check_T(T: int, T_max: int) -> None:
    if not 0 <= T <= T_max:
        raise ValueError(f"T = {T} outside [0, T_max = {T_max}]")


def empty_mx8(rows: int, cols: int, device="cuda") -> Mx8:
    if cols % 32:
        raise ValueError("the block form needs whole blocks of 32 columns")
    return Mx8(torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=device),
               torch.empty(rows, cols // 32, dtype=torch.float8_e8m0fnu, device=device))


def quantize_mx8(t: torch.Tensor, out: Optional[Mx8] = None, stream=None) -> Mx8:
    """The 8-bit block form of a bf16 or fp32 matrix [rows, cols], cols a
    multiple of 64 (a weight on loading, or rows that no norm made)."""
    types = {v: k for k, v in _TORCH.items()}
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in types or not t.is_contiguous():
        raise ValueError("quantize_mx8: expected a contiguous bf16 or fp32 matrix")
    rows, cols = t.shape
    if out is None:
        with _made_on(t.device, stream):
            out = empty_mx8(rows, cols, t.device)
    _check_mx8("out", out, None, (rows, cols), t.device)
    with _on(t.device):
        L.moe_mx8_quantize(rows, cols, types[t.dtype], t, out.q, out.scale, stream)
    return out


@dataclasses.dataclass
class NormOut:
    """Views of a norm's outputs for one microbatch."""
    r: Optional[torch.Tensor]  # the new residual stream; None without a residual (it is x)
    y: object                  # [T, d] tensor, or Mx8
    rstd: torch.Tensor


class RmsNorm:
    def __init__(self, T_max: int, d: int, dtype: int = L.MOE_DTYPE_BF16, eps: float = 1e-6, mx8: bool = False,
                 device: str = "cuda"):
        """``mx8``: y in the 8-bit block form (for ``GatedFfn`` in MX8)."""
        self.T_max, self.d, self.dtype, self.eps, self.mx8 = T_max, d, dtype, eps, mx8
        self.ws_bytes = L.moe_rmsnorm_workspace_size(self.shape(T_max))
        self.device = dev = _device(device)
        self.td = _TORCH[dtype]
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)
        self.r = torch.empty(T_max, d, dtype=self.td, device=dev)
        self.y = empty_mx8(T_max, d, dev) if mx8 else torch.empty(T_max, d, dtype=self.td, device=dev)
        self.rstd = torch.empty(T_max, dtype=torch.float32, device=dev)
        self.dx = None  # made by the first backward: serving needs none

    def shape(self, T: int, overwrite: bool = False) -> L.moe_norm_shape:
        return L.make_norm_shape(T, self.d, self.dtype, self.eps, L.MOE_NORM_OVERWRITE_DW if overwrite else 0)

    def check_forward(self, T: int, x, weight, residual=None) -> None:
        _check_T(T, self.T_max)
        _check("x", x, T, (self.d,), self.td, self.device)
        _check("weight", weight, None, (self.d,), self.td, self.device)
        if residual is not None:
            _check("residual", residual, T, (self.d,), self.td, self.device)

    def forward(self, T: int, x, weight, residual=None, stream=None) -> NormOut:
        """y = norm(x + residual) * weight; r = x + residual is the new
        residual stream (in the object's buffer, valid until the next
        forward)."""
        self.check_forward(T, x, weight, residual)
        return self._forward(T, x, weight, residual, stream)

    def _forward(self, T: int, x, weight, residual, stream) -> NormOut:
        r = self.r if residual is not None else None
        with _on(self.device):
            L.moe_rmsnorm_fwd(self.shape(T), x, residual, weight, r, self.y.q if self.mx8 else self.y,
                              self.y.scale if self.mx8 else None, self.rstd, stream)
        return NormOut(None if r is None else r[:T], self.y.rows(T) if self.mx8 else self.y[:T], self.rstd[:T])

    def check_backward(self, T: int, dy, r, weight, dw, dres=None, out=None) -> None:
        _check_T(T, self.T_max)
        for name, t in (("dy", dy), ("r", r)) + ((("dres", dres),) if dres is not None else ()):
            _check(name, t, T, (self.d,), self.td, self.device)
        _check("weight", weight, None, (self.d,), self.td, self.device)
        _check("dw", dw, None, (self.d,), torch.float32, self.device)
        if out is not None:
            _check("out", out, T, (self.d,), self.td, self.device)

    def backward(self, T: int, dy, r, weight, dw, dres=None, overwrite: bool = False, out=None, stream=None):
        """Gradient of x (and of the residual alike) from dL/dy, with the
        ``rstd`` of the last forward; ``r``: that forward's r, or its x if it
        had no residual; ``dres``: the gradient that reaches r directly.
        ``dw`` [d] fp32 accumulates (``overwrite``: is written)."""
        self.check_backward(T, dy, r, weight, dw, dres, out)
        return self._backward(T, dy, r, weight, dw, dres, overwrite, out, stream)

    def _backward(self, T: int, dy, r, weight, dw, dres, overwrite, out, stream):
        if out is None:
            if self.dx is None:
                with _made_on(self.device, stream):
                    self.dx = torch.empty(self.T_max, self.d, dtype=self.td, device=self.device)
            out = self.dx
        with _on(self.device):
            L.moe_rmsnorm_bwd(self.shape(T, overwrite), dy, r, weight, self.rstd, dres, out, dw, self.ws,
                              self.ws.numel(), stream)
        return out[:T]


class GatedFfn:
    def __init__(self, T_max: int, d: int, F: int, dtype: int = L.MOE_DTYPE_BF16, save: bool = True,
                 device: str = "cuda"):
        """``save``: keep h and a for a backward (bf16). Without it, and always
        in MOE_DTYPE_MX8, only the forward runs."""
        self.T_max, self.d, self.F, self.dtype = T_max, d, F, dtype
        self.mx8 = dtype == L.MOE_DTYPE_MX8
        self.save = save and not self.mx8
        fwd, wgrad = L.moe_ffn_workspace_size(self.shape(T_max))
        self.device = dev = _device(device)
        bf = torch.bfloat16
        self.ws = torch.empty(max(wgrad if self.save else fwd, 256), dtype=torch.uint8, device=dev)
        self.y = torch.empty(T_max, d, dtype=bf, device=dev)
        self.h = torch.empty(T_max, 2 * F, dtype=bf, device=dev) if self.save else None
        self.a = torch.empty(T_max, F, dtype=bf, device=dev) if self.save else None
        self.dh = torch.empty(T_max, 2 * F, dtype=bf, device=dev) if self.save else None
        self.dx = torch.empty(T_max, d, dtype=bf, device=dev) if self.save else None

    def shape(self, T: int, overwrite: bool = False) -> L.moe_ffn_shape:
        return L.make_ffn_shape(T, self.d, self.F, self.dtype, L.MOE_FFN_OVERWRITE_DW if overwrite else 0)

    def _check_weights(self, w_gu, w_down):
        for name, w, shape in (("w_gu", w_gu, (2 * self.F, self.d)), ("w_down", w_down, (self.d, self.F))):
            if self.mx8:
                _check_mx8(name, w, None, shape, self.device)
            else:
                _check(name, w, None, shape, torch.bfloat16, self.device)

    def _rows(self, name, t, T):
        _check(name, t, T, (self.d,), torch.bfloat16, self.device)

    def _backward_ready(self):
        if not self.save:
            raise ValueError("this GatedFfn keeps nothing for a backward (save=False or MOE_DTYPE_MX8)")

    def check_forward(self, T: int, x, w_gu, w_down, add=None, out=None) -> None:
        _check_T(T, self.T_max)
        self._check_weights(w_gu, w_down)
        if self.mx8:
            _check_mx8("x", x, T, (self.d,), self.device)
        else:
            self._rows("x", x, T)
        for name, t in (("out", out), ("add", add)):
            if t is not None:
                self._rows(name, t, T)
        if self.save:
            _check_apart("x", x, T, self.y if out is None else out, "the output")

    def forward(self, T: int, x, w_gu, w_down, add=None, out=None, stream=None):
        """y = FFN(x) + add into ``out`` (which may be ``add``) or the object's
        buffer. MX8: x and the weights are ``Mx8``. Where a backward follows
        the output is not x, which ``wgrad`` reads again."""
        self.check_forward(T, x, w_gu, w_down, add, out)
        return self._forward(T, x, w_gu, w_down, add, out, stream)

    def _forward(self, T: int, x, w_gu, w_down, add, out, stream):
        out = self.y if out is None else out
        q = (lambda m: (m.q, m.scale)) if self.mx8 else (lambda m: (m, None))
        with _on(self.device):
            L.moe_ffn_fwd(self.shape(T), *q(x), *q(w_gu), *q(w_down), add, self.h, self.a, out, self.ws,
                          self.ws.numel(), stream)
        return out[:T]

    def check_dgrad(self, T: int, dy, w_gu, w_down, add=None, out=None) -> None:
        self._backward_ready()
        _check_T(T, self.T_max)
        self._check_weights(w_gu, w_down)
        self._rows("dy", dy, T)
        for name, t in (("out", out), ("add", add)):
            if t is not None:
                self._rows(name, t, T)
        _check_apart("dy", dy, T, self.dx if out is None else out, "the output")

    def dgrad(self, T: int, dy, w_gu, w_down, add=None, out=None, stream=None):
        """Gradient of x (plus ``add``) from the last forward's h into ``out``
        (which may be ``add``, not dy: ``wgrad`` reads that again) or the
        object's buffer; keeps dh for ``wgrad``."""
        self.check_dgrad(T, dy, w_gu, w_down, add, out)
        return self._dgrad(T, dy, w_gu, w_down, add, out, stream)

    def _dgrad(self, T: int, dy, w_gu, w_down, add, out, stream):
        out = self.dx if out is None else out
        with _on(self.device):
            L.moe_ffn_dgrad(self.shape(T), dy, self.h, w_gu, w_down, add, self.dh, out, stream)
        return out[:T]

    def check_wgrad(self, T: int, dy, x, dw_gu, dw_down) -> None:
        self._backward_ready()
        _check_T(T, self.T_max)
        self._rows("dy", dy, T)
        self._rows("x", x, T)
        _check("dw_gu", dw_gu, None, (2 * self.F, self.d), torch.float32, self.device)
        _check("dw_down", dw_down, None, (self.d, self.F), torch.float32, self.device)

    def wgrad(self, T: int, dy, x, dw_gu, dw_down, overwrite: bool = False, stream=None):
        """Weight gradients from the last forward's a and the last dgrad's dh;
        may run any time before either is written again."""
        self.check_wgrad(T, dy, x, dw_gu, dw_down)
        self._wgrad(T, dy, x, dw_gu, dw_down, overwrite, stream)

    def _wgrad(self, T: int, dy, x, dw_gu, dw_down, overwrite, stream):
        with _on(self.device):
            L.moe_ffn_wgrad(self.shape(T, overwrite), dy, x, self.a, self.dh, dw_gu, dw_down, self.ws,
                            self.ws.numel(), stream)


@dataclasses.dataclass
class LayerNormOut:
    """Views of a layer norm's outputs for one microbatch."""
    r: Optional[torch.Tensor]  # the new residual stream; None without a residual (it is x)
    y: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor


class LayerNorm:
    def __init__(self, T_max: int, d: int, dtype: int = L.MOE_DTYPE_BF16, eps: float = 1e-5, device: str = "cuda"):
        self.T_max, self.d, self.dtype, self.eps = T_max, d, dtype, eps
        self.ws_bytes = L.moe_layernorm_workspace_size(self.shape(T_max))
        self.device = dev = _device(device)
        self.td = _TORCH[dtype]
        self.ws = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)
        self.r = torch.empty(T_max, d, dtype=self.td, device=dev)
        self.y = torch.empty(T_max, d, dtype=self.td, device=dev)
        self.mean = torch.empty(T_max, dtype=torch.float32, device=dev)
        self.rstd = torch.empty(T_max, dtype=torch.float32, device=dev)
        self.dx = None  # made by the first backward: serving needs none

    def shape(self, T: int, overwrite: bool = False) -> L.moe_norm_shape:
        return L.make_norm_shape(T, self.d, self.dtype, self.eps, L.MOE_NORM_OVERWRITE_DW if overwrite else 0)

    def _vector(self, name, t, dtype):
        _check(name, t, None, (self.d,), dtype, self.device)

    def check_forward(self, T: int, x, weight, bias=None, residual=None) -> None:
        _check_T(T, self.T_max)
        _check("x", x, T, (self.d,), self.td, self.device)
        self._vector("weight", weight, self.td)
        if bias is not None:
            self._vector("bias", bias, self.td)
        if residual is not None:
            _check("residual", residual, T, (self.d,), self.td, self.device)

    def forward(self, T: int, x, weight, bias=None, residual=None, stream=None) -> LayerNormOut:
        """y = norm(x + residual) * weight + bias; r = x + residual is the new
        residual stream (in the object's buffer, valid until the next
        forward)."""
        self.check_forward(T, x, weight, bias, residual)
        r = self.r if residual is not None else None
        with _on(self.device):
            L.moe_layernorm_fwd(self.shape(T), x, residual, weight, bias, r, self.y, self.mean, self.rstd, stream)
        return LayerNormOut(None if r is None else r[:T], self.y[:T], self.mean[:T], self.rstd[:T])

    def check_backward(self, T: int, dy, r, weight, dw, db=None, dres=None, out=None) -> None:
        _check_T(T, self.T_max)
        for name, t in (("dy", dy), ("r", r)) + ((("dres", dres),) if dres is not None else ()):
            _check(name, t, T, (self.d,), self.td, self.device)
        self._vector("weight", weight, self.td)
        self._vector("dw", dw, torch.float32)
        if db is not None:
            self._vector("db", db, torch.float32)
        if out is not None:
            _check("out", out, T, (self.d,), self.td, self.device)

    def backward(self, T: int, dy, r, weight, dw, db=None, dres=None, overwrite: bool = False, out=None, stream=None):
        """Gradient of x (and of the residual alike) from dL/dy, with the mean
        and ``rstd`` of the last forward; ``r``: that forward's r, or its x if
        it had no residual; ``dres``: the gradient that reaches r directly.
        ``dw`` and ``db`` [d] fp32 accumulate (``overwrite``: are written)."""
        self.check_backward(T, dy, r, weight, dw, db, dres, out)
        if out is None:
            if self.dx is None:
                with _made_on(self.device, stream):
                    self.dx = torch.empty(self.T_max, self.d, dtype=self.td, device=self.device)
            out = self.dx
        with _on(self.device):
            L.moe_layernorm_bwd(self.shape(T, overwrite), dy, r, weight, self.mean, self.rstd, dres, out, dw, db, self.ws,
                                self.ws.numel(), stream)
        return out[:T]


class Linear:
    def __init__(self, T_max: int, K: int, N: int, act: int = L.MOE_ACT_NONE, save: bool = True, device: str = "cuda"):
        """y = act(x w^T + bias) + residual with w [N, K], bf16. ``save``: a
        backward follows (z is kept where there is an activation). Without it
        only the forward runs."""
        self.T_max, self.K, self.N, self.act, self.save = T_max, K, N, act, save
        wgrad = L.moe_linear_workspace_size(self.shape(T_max))
        self.device = dev = _device(device)
        new = lambda cols: torch.empty(T_max, cols, dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.ws = torch.empty(max(wgrad if save else 0, 256), dtype=torch.uint8, device=dev)
        self.y = new(N)
        self.z = new(N) if save and act != L.MOE_ACT_NONE else None
        self.dz = None  # made by the first dact: a product inside a chain needs none
        self.dx = new(K) if save else None

    def shape(self, T: int, overwrite: bool = False) -> L.moe_linear_shape:
        return L.make_linear_shape(T, self.K, self.N, L.MOE_DTYPE_BF16, self.act,
                                   L.MOE_LINEAR_OVERWRITE_DW if overwrite else 0)

    def _rows(self, name, t, T, cols):
        _check(name, t, T, (cols,), torch.bfloat16, self.device)

    def _weight(self, w):
        _check("w", w, None, (self.N, self.K), torch.bfloat16, self.device)

    def _backward_ready(self):
        if not self.save:
            raise ValueError("this Linear keeps nothing for a backward (save=False)")

    def check_forward(self, T: int, x, w, bias=None, residual=None, out=None) -> None:
        _check_T(T, self.T_max)
        self._weight(w)
        self._rows("x", x, T, self.K)
        if bias is not None:
            _check("bias", bias, None, (self.N,), torch.bfloat16, self.device)
        for name, t in (("residual", residual), ("out", out)):
            if t is not None:
                self._rows(name, t, T, self.N)
        written = self.y if out is None else out
        _check_apart("x", x, T, written, "the output")
        if self.z is not None:
            _check_apart("x", x, T, self.z, "z")
            _check_apart("the output", written, T, self.z, "z")
            if residual is not None:
                _check_apart("residual", residual, T, self.z, "z")

    def forward(self, T: int, x, w, bias=None, residual=None, out=None, stream=None):
        """y into ``out`` (which may be ``residual``) or the object's buffer."""
        self.check_forward(T, x, w, bias, residual, out)
        out = self.y if out is None else out
        with _on(self.device):
            L.moe_linear_fwd(self.shape(T), x, w, bias, residual, self.z, out, stream)
        return out[:T]

    def check_dact(self, T: int, dy, out=None) -> None:
        self._backward_ready()
        if self.z is None:
            raise ValueError("without an activation dz is dy")
        _check_T(T, self.T_max)
        self._rows("dy", dy, T, self.N)
        if out is not None:
            self._rows("out", out, T, self.N)

    def dact(self, T: int, dy, out=None, stream=None):
        """dz = dy * act'(z) with the last forward's z, into ``out`` (which may
        be dy) or the object's buffer: for an activation that ends a chain."""
        self.check_dact(T, dy, out)
        if out is None:
            if self.dz is None:
                with _made_on(self.device, stream):
                    self.dz = torch.empty(self.T_max, self.N, dtype=torch.bfloat16, device=self.device)
            out = self.dz
        with _on(self.device):
            L.moe_linear_dact(self.shape(T), dy, self.z, out, stream)
        return out[:T]

    def check_dgrad(self, T: int, dz, w, below: Optional["Linear"] = None, add=None, out=None) -> None:
        self._backward_ready()
        _check_T(T, self.T_max)
        self._weight(w)
        self._rows("dz", dz, T, self.N)
        for name, t in (("add", add), ("out", out)):
            if t is not None:
                self._rows(name, t, T, self.K)
        if below is not None:
            if below.z is None or below.N != self.K:
                raise ValueError(f"below: expected a Linear with an activation and N = {self.K} that keeps its z")
            self._rows("below.z", below.z, T, self.K)
        _check_apart("dz", dz, T, self.dx if out is None else out, "the output")

    def dgrad(self, T: int, dz, w, below: Optional["Linear"] = None, add=None, out=None, stream=None):
        """Gradient of x, plus ``add``, into ``out`` (which may be ``add``, not
        dz: ``wgrad`` reads that again) or the object's buffer. ``below``: the
        Linear whose last output was x; the result, times the derivative of its
        activation, is then its dz."""
        self.check_dgrad(T, dz, w, below, add, out)
        out = self.dx if out is None else out
        z, act = (None, L.MOE_ACT_NONE) if below is None else (below.z, below.act)
        with _on(self.device):
            L.moe_linear_dgrad(self.shape(T), dz, w, z, act, add, out, stream)
        return out[:T]

    def check_wgrad(self, T: int, dz, x, dw, db=None) -> None:
        self._backward_ready()
        _check_T(T, self.T_max)
        self._rows("dz", dz, T, self.N)
        self._rows("x", x, T, self.K)
        _check("dw", dw, None, (self.N, self.K), torch.float32, self.device)
        if db is not None:
            _check("db", db, None, (self.N,), torch.float32, self.device)

    def wgrad(self, T: int, dz, x, dw, db=None, overwrite: bool = False, stream=None):
        """Weight and bias gradients; may run any time before dz or x is
        written again."""
        self.check_wgrad(T, dz, x, dw, db)
        with _on(self.device):
            L.moe_linear_wgrad(self.shape(T, overwrite), dz, x, dw, db, self.ws, self.ws.numel(), stream)
