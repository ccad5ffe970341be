"""Outputs of the layer norm, the dense product and the orthogonalisation in the
memory of another tensor of their call (CPU only): refused before anything
could be launched."""
import pytest

torch = pytest.importorskip("torch")
import token_dispatch_grouped_amd as moe  # noqa: E402
from token_dispatch_grouped_amd import _lib as L  # noqa: E402

BF16, F32 = L.MOE_DTYPE_BF16, L.MOE_DTYPE_F32


def at(i):
    return (i + 1) << 28  # far enough apart


def refused(call, args, *words):
    with pytest.raises(moe.MoeError) as ei:
        call(*args, stream=0)
    assert ei.value.status == L.MOE_ERR_INVALID_ARGUMENT, str(ei.value)
    assert "shares memory" in str(ei.value) and all(w in str(ei.value) for w in words), str(ei.value)


T, D = 40, 128


def _norm(dtype, flags=0, rows=T):
    s = moe.make_norm_shape(rows, D, dtype, 1e-5, flags)
    return s, moe.moe_layernorm_workspace_size(s)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layernorm_forward_statistics_in_other_tensors(dtype):
    """mean and rstd are written while other rows are still read: neither may lie in the other, nor in a tensor that the
    call reads or writes."""
    width = 2 if dtype == BF16 else 4
    names = ("x", "residual", "weight", "bias", "r", "y", "mean", "rstd")
    sizes = dict(zip(names, (T * D * width, T * D * width, D * width, D * width, T * D * width, T * D * width, 4 * T, 4 * T)))
    s, _ = _norm(dtype)
    base = {n: at(i) for i, n in enumerate(names)}
    for out in ("mean", "rstd"):
        for other in names:
            if other == out:
                continue
            for place in (base[other], base[other] + sizes[other] - 16, base[other] - 4 * T + 16):
                refused(lambda *a, stream: moe.moe_layernorm_fwd(s, *a, stream=stream),
                        {**base, out: place}.values(), out, other)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layernorm_gradients_in_other_tensors(dtype):
    """dw and db apart from each other and from every tensor of the call; dx apart from the statistics."""
    width = 2 if dtype == BF16 else 4
    names = ("dy", "r", "weight", "mean", "rstd", "dres", "dx", "dw", "db")
    row = D * width
    sizes = dict(zip(names, (T * row, T * row, row, 4 * T, 4 * T, T * row, T * row, 4 * D, 4 * D)))
    base = {n: at(i) for i, n in enumerate(names)}
    for flags in (0, L.MOE_NORM_OVERWRITE_DW):
        s, n = _norm(dtype, flags)
        call = lambda *a, stream: moe.moe_layernorm_bwd(s, *a, at(20), n, stream=stream)  # noqa: E731
        for out in ("dw", "db"):
            for other in names:
                if other == out:
                    continue
                for place in (base[other], base[other] + sizes[other] - 16, base[other] - 4 * D + 16):
                    refused(call, {**base, out: place}.values(), out, other)
        for other in ("mean", "rstd"):
            for place in (base[other], base[other] + sizes[other] - 16, base[other] - T * row + 16):
                refused(call, {**base, "dx": place}.values(), "dx", other)


def test_layernorm_gradients_of_no_rows_in_one_tensor():
    s, n = _norm(BF16, L.MOE_NORM_OVERWRITE_DW, 0)
    refused(lambda *a, stream: moe.moe_layernorm_bwd(s, *a, None, 0, stream=stream), [None] * 7 + [at(0), at(0)], "dw", "db")


def _scratch(call, need, tensors):
    """Each tensor over the workspace's first and last bytes, and all around it."""
    ws = at(20)
    for name, size in tensors.items():
        for place in (ws, ws + need - 16, ws - size + 16):
            refused(lambda *a, stream: call(*a, ws, need, stream=stream),
                    {**{n: at(i) for i, n in enumerate(tensors)}, name: place}.values(), "ws", name)


@pytest.mark.parametrize("flags", [0, 1])
def test_workspace_in_other_tensors(flags):
    """The calls write their workspace before the last tensor is read."""
    s, n = _norm(F32, flags)
    row = 4 * D
    _scratch(lambda *a, stream: moe.moe_layernorm_bwd(s, *a, stream=stream), n,
             dict(dy=T * row, r=T * row, weight=row, mean=4 * T, rstd=4 * T, dres=T * row, dx=T * row, dw=row, db=row))
    for rows, K, N in ((T, 128, 192), (9001, 1088, 1088)):
        lin = moe.make_linear_shape(rows, K, N, flags=flags)
        _scratch(lambda *a, stream: moe.moe_linear_wgrad(lin, *a, stream=stream), moe.moe_linear_workspace_size(lin),
                 dict(dz=rows * N * 2, x=rows * K * 2, dw=N * K * 4, db=N * 4))
    orth = moe.make_orth_shape(2, 100, 70, BF16 if flags else F32)
    n = moe.moe_orthogonalize_workspace_size(orth)
    _scratch(lambda *a, stream: moe.moe_orthogonalize(orth, *a, stream=stream), n,
             dict(x=14000 * (2 if flags else 4), o=14000 * 2))
    orth = moe.make_orth_shape(2, 100, 70)
    cfg = moe.make_muon_config(0.1, nesterov=bool(flags))
    _scratch(lambda *a, stream: moe.moe_muon_step(cfg, orth, *a, stream=stream), n,
             dict(param=56000, grad=56000, momentum=56000, param_bf16=28000))
