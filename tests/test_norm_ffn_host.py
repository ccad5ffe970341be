"""Refusals of the norm, the 8-bit block form and the dense block (CPU only):
every call below returns its status before anything could be launched."""
import pytest

import token_dispatch_grouped_amd as moe
from token_dispatch_grouped_amd import _lib as L

FAKE = 1 << 12  # a 16-byte aligned address that nothing reads
BF16, F32, MX8 = L.MOE_DTYPE_BF16, L.MOE_DTYPE_F32, L.MOE_DTYPE_MX8
ARG, UNS, WS, MIS = (L.MOE_ERR_INVALID_ARGUMENT, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE, L.MOE_ERR_MISALIGNED)


def refused(status, call, *args, word=""):
    with pytest.raises(moe.MoeError) as ei:
        call(*args, stream=0)
    assert ei.value.status == status and word in str(ei.value), str(ei.value)


def norm_fwd(s, x=FAKE, residual=FAKE, w=FAKE, r=FAKE, y=FAKE, ys=None, rstd=FAKE):
    return (s, x, residual, w, r, y, ys, rstd)


NORM_SHAPES = [
    (dict(T=-1), ARG), (dict(d=0), ARG), (dict(d=96), UNS), (dict(d=65600), UNS), (dict(T=1 << 24), UNS),
    (dict(dtype=MX8), UNS), (dict(dtype=7), UNS), (dict(eps=0.0), ARG), (dict(eps=-1e-6), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(flags=2), UNS),
]


@pytest.mark.parametrize("kw,status", NORM_SHAPES)
def test_norm_shapes(kw, status):
    s = moe.make_norm_shape(**{**dict(T=4, d=128, dtype=BF16, eps=1e-6, flags=0), **kw})
    refused(status, moe.moe_rmsnorm_fwd, *norm_fwd(s))
    refused(status, moe.moe_rmsnorm_bwd, s, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, 1 << 30)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_rmsnorm_workspace_size(s)
    assert ei.value.status == status


def test_norm_pointers():
    s = moe.make_norm_shape(4, 128, BF16)
    for name, kw in (("x", dict(x=None)), ("weight", dict(w=None)), ("y", dict(y=None)), ("rstd", dict(rstd=None)),
                     ("r", dict(r=None))):
        refused(ARG, moe.moe_rmsnorm_fwd, *norm_fwd(s, **kw), word=name)
    refused(ARG, moe.moe_rmsnorm_fwd, *norm_fwd(s, residual=None), word="must be NULL")  # r without a residual
    for kw in (dict(x=FAKE + 8), dict(residual=FAKE + 2), dict(y=FAKE + 1), dict(ys=FAKE + 4)):
        refused(MIS, moe.moe_rmsnorm_fwd, *norm_fwd(s, **kw))
    n = moe.moe_rmsnorm_workspace_size(s)
    assert n > 0
    bwd = lambda **k: [k.get(a, b) for a, b in (("s", s), ("dy", FAKE), ("r", FAKE), ("w", FAKE), ("rstd", FAKE),  # noqa: E731
                                                ("dres", None), ("dx", FAKE), ("dw", FAKE), ("ws", FAKE), ("n", n))]
    for name in ("dy", "r", "rstd", "dx", "dw"):
        refused(ARG, moe.moe_rmsnorm_bwd, *bwd(**{name: None}), word=name)
    refused(WS, moe.moe_rmsnorm_bwd, *bwd(ws=None))
    refused(WS, moe.moe_rmsnorm_bwd, *bwd(n=n - 1))
    refused(MIS, moe.moe_rmsnorm_bwd, *bwd(ws=FAKE + 8))
    refused(MIS, moe.moe_rmsnorm_bwd, *bwd(dres=FAKE + 8))


def test_empty_calls_are_no_ops():
    moe.moe_rmsnorm_fwd(moe.make_norm_shape(0, 128, BF16), None, None, None, None, None, None, None, stream=0)
    moe.moe_rmsnorm_bwd(moe.make_norm_shape(0, 128, BF16), None, None, None, None, None, None, None, None, 0, stream=0)
    moe.moe_mx8_quantize(0, 128, BF16, None, None, None, stream=0)
    for dt in (BF16, MX8):
        s = moe.make_ffn_shape(0, 128, 128, dt)
        moe.moe_ffn_fwd(s, None, None, None, None, None, None, None, None, None, None, None, 0, stream=0)
    moe.moe_ffn_dgrad(moe.make_ffn_shape(0, 128, 128), None, None, None, None, None, None, None, stream=0)
    moe.moe_ffn_wgrad(moe.make_ffn_shape(0, 128, 128), None, None, None, None, None, None, None, 0, stream=0)
    # with OVERWRITE_DW the gradient is written (zeros), so it is needed
    refused(ARG, moe.moe_rmsnorm_bwd, moe.make_norm_shape(0, 128, BF16, 1e-6, L.MOE_NORM_OVERWRITE_DW), None, None, None,
            None, None, None, None, None, 0, word="dw")
    refused(ARG, moe.moe_ffn_wgrad, moe.make_ffn_shape(0, 128, 128, BF16, L.MOE_FFN_OVERWRITE_DW), None, None, None,
            None, None, FAKE, None, 0, word="dw_gu")


def test_quantize_refusals():
    for args, st in (((-1, 128, BF16), ARG), ((4, 0, BF16), ARG), ((4, 96, BF16), UNS), ((4, 65600, F32), UNS),
                     ((4, 128, MX8), UNS), ((1 << 32, 128, BF16), UNS), (((1 << 32) // 16, 128, BF16), UNS)):
        refused(st, moe.moe_mx8_quantize, *args, FAKE, FAKE, FAKE)
    for i in range(3):
        p = [FAKE] * 3
        p[i] = None
        refused(ARG, moe.moe_mx8_quantize, 4, 128, BF16, *p)
        p[i] = FAKE + 4
        refused(MIS, moe.moe_mx8_quantize, 4, 128, BF16, *p)


FFN_SHAPES = [
    (dict(T=-1), ARG), (dict(d=0), ARG), (dict(F=0), ARG), (dict(d=96), UNS), (dict(F=96), UNS), (dict(d=65600), UNS),
    (dict(F=65600), UNS), (dict(T=1 << 24), UNS), (dict(dtype=F32), UNS), (dict(dtype=9), UNS), (dict(flags=4), UNS),
    (dict(dtype=MX8, d=64), UNS), (dict(dtype=MX8, F=192), UNS), (dict(T=(1 << 24) - 1, d=65536), UNS),
]


@pytest.mark.parametrize("kw,status", FFN_SHAPES)
def test_ffn_shapes(kw, status):
    s = moe.make_ffn_shape(**{**dict(T=4, d=128, F=128, dtype=BF16, flags=0), **kw})
    refused(status, moe.moe_ffn_fwd, s, FAKE, None, FAKE, None, FAKE, None, None, None, None, FAKE, FAKE, 1 << 40)
    refused(status, moe.moe_ffn_dgrad, s, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE)
    refused(status, moe.moe_ffn_wgrad, s, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_ffn_workspace_size(s)
    assert ei.value.status == status


def test_ffn_pointers():
    s = moe.make_ffn_shape(4, 128, 128)
    fwd, wgrad = moe.moe_ffn_workspace_size(s)
    names = ("x", "x_scale", "w_gu", "w_gu_scale", "w_down", "w_down_scale", "add", "h", "a", "y")

    def call(shape, ws=FAKE, n=1 << 30, **kw):
        base = dict(x=FAKE, w_gu=FAKE, w_down=FAKE, y=FAKE)
        if shape.dtype == MX8:
            base.update(x_scale=FAKE, w_gu_scale=FAKE, w_down_scale=FAKE)
        base.update(kw)
        return (shape,) + tuple(base.get(k) for k in names) + (ws, n)

    for k in ("x", "w_gu", "w_down", "y"):
        refused(ARG, moe.moe_ffn_fwd, *call(s, **{k: None}), word=k)
        refused(MIS, moe.moe_ffn_fwd, *call(s, **{k: FAKE + 8}), word=k)
    for k in ("x_scale", "w_gu_scale", "w_down_scale"):
        refused(ARG, moe.moe_ffn_fwd, *call(s, **{k: FAKE}), word="must be NULL")
    refused(ARG, moe.moe_ffn_fwd, *call(s, h=FAKE), word="a is NULL")  # both or neither
    refused(ARG, moe.moe_ffn_fwd, *call(s, a=FAKE), word="h is NULL")
    refused(WS, moe.moe_ffn_fwd, *call(s, ws=None))
    refused(WS, moe.moe_ffn_fwd, *call(s, n=fwd - 1))
    m = moe.make_ffn_shape(4, 128, 128, MX8)
    for k in ("x_scale", "w_gu_scale", "w_down_scale"):
        refused(ARG, moe.moe_ffn_fwd, *call(m, **{k: None}), word=k)
    for k in ("h", "a"):
        refused(ARG, moe.moe_ffn_fwd, *call(m, **{k: FAKE}), word="must be NULL")
    refused(WS, moe.moe_ffn_fwd, *call(m, n=moe.moe_ffn_workspace_size(m)[0] - 1))
    refused(UNS, moe.moe_ffn_dgrad, m, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, word="BF16")
    refused(UNS, moe.moe_ffn_wgrad, m, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, word="BF16")
    for i, k in enumerate(("dy", "h", "w_gu", "w_down", None, "dh", "dx")):
        args = [FAKE] * 7
        if k:
            args[i] = None
            refused(ARG, moe.moe_ffn_dgrad, s, *args, word=k)
        args[i] = FAKE + 8
        refused(MIS, moe.moe_ffn_dgrad, s, *args)
    for i, k in enumerate(("dy", "x", "a", "dh", "dw_gu", "dw_down")):
        args = [FAKE] * 6
        args[i] = None
        refused(ARG, moe.moe_ffn_wgrad, s, *args, FAKE, wgrad, word=k)
    refused(WS, moe.moe_ffn_wgrad, s, *[FAKE] * 6, FAKE, wgrad - 1)
    refused(WS, moe.moe_ffn_wgrad, s, *[FAKE] * 6, None, 0)


@pytest.mark.parametrize("d,F", [(64, 64), (512, 320), (2048, 1408), (4096, 2816), (65536, 128)])
def test_workspaces_never_shrink_with_T(d, F):
    last = (0, 0, 0, 0)
    for T in list(range(0, 700, 7)) + [767, 768, 1000, 2559, 2560, 2561, 4096, 7001, 16384, 20480, 20500, 32768, 40000]:
        now = moe.moe_ffn_workspace_size(moe.make_ffn_shape(T, d, F))
        now += moe.moe_ffn_workspace_size(moe.make_ffn_shape(T, d, max(128, F // 128 * 128), MX8))[:1] if d % 128 == 0 else (0,)
        now += (moe.moe_rmsnorm_workspace_size(moe.make_norm_shape(T, d, BF16)),)
        assert all(a <= b for a, b in zip(last, now)), (T, last, now)
        last = now


def test_the_layers_calls_refuse_mx8():
    s = L.make_shape(4, 128, 4, 2, 128, MX8)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_permute(s, FAKE, FAKE, FAKE, stream=0)
    assert ei.value.status == UNS
