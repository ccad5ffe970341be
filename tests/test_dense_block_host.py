"""Refusals of the layer norm, the dense product and the orthogonalisation (CPU
only): every call below returns its status before anything could be launched,
and the Python objects refuse wrong tensors before anything is called."""
import pytest

torch = pytest.importorskip("torch")
import token_dispatch_grouped_amd as moe  # noqa: E402
from token_dispatch_grouped_amd import _lib as L, block, optim  # noqa: E402

FAKE = 1 << 12  # a 16-byte aligned address that nothing reads
BF16, F32, MX8 = L.MOE_DTYPE_BF16, L.MOE_DTYPE_F32, L.MOE_DTYPE_MX8
ARG, UNS, WS, MIS = (L.MOE_ERR_INVALID_ARGUMENT, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE, L.MOE_ERR_MISALIGNED)
BIG = 1 << 50


def refused(status, call, *args, word=""):
    with pytest.raises(moe.MoeError) as ei:
        call(*args, stream=0)
    assert ei.value.status == status and word in str(ei.value), str(ei.value)


def each_pointer(call, args, names, optional=()):
    """Every needed pointer missing, and every pointer off its alignment. args: the pointers, in order."""
    for i, name in enumerate(names):
        a = list(args)
        if name not in optional:
            a[i] = None
            refused(ARG, call, *a, word=name)
        a[i] = FAKE + 8
        refused(MIS, call, *a, word=name)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(d=0), ARG), (dict(d=96), UNS), (dict(d=65600), UNS), (dict(T=1 << 24), UNS),
    (dict(dtype=MX8), UNS), (dict(dtype=7), UNS), (dict(eps=0.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(flags=2), UNS)])
def test_layernorm_shapes(kw, status):
    s = moe.make_norm_shape(**{**dict(T=4, d=128, dtype=BF16, eps=1e-6, flags=0), **kw})
    refused(status, moe.moe_layernorm_fwd, s, *[FAKE] * 8)
    refused(status, moe.moe_layernorm_bwd, s, *[FAKE] * 9, FAKE, BIG)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_layernorm_workspace_size(s)
    assert ei.value.status == status


def test_layernorm_pointers():
    s = moe.make_norm_shape(4, 128, BF16)
    each_pointer(lambda *a, stream: moe.moe_layernorm_fwd(s, *a, stream=stream), [FAKE] * 8,
                 ("x", "residual", "weight", "bias", "r", "y", "mean", "rstd"), ("residual", "bias"))
    refused(ARG, moe.moe_layernorm_fwd, s, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, word="must be NULL")
    n = moe.moe_layernorm_workspace_size(s)
    each_pointer(lambda *a, stream: moe.moe_layernorm_bwd(s, *a, FAKE, n, stream=stream), [FAKE] * 9,
                 ("dy", "r", "weight", "mean", "rstd", "dres", "dx", "dw", "db"), ("dres", "db"))
    for ws, size, st in ((None, n, WS), (FAKE, n - 1, WS), (FAKE + 8, n, MIS)):
        refused(st, moe.moe_layernorm_bwd, s, *[FAKE] * 9, ws, size)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(K=0), ARG), (dict(N=-64), ARG), (dict(K=96), UNS), (dict(N=32), UNS), (dict(K=65600), UNS),
    (dict(N=65600), UNS), (dict(T=1 << 24), UNS), (dict(dtype=F32), UNS), (dict(dtype=MX8), UNS), (dict(act=5), UNS),
    (dict(act=-1), UNS), (dict(flags=2), UNS), (dict(T=(1 << 24) - 1, N=65536), UNS), (dict(T=(1 << 24) - 1, K=65536), UNS)])
def test_linear_shapes(kw, status):
    s = moe.make_linear_shape(**{**dict(T=4, K=128, N=128, dtype=BF16, act=1, flags=0), **kw})
    refused(status, moe.moe_linear_fwd, s, FAKE, FAKE, None, None, None, FAKE)
    refused(status, moe.moe_linear_dact, s, FAKE, FAKE, FAKE)
    refused(status, moe.moe_linear_dgrad, s, FAKE, FAKE, None, 0, None, FAKE)
    refused(status, moe.moe_linear_wgrad, s, FAKE, FAKE, FAKE, FAKE, FAKE, BIG)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_linear_workspace_size(s)
    assert ei.value.status == status


def test_linear_pointers():
    s = moe.make_linear_shape(4, 128, 192, act=moe.MOE_ACT_GELU)
    far = [FAKE * (i + 1) for i in range(6)]
    each_pointer(lambda *a, stream: moe.moe_linear_fwd(s, *a, stream=stream), far,
                 ("x", "w", "bias", "residual", "z", "y"), ("bias", "residual", "z"))
    refused(ARG, moe.moe_linear_fwd, s, FAKE, FAKE, None, None, FAKE, FAKE, word="z")
    refused(ARG, moe.moe_linear_fwd, s, FAKE, FAKE, None, 2 * FAKE, 2 * FAKE, FAKE, word="z")
    each_pointer(lambda *a, stream: moe.moe_linear_dact(s, *a, stream=stream), [FAKE] * 3, ("dy", "z", "dz"))
    refused(ARG, moe.moe_linear_dact, moe.make_linear_shape(4, 128, 192), FAKE, FAKE, FAKE, word="dz is dy")
    each_pointer(lambda dz, w, z, add, dx, stream: moe.moe_linear_dgrad(s, dz, w, z, 2, add, dx, stream=stream), [FAKE] * 5,
                 ("dz", "w", "z_in", "add", "dx"), ("add",))
    refused(ARG, moe.moe_linear_dgrad, s, FAKE, FAKE, FAKE, 0, None, FAKE, word="must be NULL")
    for bad in (-1, 5):
        refused(UNS, moe.moe_linear_dgrad, s, FAKE, FAKE, FAKE, bad, None, FAKE, word="activation")
    n = moe.moe_linear_workspace_size(s)
    each_pointer(lambda *a, stream: moe.moe_linear_wgrad(s, *a, FAKE, n, stream=stream), [FAKE] * 4, ("dz", "x", "dw", "db"),
                 ("db",))
    for ws, size, st in ((None, n, WS), (FAKE, n - 1, WS), (FAKE + 8, n, MIS)):
        refused(st, moe.moe_linear_wgrad, s, *[FAKE] * 4, ws, size)


def test_outputs_in_other_tensors_memory():
    """An output over an input that another workgroup still reads, in whole or shifted by a row, is refused."""
    A = lambda i: (i + 1) << 24  # noqa: E731  far enough apart
    row, T, K, N = 256, 4, 128, 192  # bytes of a row of 128 bf16 values
    ln = moe.make_norm_shape(T, 128, BF16)
    for out in (dict(r=A(0) + row), dict(r=A(1) + row), dict(y=A(0) + row), dict(y=A(1) + 3 * row), dict(y=A(4)), dict(r=A(2)),
                dict(y=A(3))):
        a = {**dict(x=A(0), residual=A(1), weight=A(2), bias=A(3), r=A(4), y=A(5), mean=A(6), rstd=A(7)), **out}
        refused(ARG, moe.moe_layernorm_fwd, ln, *a.values(), word="shares memory")
    n = moe.moe_layernorm_workspace_size(ln)
    for dx in (A(0) + row, A(1) + row, A(5) + row, A(2)):
        refused(ARG, moe.moe_layernorm_bwd, ln, *[A(i) for i in range(6)], dx, A(7), A(8), A(9), n, word="shares memory")
    lin = moe.make_linear_shape(T, K, N, act=moe.MOE_ACT_GELU)
    for out in (dict(y=A(0)), dict(z=A(0)), dict(y=A(1) + 64), dict(z=A(1)), dict(y=A(3) + 2 * N), dict(z=A(3) + 2 * N),
                dict(z=A(5) + 2 * N), dict(y=A(2))):
        a = {**dict(x=A(0), w=A(1), bias=A(2), residual=A(3), z=A(4), y=A(5)), **out}
        refused(ARG, moe.moe_linear_fwd, lin, *a.values(), word="shares memory")
    for dz in (A(0) + 2 * N, A(1) + 2 * N):
        refused(ARG, moe.moe_linear_dact, lin, A(0), A(1), dz, word="shares memory")
    for dx in (A(0), A(1), A(2) + row, A(3) + row):
        refused(ARG, moe.moe_linear_dgrad, lin, A(0), A(1), A(2), moe.MOE_ACT_GELU, A(3), dx, word="shares memory")
    n = moe.moe_linear_workspace_size(lin)
    for dw, db in ((A(0), A(3)), (A(1), A(3)), (A(2), A(0)), (A(2), A(1)), (A(2), A(2) + 1024)):
        refused(ARG, moe.moe_linear_wgrad, lin, A(0), A(1), dw, db, A(5), n, word="shares memory")
    orth = moe.make_orth_shape(2, 100, 70)
    n = moe.moe_orthogonalize_workspace_size(orth)
    for a in ((A(0), A(0), A(2), A(3)), (A(0), A(1), A(1), A(3)), (A(0), A(1), A(0) + 400, A(3)), (A(0), A(1), A(2), A(0)),
              (A(0), A(1), A(2), A(1) + 64)):
        refused(ARG, moe.moe_muon_step, moe.make_muon_config(0.1), orth, *a, A(5), n, word="shares memory")


ORTH = dict(batch=2, rows=100, cols=70, dtype=F32, steps=5, coef=moe._lib.ORTH_COEF, eps=1e-7)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), ARG), (dict(rows=0), ARG), (dict(cols=-1), ARG), (dict(rows=65537), UNS), (dict(cols=65537), UNS),
    (dict(dtype=MX8), UNS), (dict(steps=0), UNS), (dict(steps=17), UNS), (dict(eps=0.0), ARG), (dict(eps=float("inf")), ARG),
    (dict(coef=(float("nan"), 0, 0)), ARG), (dict(coef=(3.0, 0.0, 0.0)), UNS), (dict(coef=(1.0, 20.0, 0.0)), UNS),
    (dict(coef=(0.0, 40.0, -40.0)), UNS), (dict(coef=(1.0, 0.0, 3.0)), UNS), (dict(batch=1 << 22), UNS),
    (dict(batch=5, rows=65536, cols=65536), UNS)])
def test_orth_shapes(kw, status):
    s = moe.make_orth_shape(**{**ORTH, **kw})
    refused(status, moe.moe_orthogonalize, s, FAKE, FAKE, FAKE, BIG)
    refused(status, moe.moe_muon_step, moe.make_muon_config(0.1), s, FAKE, FAKE, FAKE, None, FAKE, BIG)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_orthogonalize_workspace_size(s)
    assert ei.value.status == status


@pytest.mark.parametrize("steps,coef", [(16, (3.4445, -4.7750, 2.0315)), (16, (1.5, -0.5, 0.0)), (1, (3.0, 0.0, 0.0)),
                                        (2, (3.0, 0.0, 0.0)), (8, (2.0, -1.5, 0.5)), (16, (0.0, 0.0, 0.0))])
def test_orth_coefficients_in_range(steps, coef):
    assert moe.moe_orthogonalize_workspace_size(moe.make_orth_shape(1, 8, 8, F32, steps, coef)) > 0


def test_orth_pointers():
    s = moe.make_orth_shape(2, 100, 70)
    n = moe.moe_orthogonalize_workspace_size(s)
    each_pointer(lambda *a, stream: moe.moe_orthogonalize(s, *a, FAKE, n, stream=stream), [FAKE] * 2, ("x", "o"))
    cfg = moe.make_muon_config(0.1)
    each_pointer(lambda *a, stream: moe.moe_muon_step(cfg, s, *a, FAKE, n, stream=stream), [FAKE] * 4,
                 ("param", "grad", "momentum", "param_bf16"), ("param_bf16",))
    for ws, size, st in ((None, n, WS), (FAKE, n - 1, WS), (FAKE + 8, n, MIS)):
        refused(st, moe.moe_orthogonalize, s, FAKE, FAKE, ws, size)
        refused(st, moe.moe_muon_step, cfg, s, *[FAKE] * 4, ws, size)
    refused(UNS, moe.moe_muon_step, cfg, moe.make_orth_shape(2, 100, 70, BF16), *[FAKE] * 4, FAKE, BIG, word="F32")
    for kw, st in ((dict(lr=float("nan")), ARG), (dict(weight_decay=float("inf")), ARG), (dict(scale=float("inf")), ARG),
                   (dict(grad_scale=float("nan")), ARG), (dict(momentum=1.0), ARG), (dict(momentum=-0.1), ARG)):
        refused(st, moe.moe_muon_step, moe.make_muon_config(**{**dict(lr=0.1), **kw}), s, *[FAKE] * 4, FAKE, n)
    cfg.flags = 4
    refused(UNS, moe.moe_muon_step, cfg, s, *[FAKE] * 4, FAKE, n, word="flag")


def test_empty_calls_are_no_ops():
    none = moe.make_norm_shape(0, 128, BF16)
    moe.moe_layernorm_fwd(none, *[None] * 8, stream=0)
    moe.moe_layernorm_bwd(none, *[None] * 10, 0, stream=0)
    lin = moe.make_linear_shape(0, 128, 64, act=1)
    moe.moe_linear_fwd(lin, *[None] * 6, stream=0)
    moe.moe_linear_dact(lin, None, None, None, stream=0)
    moe.moe_linear_dgrad(lin, None, None, None, 0, None, None, stream=0)
    moe.moe_linear_wgrad(lin, *[None] * 5, 0, stream=0)
    orth = moe.make_orth_shape(0, 10, 10)
    moe.moe_orthogonalize(orth, None, None, None, 0, stream=0)
    moe.moe_muon_step(moe.make_muon_config(0.1), orth, *[None] * 5, 0, stream=0)
    # with OVERWRITE_DW the gradient is written (zeros), so it is needed
    refused(ARG, moe.moe_layernorm_bwd, moe.make_norm_shape(0, 128, BF16, 1e-6, L.MOE_NORM_OVERWRITE_DW), *[None] * 10, 0,
            word="dw")
    refused(ARG, moe.moe_linear_wgrad, moe.make_linear_shape(0, 128, 64, flags=L.MOE_LINEAR_OVERWRITE_DW), *[None] * 5, 0,
            word="dw")


@pytest.mark.parametrize("K,N", [(64, 64), (512, 320), (2048, 1408), (8192, 2048), (65536, 128)])
def test_workspaces_never_shrink(K, N):
    last = (0, 0)
    for T in list(range(0, 700, 7)) + [767, 768, 1000, 2559, 2560, 2561, 4096, 7001, 16384, 20480, 20500, 32768, 40000]:
        now = (moe.moe_linear_workspace_size(moe.make_linear_shape(T, K, N)),
               moe.moe_layernorm_workspace_size(moe.make_norm_shape(T, K, BF16)))
        assert all(a <= b for a, b in zip(last, now)), (T, last, now)
        last = now
    sizes = [moe.moe_orthogonalize_workspace_size(moe.make_orth_shape(b, 65, 130)) for b in range(9)]
    assert sizes == sorted(sizes) and sizes[0] == 0


def test_orthogonalisation_workspace_serves_every_smaller_batch():
    """Also where a smaller batch takes the sums of X X^T in slices and a larger one does not."""
    for rows, cols in ((1500, 4200), (4200, 1500), (2048, 8192), (2816, 4096), (2817, 4096), (64, 65536), (2048, 4032)):
        sizes = [moe.moe_orthogonalize_workspace_size(moe.make_orth_shape(b, rows, cols)) for b in range(6)]
        assert sizes == sorted(sizes) and sizes[0] == 0


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


F = torch.float32


def test_layernorm_object():
    n = block.LayerNorm(8, 128, device="cpu")
    x, w = t(8, 128), t(128)
    for bad in (t(8, 128, dtype=F), t(7, 128), t(8, 64), t(128, 8).t(), t(2, 8, 128), None, 3):
        with pytest.raises(ValueError, match="x"):
            n.forward(8, bad, w)
    for kw, word in ((dict(weight=t(128, dtype=F)), "weight"), (dict(bias=t(64)), "bias"), (dict(residual=t(6, 128)), "residual")):
        with pytest.raises(ValueError, match=word):
            n.forward(8, x, **{**dict(weight=w), **kw})
    for T in (-1, 9):
        with pytest.raises(ValueError, match="T ="):
            n.forward(T, x, w)
    dw = t(128, dtype=F)
    for args, kw, word in (((8, x, x, w, t(128)), {}, "dw"), ((8, x, x, w, dw), dict(db=t(64, dtype=F)), "db"),
                           ((8, x, x, w, dw), dict(dres=t(8, 64)), "dres"), ((8, x, x, w, dw), dict(out=t(4, 128)), "out")):
        with pytest.raises(ValueError, match=word):
            n.backward(*args, **kw)
    with pytest.raises(moe.MoeError):
        block.LayerNorm(8, 100, device="cpu")


def test_linear_object():
    f = block.Linear(8, 128, 192, moe.MOE_ACT_GELU, device="cpu")
    x, w, y = t(8, 128), t(192, 128), t(8, 192)
    for args, kw, word in (((8, t(8, 64), w), {}, "x"), ((8, x, t(128, 192)), {}, "w"), ((9, x, w), {}, "T ="),
                           ((8, x, w), dict(bias=t(128)), "bias"), ((8, x, w), dict(residual=t(8, 128)), "residual"),
                           ((8, x, w), dict(out=t(4, 192)), "out"), ((8, x, w), dict(out=f.z), "z"),
                           ((8, x, w), dict(residual=f.z), "z")):
        with pytest.raises(ValueError, match=word):
            f.forward(*args, **kw)
    sq = block.Linear(8, 128, 128, device="cpu")
    with pytest.raises(ValueError, match="copy"):
        sq.forward(8, x, t(128, 128), out=x)
    with pytest.raises(ValueError, match="dz is dy"):
        sq.dact(8, x)
    for dz, kw, word in ((t(8, 128), {}, "dz"), (y, dict(add=y), "add"), (y, dict(out=t(8, 64)), "out"),
                         (y, dict(below=sq), "below"), (y, dict(below=f), "below")):
        with pytest.raises(ValueError, match=word):
            f.dgrad(8, dz, w, **kw)
    with pytest.raises(ValueError, match="copy"):
        sq.dgrad(8, x, t(128, 128), out=x)
    for dw, db, word in ((t(192, 128), None, "dw"), (t(192, 128, dtype=F), t(192), "db")):
        with pytest.raises(ValueError, match=word):
            f.wgrad(8, y, x, dw, db)
    g = block.Linear(8, 128, 192, moe.MOE_ACT_RELU, save=False, device="cpu")
    for call in (lambda: g.dact(8, y), lambda: g.dgrad(8, y, w), lambda: g.wgrad(8, y, x, t(192, 128, dtype=F))):
        with pytest.raises(ValueError, match="backward"):
            call()
    with pytest.raises(moe.MoeError):
        block.Linear(8, 128, 100, device="cpu")
    with pytest.raises(moe.MoeError):
        block.Linear(8, 128, 128, 9, device="cpu")


def test_orthogonalizer_and_muon_objects():
    o = optim.Orthogonalizer(2, 30, 40, device="cpu")
    for args, kw, word in (((2, t(2, 30, 40)), {}, "x"), ((3, t(3, 30, 40, dtype=F)), {}, "T ="),
                           ((2, t(2, 30, 40, dtype=F)), dict(out=t(2, 40, 30)), "out")):
        with pytest.raises(ValueError, match=word):
            o.forward(*args, **kw)
    for weights, kw, word in (([t(8)], {}, "dimensions"), ([t(4, 6).t()], {}, "contiguous"),
                              ([t(4, 6, dtype=torch.float16)], {}, "contiguous"), ([t(2, 5, 6)], dict(parts=[2]), "stack"),
                              ([t(2, 6, 6)], dict(parts=[1, 1]), "parts"), ([t(2, 6, 6)], dict(parts=[0]), "stack")):
        with pytest.raises(ValueError, match=word):
            optim.ExpertMuon(weights, 0.1, **kw)
    opt = optim.ExpertMuon([t(2, 8, 6), t(5, 7)], 0.1, parts=[2, 1])
    assert [(s.batch, s.rows, s.cols) for s in opt.shapes] == [(4, 4, 6), (1, 5, 7)]
    good = [t(2, 8, 6, dtype=F), t(5, 7, dtype=F)]
    for bad in (good[:1], [good[0], t(7, 5, dtype=F)], [good[0], t(5, 7)], [good[0], t(7, 5, dtype=F).t()]):
        with pytest.raises(ValueError, match="gradient"):
            opt.step(bad)
    assert all(not m.any() for m in opt.momenta)


def test_muon_refuses_weights_without_rows_or_columns():
    for shape in ((0, 6), (4, 0), (2, 0, 6)):
        with pytest.raises(ValueError, match="rows and columns"):
            optim.ExpertMuon([t(*shape)], 0.1)
    assert [s.batch for s in optim.ExpertMuon([t(0, 4, 6)], 0.1).shapes] == [0]
