"""The layer norm and its backward pass against the fp64 oracle, through the C
ABI.

Tolerances, per element and derived: u = 2^-24 is half an fp32 step. A row's
sums are chains of at most d/64 + 16 additions (a thread's own values, then the
tree). The mean's first sum only has to be near: what it is off by is summed
again, over values r - m0 of the size of the spread, so the mean is off by
half a step of its own and by A = (d/64 + 24) u of the spread sd, however large
it is beside sd; rstd carries A, n = (r - mean) rstd then A (|n| + 2), and y that
times |weight|, A |bias| and half a step of its type.
"""
import numpy as np
import pytest

import oracle
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5


def _moe():
    import token_dispatch_grouped_amd as m
    return m


def _torch(bf16):
    import torch
    return torch.bfloat16 if bf16 else torch.float32


def _dt(bf16):
    m = _moe()
    return m.MOE_DTYPE_BF16 if bf16 else m.MOE_DTYPE_F32


def _rand(rng, *shape, bf16=True, std=1.0, mean=0.0):
    import torch
    return torch.from_numpy(rng.normal(mean, std, shape).astype(np.float32)).to(_torch(bf16)).cuda()


def _h(t):
    return t.double().cpu().numpy()


def _arith(d):
    return (d / 64 + 24) * U


def _half(bf16):
    return 2.0 ** -8 if bf16 else 0.0


def _round_r(bf16):
    if bf16:
        return lambda v: bf16_bits_to_f32(f32_to_bf16_bits(v.astype(np.float32))).astype(np.float64)
    return lambda v: v.astype(np.float32).astype(np.float64)


def _nan(*shape, dtype=None):
    import torch
    return torch.full(shape, float("nan"), dtype=dtype or torch.float32, device="cuda")


def _fwd(m, x, res, w, b, bf16, r_alias=False, eps=EPS):
    import torch
    T, d = x.shape
    r = None if res is None else (res if r_alias else torch.full_like(x, float("nan")))
    mean, rstd, y = _nan(T), _nan(T), torch.full_like(x, float("nan"))
    m.moe_layernorm_fwd(m.make_norm_shape(T, d, _dt(bf16), eps), x, res, w, b, r, y, mean, rstd)
    torch.cuda.synchronize()
    return r, y, mean, rstd


def _check_fwd(out, x, res, w, b, bf16):
    r, y, mean, rstd = out
    d = x.shape[1]
    r64, mean64, rstd64, n64, y64 = oracle.layernorm_fwd(_h(x), _h(w), None if b is None else _h(b), EPS,
                                                         None if res is None else _h(res), _round_r(bf16))
    if res is not None:
        assert np.array_equal(_h(r), r64)  # one correctly rounded addition
    sd = np.std(r64, axis=1)
    assert np.all(np.abs(_h(mean) - mean64) <= U * np.abs(mean64) + _arith(d) * sd)
    assert np.all(np.abs(_h(rstd) - rstd64) <= _arith(d) * rstd64)
    bar = _arith(d) * ((np.abs(n64) + 2) * np.abs(_h(w)) + (0 if b is None else np.abs(_h(b))))
    assert np.all(np.abs(_h(y) - y64) <= bar + _half(bf16) * (np.abs(y64) + bar))


# rows on both sides of the switch to one wavefront a row (2048), lengths on both sides of every split of a row
SHAPES = [(1, 64), (1, 2048), (3, 4096), (5, 4160), (7, 8192), (2, 8256), (2, 65536), (257, 1088), (2047, 192),
          (2048, 512), (2049, 576), (2050, 1088), (2051, 2112), (2048, 4096), (2100, 4160)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(T, d, bf16):
    m = _moe()
    rng = np.random.default_rng(T * 7 + d)
    x, w, b = _rand(rng, T, d, bf16=bf16, mean=0.5), _rand(rng, d, bf16=bf16), _rand(rng, d, bf16=bf16)
    for res, bias in ((None, b), (_rand(rng, T, d, bf16=bf16, std=2.0), b), (None, None)):
        print(f"[ln] T={T} d={d} bf16={bf16} residual={res is not None} bias={bias is not None}", flush=True)
        _check_fwd(_fwd(m, x, res, w, bias, bf16), x, res, w, bias, bf16)


@pytest.mark.parametrize("T,d", [(5, 256), (2100, 512), (2, 16384)])
def test_rows_whose_mean_is_many_times_their_spread(T, d):
    m = _moe()
    rng = np.random.default_rng(T + d)
    w, b = _rand(rng, d, bf16=False), _rand(rng, d, bf16=False)
    for mean in (1e3, -1e5):
        x = _rand(rng, T, d, bf16=False, mean=mean)
        _check_fwd(_fwd(m, x, None, w, b, False), x, None, w, b, False)
    x = _rand(rng, T, d, bf16=False)
    x[:] = 1234.5678  # no spread at all: y is the bias
    y = _fwd(m, x, None, w, b, False)[1]
    # r - mean is at most half a step of the mean, times 1 / sqrt(eps)
    assert np.all(np.abs(_h(y) - _h(b)) <= 1234.6 * 2 * U / np.sqrt(EPS) * np.abs(_h(w)) + U * np.abs(_h(b)))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,d", [(6, 256), (2100, 512), (3, 16384)])
def test_rows_past_the_range_of_their_sums(T, d, bf16):
    """Rows up to fp32's largest values have the norm of any other row."""
    m = _moe()
    rng = np.random.default_rng(T + d + 1)
    w, b = _rand(rng, d, bf16=bf16), _rand(rng, d, bf16=bf16)
    for top in (2.0 ** 62, 2.0 ** 100, 2.0 ** 124):
        x = _rand(rng, T, d, bf16=bf16, mean=0.25) * top
        assert np.isfinite(_h(x)).all()
        _check_fwd(_fwd(m, x, None, w, b, bf16), x, None, w, b, bf16)
    x[:] = 2.0 ** 120  # no spread, sums past the range
    r, y, mean, rstd = _fwd(m, x, None, w, b, bf16, eps=1e-30)
    assert np.all(_h(y) == _h(b)) and np.all(_h(mean) == 2.0 ** 120)


def test_residual_in_place():
    import torch
    m = _moe()
    rng = np.random.default_rng(3)
    for T, d in ((5, 256), (3000, 512), (2, 16384)):
        x, res, w, b = _rand(rng, T, d), _rand(rng, T, d), _rand(rng, d), _rand(rng, d)
        r, y, _, _ = _fwd(m, x, res, w, b, True)
        r2, y2, _, _ = _fwd(m, x, res, w, b, True, r_alias=True)
        assert r2.data_ptr() == res.data_ptr() and torch.equal(r, r2) and torch.equal(y, y2)


def test_zero_and_non_finite_rows():
    """A zero row gives the bias; an infinity or NaN stays in its own row; rows behind the last are not written."""
    import torch
    m = _moe()
    rng = np.random.default_rng(4)
    for T in (9, 2500):
        x, w, b = _rand(rng, T, 512), _rand(rng, 512), _rand(rng, 512)
        clean = _fwd(m, x, None, w, b, True)[1].clone()
        x[2] = 0
        x[4, 77] = float("nan")
        x[6, 100] = float("inf")
        y = _fwd(m, x, None, w, b, True)[1]
        assert torch.equal(y[2], b) and torch.isnan(y[4]).all() and torch.isnan(y[6]).all()
        keep = [i for i in range(T) if i not in (2, 4, 6)]
        assert torch.equal(y[keep], clean[keep])
        y, mean, rstd = torch.full_like(x, 7.0), _nan(T), _nan(T)
        m.moe_layernorm_fwd(m.make_norm_shape(T - 3, 512, m.MOE_DTYPE_BF16, EPS), x, None, w, b, None, y, mean, rstd)
        torch.cuda.synchronize()
        assert (y[T - 3:] == 7).all() and torch.isnan(mean[T - 3:]).all() and torch.isnan(rstd[T - 3:]).all()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,d", SHAPES + [(8200, 128), (20011, 64)])
def test_backward(T, d, bf16):
    """dx per element: every term with the fp32 error of its own size, the two means' from a chain of d/64 + 16
    additions of signed terms; n from one fused multiply-add, off by a step of mean * rstd. dw, db: T / 512 + 1 rows of
    a workgroup at most, its 4 slots, 512 / 64 partial rows a thread, then 64 threads."""
    import torch
    m = _moe()
    rng = np.random.default_rng(T * 5 + d)
    r, w = _rand(rng, T, d, bf16=bf16, mean=0.5), _rand(rng, d, bf16=bf16)
    dy = _rand(rng, T, d, bf16=bf16, std=0.3)
    mean = np.mean(_h(r), axis=1).astype(np.float32)
    rstd = (1 / np.sqrt(np.var(_h(r), axis=1) + EPS)).astype(np.float32)
    mean_t, rstd_t = torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda()
    s = m.make_norm_shape(T, d, _dt(bf16), EPS, m.MOE_NORM_OVERWRITE_DW)
    acc = m.make_norm_shape(T, d, _dt(bf16), EPS)
    ws = torch.full((m.moe_layernorm_workspace_size(s),), 0xFF, dtype=torch.uint8, device="cuda")
    for dres in (None, _rand(rng, T, d, bf16=bf16, std=0.3)):
        print(f"[ln bwd] T={T} d={d} bf16={bf16} dres={dres is not None}", flush=True)
        dx, dw, db = torch.full_like(dy, float("nan")), _nan(d), _nan(d)
        m.moe_layernorm_bwd(s, dy, r, w, mean_t, rstd_t, dres, dx, dw, db, ws, ws.numel())
        dx64, dw64, db64 = oracle.layernorm_bwd(_h(dy), _h(r), _h(w), mean, rstd, None if dres is None else _h(dres))
        rs = rstd[:, None].astype(np.float64)
        n = np.abs((_h(r) - mean[:, None]) * rs) + np.abs(mean[:, None] * rs)
        g = np.abs(_h(dy) * _h(w))
        c = (d / 64 + 20) / 8
        terms = rs * (g + c * np.mean(g, axis=1, keepdims=True) + n * c * np.mean(g * n, axis=1, keepdims=True))
        terms = terms + (0 if dres is None else np.abs(_h(dres)))
        assert np.all(np.abs(_h(dx) - dx64) <= 8 * U * terms + _half(bf16) * np.abs(dx64))
        chain = T / 512 + 1 + 4 + 8 + 64 + 4
        assert np.all(np.abs(_h(dw) - dw64) <= chain * U * np.sum(np.abs(_h(dy)) * n, axis=0))
        assert np.all(np.abs(_h(db) - db64) <= chain * U * np.sum(np.abs(_h(dy)), axis=0))
        # accumulation, a repeat bit for bit, and dx in place of dy or dres; without db
        dw2, db2 = dw.clone(), db.clone()
        dx2 = dy.clone() if dres is None else dres.clone()
        m.moe_layernorm_bwd(acc, dx2 if dres is None else dy, r, w, mean_t, rstd_t, None if dres is None else dx2, dx2,
                            dw2, db2, ws, ws.numel())
        torch.cuda.synchronize()
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw + dw) and torch.equal(db2, db + db)
        dw3 = _nan(d)
        m.moe_layernorm_bwd(s, dy, r, w, mean_t, rstd_t, dres, dx2, dw3, None, ws, ws.numel())
        torch.cuda.synchronize()
        assert torch.equal(dw3, dw)


@pytest.mark.parametrize("T,d", [(5, 256), (300, 2112), (2100, 512), (2, 16384)])
def test_backward_of_rows_whose_mean_is_many_times_their_spread(T, d):
    """As test_backward, but with no term of the size of mean * rstd: r - mean of neighbours in fp32 is off by half a
    step of itself at most, so n by that, rstd's scaling and the product, 2 steps of n; the means and sums as there."""
    import torch
    m = _moe()
    rng = np.random.default_rng(T + 3 * d)
    w, dy = _rand(rng, d, bf16=False), _rand(rng, T, d, bf16=False, std=0.3)
    s = m.make_norm_shape(T, d, m.MOE_DTYPE_F32, EPS, m.MOE_NORM_OVERWRITE_DW)
    ws = torch.empty(m.moe_layernorm_workspace_size(s), dtype=torch.uint8, device="cuda")
    for at, sd in ((1e3, 1.0), (-1e5, 1.0), (1e3, 0.05), (0.25 * 2.0 ** 124, 2.0 ** 124)):
        r = _rand(rng, T, d, bf16=False, mean=at, std=sd)
        assert np.isfinite(_h(r)).all()
        mean = np.mean(_h(r), axis=1).astype(np.float32)
        rstd = (1 / np.sqrt(np.var(_h(r), axis=1) + EPS)).astype(np.float32)
        dx, dw, db = _nan(T, d), _nan(d), _nan(d)
        m.moe_layernorm_bwd(s, dy, r, w, torch.from_numpy(mean).cuda(), torch.from_numpy(rstd).cuda(), None, dx, dw, db,
                            ws, ws.numel())
        torch.cuda.synchronize()
        dx64, dw64, db64 = oracle.layernorm_bwd(_h(dy), _h(r), _h(w), mean, rstd)
        rs = rstd[:, None].astype(np.float64)
        n = np.abs(_h(r) - mean[:, None]) * rs
        g = np.abs(_h(dy) * _h(w))
        c = (d / 64 + 20) / 8
        terms = rs * (g + c * np.mean(g, axis=1, keepdims=True) + n * c * np.mean(g * n, axis=1, keepdims=True))
        tiny = 2.0 ** -149 * (2 if sd > 1 else 0)  # dx of rows past 2^120 are subnormal numbers
        assert np.all(np.abs(_h(dx) - dx64) <= 8 * U * terms + tiny)
        chain = T / 512 + 1 + 4 + 8 + 64 + 4
        assert np.all(np.abs(_h(dw) - dw64) <= chain * U * np.sum(np.abs(_h(dy)) * n, axis=0))
        assert np.all(np.abs(_h(db) - db64) <= chain * U * np.sum(np.abs(_h(dy)), axis=0))


def test_gradients_against_differences():
    """fp32, through the forward itself: differences of h = 1e-2 of a loss whose third derivatives are of order 1 are
    off by h^2 of it and by a few steps of y (2^-22) over h."""
    import torch
    m = _moe()
    rng = np.random.default_rng(8)
    T, d, h = 3, 64, 1e-2
    x, w, b = _rand(rng, T, d, bf16=False), _rand(rng, d, bf16=False), _rand(rng, d, bf16=False)
    dy = _rand(rng, T, d, bf16=False)
    _, _, mean, rstd = _fwd(m, x, None, w, b, False)
    dx, dw, db = _nan(T, d), _nan(d), _nan(d)
    s = m.make_norm_shape(T, d, m.MOE_DTYPE_F32, EPS, m.MOE_NORM_OVERWRITE_DW)
    ws = torch.empty(m.moe_layernorm_workspace_size(s), dtype=torch.uint8, device="cuda")
    m.moe_layernorm_bwd(s, dy, x, w, mean, rstd, None, dx, dw, db, ws, ws.numel())
    loss = lambda: float((_fwd(m, x, None, w, b, False)[1].double() * dy.double()).sum())  # noqa: E731
    size = float(dy.abs().sum())
    for got, v, at in ((dx, x, [(0, 0), (1, 17), (2, 63)]), (dw, w, [(5,), (40,)]), (db, b, [(6,), (63,)])):
        for i in at:
            old = float(v[i])
            v[i] = old + h
            hi, up = float(v[i]), loss()
            v[i] = old - h
            lo, down = float(v[i]), loss()
            v[i] = old
            want = (up - down) / (hi - lo)
            assert abs(float(got[i]) - want) <= 20 * h * h + size * 2.0 ** -22 / h


def test_backward_of_no_rows():
    import torch
    m = _moe()
    dw, db = torch.full((128,), 3.0, device="cuda"), torch.full((128,), 4.0, device="cuda")
    none = [None] * 7
    m.moe_layernorm_bwd(m.make_norm_shape(0, 128, m.MOE_DTYPE_BF16), *none, dw, db, None, 0)
    torch.cuda.synchronize()
    assert (dw == 3).all() and (db == 4).all()
    m.moe_layernorm_bwd(m.make_norm_shape(0, 128, m.MOE_DTYPE_BF16, EPS, m.MOE_NORM_OVERWRITE_DW), *none, dw, db, None, 0)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()
