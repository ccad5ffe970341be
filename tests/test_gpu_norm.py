"""The RMS norm (forward, 8-bit output, backward) and the 8-bit block form
against the fp64 oracle, through the C ABI.

Tolerances, per element and derived: u = 2^-24 is half an fp32 step. A row's
sum of squares is a chain of at most d/64 + 16 additions of terms with one
rounding each (a thread's own values, then the tree), all of one sign, so
rstd and y carry at most (d/64 + 24) u relative from fp32 arithmetic (the
square root halves the sum's share; division, root and two products add the
rest). A bf16 result adds 2^-8 relative, half its step, an fp32 one nothing.
"""
import numpy as np
import pytest

import oracle
from workloads import f32_to_bf16_bits, bf16_bits_to_f32

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


def _moe():
    import token_dispatch_grouped_amd as m
    return m


def _torch(bf16):
    import torch
    return torch.bfloat16 if bf16 else torch.float32


def _dt(bf16):
    m = _moe()
    return m.MOE_DTYPE_BF16 if bf16 else m.MOE_DTYPE_F32


def _rand(rng, *shape, bf16=True, std=1.0):
    import torch
    return torch.from_numpy(rng.normal(0, std, shape).astype(np.float32)).to(_torch(bf16)).cuda()


def _h(t):
    return t.double().cpu().numpy()


def _arith(d):
    return (d / 64 + 24) * U


def _half(bf16):
    return 2.0 ** -8 if bf16 else 0.0


def _values(q, scale):
    """float64 values and scales of the block form's bytes."""
    import torch
    v = q.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)
    S = np.ldexp(1.0, scale.cpu().numpy().astype(np.int64) - 127)
    return v, S


def _round_r(bf16):
    if bf16:
        return lambda v: bf16_bits_to_f32(f32_to_bf16_bits(v.astype(np.float32))).astype(np.float64)
    return lambda v: v.astype(np.float32).astype(np.float64)


def _check_mx8(q, scale, y64, rel):
    """The block form of values known to `rel`: each scale is the definition's for some value in reach, each element
    within half an e4m3 step (2^-4 relative, 2^-10 S below the normal range) of the true value."""
    v, S = _values(q, scale)
    n, m = y64.shape
    b = np.abs(y64).reshape(n, -1, 32)
    top = b.max(axis=2)
    ok = (top > 0) & (S > 2.0 ** -127)
    assert np.all(top[ok] * (1 - rel) <= 448 * S[ok]) and np.all(top[ok] * (1 + rel) >= 448 * S[ok] / 2)
    Sx = np.repeat(S, 32, axis=1)
    err = np.abs(v * Sx - y64)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(y64), 2.0 ** -10 * Sx) * (1 + 1e-9) + rel * np.abs(y64))


def _fwd(m, x, res, w, mx8, bf16, r_alias=False):
    import torch
    T, d = x.shape
    r = None if res is None else (res if r_alias else torch.full_like(x, float("nan")))
    rstd = torch.full((T,), float("nan"), device="cuda")
    if mx8:
        y = torch.full((T, d), 0xAA, dtype=torch.uint8, device="cuda")
        ys = torch.full((T, d // 32), 0xAA, dtype=torch.uint8, device="cuda")
    else:
        y, ys = torch.full_like(x, float("nan")), None
    m.moe_rmsnorm_fwd(m.make_norm_shape(T, d, _dt(bf16), EPS), x, res, w, r, y, ys, rstd)
    torch.cuda.synchronize()
    return r, y, ys, rstd


# rows on both sides of the switch to one wavefront a row (2048), lengths on both sides of every split of a row:
# 16-byte chunks of 8 bf16 / 4 fp32 values, 64 or 256 threads, 1, 2, 4 (8) chunks a thread, and longer rows
SHAPES = [(1, 64), (1, 2048), (3, 4096), (5, 4160), (7, 8192), (2, 8256), (2, 65536), (257, 1088), (2047, 192),
          (2048, 512), (2049, 576), (2050, 1088), (2051, 2112), (2048, 4096), (2100, 4160)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(T, d, bf16):
    m = _moe()
    rng = np.random.default_rng(T * 7 + d)
    x, w = _rand(rng, T, d, bf16=bf16), _rand(rng, d, bf16=bf16)
    for res in (None, _rand(rng, T, d, bf16=bf16, std=2.0)):
        r64, rstd64, y64 = oracle.rmsnorm_fwd(_h(x), _h(w), EPS, None if res is None else _h(res), _round_r(bf16))
        print(f"[norm] T={T} d={d} bf16={bf16} residual={res is not None}", flush=True)
        r, y, _, rstd = _fwd(m, x, res, w, False, bf16)
        if res is not None:
            assert np.array_equal(_h(r), r64)  # one correctly rounded addition
        assert np.all(np.abs(_h(rstd) - rstd64) <= _arith(d) * rstd64)
        assert np.all(np.abs(_h(y) - y64) <= (_arith(d) + _half(bf16)) * np.abs(y64))
        r2, q, s, rstd2 = _fwd(m, x, res, w, True, bf16)
        assert np.array_equal(_h(rstd2), _h(rstd))
        _check_mx8(q, s, y64, _arith(d))


def test_residual_in_place():
    m = _moe()
    rng = np.random.default_rng(3)
    for T, d in ((5, 256), (3000, 512), (2, 16384)):
        x, res, w = _rand(rng, T, d), _rand(rng, T, d), _rand(rng, d)
        r, y, _, _ = _fwd(m, x, res, w, False, True)
        r2, y2, _, _ = _fwd(m, x, res, w, False, True, r_alias=True)
        import torch
        assert r2.data_ptr() == res.data_ptr() and torch.equal(r, r2) and torch.equal(y, y2)


def test_zero_and_non_finite_rows():
    """A zero row gives zeros (eps > 0); an infinity or NaN stays in its own row."""
    import torch
    m = _moe()
    rng = np.random.default_rng(4)
    for T in (9, 2500):
        x, w = _rand(rng, T, 512), _rand(rng, 512)
        clean = _fwd(m, x, None, w, False, True)[1].clone()
        x[2] = 0
        x[4, 77] = float("nan")
        x[6, 100] = float("inf")
        y = _fwd(m, x, None, w, False, True)[1]
        assert torch.count_nonzero(y[2]) == 0 and torch.isnan(y[4]).all() and torch.isnan(y[6, 100])
        keep = [i for i in range(T) if i not in (2, 4, 6)]
        assert torch.equal(y[keep], clean[keep])
        q, s = _fwd(m, x, None, w, True, True)[1:3]
        # zeros of either sign: 0 * w is -0 (byte 0x80) where w < 0
        assert not (q[2] & 0x7F).any() and not s[2].any()
        assert (s[4] == 255).all() and ((q[4] & 0x7F) == 0x7F).all()
        assert (s[0] < 255).all()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,d", SHAPES + [(8200, 128), (20011, 64)])
def test_backward(T, d, bf16):
    """dx per element: every term of rstd (g - n mean(g n)) + dres with the fp32 error of its own size, the mean's
    from a chain of d/64 + 16 additions of signed terms; dw: T / 512 + 1 rows of a workgroup of at most 512 at most, its 4
    slots, 512 / 64 partial rows a thread, then 64 threads."""
    import torch
    m = _moe()
    rng = np.random.default_rng(T * 5 + d)
    r, w = _rand(rng, T, d, bf16=bf16), _rand(rng, d, bf16=bf16)
    dy = _rand(rng, T, d, bf16=bf16, std=0.3)
    rstd = (1 / np.sqrt(np.mean(_h(r) ** 2, axis=1) + EPS)).astype(np.float32)
    rstd_t = torch.from_numpy(rstd).cuda()
    s = m.make_norm_shape(T, d, _dt(bf16), EPS, m.MOE_NORM_OVERWRITE_DW)
    acc = m.make_norm_shape(T, d, _dt(bf16), EPS)
    ws = torch.full((m.moe_rmsnorm_workspace_size(s),), 0xFF, dtype=torch.uint8, device="cuda")
    for dres in (None, _rand(rng, T, d, bf16=bf16, std=0.3)):
        print(f"[norm bwd] T={T} d={d} bf16={bf16} dres={dres is not None}", flush=True)
        dx = torch.full_like(dy, float("nan"))
        dw = torch.full((d,), float("nan"), device="cuda")
        m.moe_rmsnorm_bwd(s, dy, r, w, rstd_t, dres, dx, dw, ws, ws.numel())
        dx64, dw64 = oracle.rmsnorm_bwd(_h(dy), _h(r), _h(w), rstd, None if dres is None else _h(dres))
        n = np.abs(_h(r) * rstd[:, None].astype(np.float64))
        g = np.abs(_h(dy) * _h(w))
        terms = rstd[:, None] * (g + n * np.mean(g * n, axis=1, keepdims=True) * (d / 64 + 20) / 8)
        terms = terms + (0 if dres is None else np.abs(_h(dres)))
        assert np.all(np.abs(_h(dx) - dx64) <= 8 * U * terms + _half(bf16) * np.abs(dx64))
        chain = T / 512 + 1 + 4 + 8 + 64 + 4
        bar = chain * U * np.sum(np.abs(_h(dy)) * n, axis=0)
        assert np.all(np.abs(_h(dw) - dw64) <= bar)
        # accumulation, a repeat bit for bit, and dx in place of dy or dres
        dw2 = dw.clone()
        dx2 = dy.clone() if dres is None else dres.clone()
        m.moe_rmsnorm_bwd(acc, dx2 if dres is None else dy, r, w, rstd_t, None if dres is None else dx2, dx2, dw2, ws,
                          ws.numel())
        torch.cuda.synchronize()
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw + dw)


def test_backward_of_no_rows():
    import torch
    m = _moe()
    dw = torch.full((128,), 3.0, device="cuda")
    m.moe_rmsnorm_bwd(m.make_norm_shape(0, 128, m.MOE_DTYPE_BF16), None, None, None, None, None, None, dw, None, 0)
    torch.cuda.synchronize()
    assert (dw == 3).all()
    m.moe_rmsnorm_bwd(m.make_norm_shape(0, 128, m.MOE_DTYPE_BF16, EPS, m.MOE_NORM_OVERWRITE_DW), None, None, None,
                      None, None, None, dw, None, 0)
    torch.cuda.synchronize()
    assert (dw == 0).all()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 64), (3, 128), (129, 1088), (1000, 4096), (2, 65536)])
def test_quantize_is_exact(rows, cols, bf16):
    """Scaling by a power of two is exact, so scales and elements equal the oracle's."""
    import torch
    m = _moe()
    rng = np.random.default_rng(rows + cols)
    x = _rand(rng, rows, cols, bf16=bf16)
    x = x * torch.exp2(torch.from_numpy(rng.integers(-40, 40, (rows, cols // 32)).astype(np.float32)).cuda()
                       .repeat_interleave(32, dim=1)).to(x.dtype)
    x[0, :32] = 0
    x[-1, -32:] = 448.0
    x[-1, -33] = 450.0
    q = torch.full((rows, cols), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, cols // 32), 0xAA, dtype=torch.uint8, device="cuda")
    m.moe_mx8_quantize(rows, cols, _dt(bf16), x, q, s)
    v, S = _values(q, s)
    q64, S64 = oracle.mx8_quantize(_h(x))
    assert np.array_equal(S, S64) and np.array_equal(v, q64)


def test_quantize_denormal_and_non_finite_blocks():
    import torch
    m = _moe()
    x = torch.zeros(4, 64, device="cuda")
    x[0, 0] = 1e-42
    x[1, 5] = float("inf")
    x[2, 40] = float("nan")
    x[3] = 3e38
    q = torch.empty(4, 64, dtype=torch.uint8, device="cuda")
    s = torch.empty(4, 2, dtype=torch.uint8, device="cuda")
    m.moe_mx8_quantize(4, 64, m.MOE_DTYPE_F32, x, q, s)
    torch.cuda.synchronize()
    assert s.tolist()[0] == [0, 0] and not q[0].any()  # 1e-42 * 2^127 is below half of e4m3's smallest step
    assert s.tolist()[1] == [255, 0] and ((q[1, :32] & 0x7F) == 0x7F).all() and not q[1, 32:].any()
    assert s.tolist()[2] == [0, 255]
    v, S = _values(q[3:], s[3:])
    assert np.all(np.abs(v * np.repeat(S, 32, axis=1) - float(np.float32(3e38))) <= 2.0 ** -4 * 3e38)
