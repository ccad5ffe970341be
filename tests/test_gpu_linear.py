"""The dense product with bias, activation and residual and its gradients
against the fp64 oracle, through the C ABI.

Tolerances, per element and derived. A product of K terms accumulated in fp32
is off by at most K 2^-23 sum|terms| (one rounding of at most a whole step a
term, the bias one more), which a slope of at most 1.13 carries through the
activation. The activation itself is computed to 2^-15 of its value (the
hardware's exponential and reciprocal, the exponent's argument off by 3 half
steps of at most 88) and, for gelu, to 2^-23 |z| (erf to 1.5e-7, halved). A bf16
result adds half its step, 2^-8 relative. Slopes are at most 1.13 and off by at
most 2^-14.
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23
HALF = 2.0 ** -8
SLOPE = 1.13
ACTS = oracle.ACTS


def _moe():
    import token_dispatch_grouped_amd as m
    return m


def _rand(rng, *shape, std=1.0):
    import torch
    return torch.from_numpy(rng.normal(0, std, shape).astype(np.float32)).bfloat16().cuda()


def _h(t):
    return t.double().cpu().numpy()


def _nan(*shape, dtype=None):
    import torch
    return torch.full(shape, float("nan"), dtype=dtype or torch.bfloat16, device="cuda")


def _bits(t):
    import torch
    return t.view(torch.int16)


def _near(got, want, tol, what):
    over = np.abs(got - want) - tol
    i = np.unravel_index(np.argmax(np.where(np.isnan(over), np.inf, over)), over.shape)
    assert over[i] <= 0, f"{what}{list(i)}: {got[i]!r} is not {want[i]!r} within {tol[i]:.3e}"


# one token, the few-row kernels' steps, tiles with ragged rows and columns, every tile shape, several rounds of the
# large tiles and a rest
SHAPES = [(1, 64, 64), (1, 2048, 1408), (2, 64, 192), (16, 128, 128), (17, 256, 320), (33, 1024, 704), (48, 320, 1472),
          (64, 512, 256), (65, 576, 128), (144, 128, 320), (145, 192, 448), (300, 1088, 576), (700, 1088, 576),
          (1000, 1984, 1408), (1300, 512, 1408), (1400, 320, 2048), (4200, 128, 2048), (9000, 1088, 320), (5000, 64, 4160),
          (65600, 128, 256)]


@pytest.mark.parametrize("T,K,N", SHAPES)
def test_forward(T, K, N):
    import torch
    m = _moe()
    rng = np.random.default_rng(T + K + N)
    x, w = _rand(rng, T, K), _rand(rng, N, K, std=2 * K ** -0.5)
    b, res = _rand(rng, N), _rand(rng, T, N)
    prod = _h(x) @ _h(w).T
    size = np.abs(_h(x)) @ np.abs(_h(w)).T
    acts = ACTS if T <= 5000 else ACTS[2:3]
    for i, act in enumerate(acts):
        print(f"[linear] T={T} K={K} N={N} {act}", flush=True)
        bias, r = (b if i % 2 == 0 else None), (res if i % 3 == 0 else None)
        s = m.make_linear_shape(T, K, N, act=ACTS.index(act))
        z, y = _nan(T, N), _nan(T, N)
        m.moe_linear_fwd(s, x, w, bias, r, z, y)
        z64 = prod if bias is None else prod + _h(bias)
        dz = (K + 1) * STEP * (size if bias is None else size + np.abs(_h(bias)))
        _near(_h(z), z64, dz + HALF * (np.abs(z64) + dz), "z")
        v64 = oracle.act(act, z64)
        dv = SLOPE * dz + (0 if act in ("none", "relu") else 2.0 ** -15 * np.abs(v64) + STEP * np.abs(z64))
        y64 = v64 if r is None else v64 + _h(r)
        dv = dv + STEP * np.abs(y64)
        _near(_h(y), y64, dv + HALF * (np.abs(y64) + dv), "y")
        # without z, and into the residual: the same bits
        y2 = _nan(T, N) if r is None else r.clone()
        m.moe_linear_fwd(s, x, w, bias, None if r is None else y2, None, y2)
        assert torch.equal(_bits(y2), _bits(y))


@pytest.mark.parametrize("T,K,N", SHAPES)
def test_dgrad(T, K, N):
    import torch
    m = _moe()
    rng = np.random.default_rng(T + K + N + 1)
    dz, w = _rand(rng, T, N, std=0.3), _rand(rng, N, K, std=N ** -0.5)
    zin, add = _rand(rng, T, K, std=2.0), _rand(rng, T, K)
    prod = _h(dz) @ _h(w)
    dp = N * STEP * (np.abs(_h(dz)) @ np.abs(_h(w)))
    s = m.make_linear_shape(T, K, N)
    acts = ACTS if T <= 5000 else ACTS[2:3]
    for i, act in enumerate(acts):
        print(f"[linear dgrad] T={T} K={K} N={N} {act}", flush=True)
        z = zin if act != "none" else None
        a = add if i % 2 == 0 else None
        dx = _nan(T, K)
        m.moe_linear_dgrad(s, dz, w, z, ACTS.index(act), a, dx)
        slope = oracle.act_slope(act, _h(zin))
        dx64 = prod * slope
        tol = SLOPE * dp + (0 if act in ("none", "relu") else 2.0 ** -14 * np.abs(prod))
        if a is not None:
            dx64 = dx64 + _h(a)
        tol = tol + STEP * np.abs(dx64)
        _near(_h(dx), dx64, tol + HALF * (np.abs(dx64) + tol), "dx")
        # in place of the addend, and in place of z_in: the same bits
        if a is not None:
            dx2 = a.clone()
            m.moe_linear_dgrad(s, dz, w, z, ACTS.index(act), dx2, dx2)
            assert torch.equal(_bits(dx2), _bits(dx))
        if z is not None:
            dx2 = z.clone()
            m.moe_linear_dgrad(s, dz, w, dx2, ACTS.index(act), a, dx2)
            assert torch.equal(_bits(dx2), _bits(dx))


# few columns: the sum in eight runs, many rows of workgroups, with 1, 2 and 3 groups of 16 tokens each
@pytest.mark.parametrize("T,K,N", [(145, 2048, 512), (1000, 512, 128), (3001, 64, 64), (700, 4096, 256), (2500, 1088, 64),
                                   (333, 65536, 64), (257, 320, 192), (192, 2048, 2048), (384, 576, 1024), (1400, 4096, 256)])
def test_forward_of_few_columns(T, K, N):
    test_forward(T, K, N)


# few tokens: 32 and 64 columns a workgroup with 1, 2 and 3 groups of 16 tokens, sums shorter than the wavefronts share
@pytest.mark.parametrize("T,K,N", [(5, 16384, 128), (20, 8256, 64), (40, 8256, 192), (100, 4096, 320), (48, 8192, 128),
                                   (17, 1024, 8192), (144, 65536, 64), (1, 64, 65536), (80, 2048, 1088), (16, 512, 2048)])
def test_dgrad_of_few_tokens(T, K, N):
    test_dgrad(T, K, N)


@pytest.mark.parametrize("T,K,N", SHAPES + [(20011, 128, 192), (32768, 320, 512), (3000, 2048, 2048), (700, 8192, 2048)])
def test_wgrad(T, K, N):
    """Sums over T tokens in fp32: T 2^-23 sum|terms|. Added to a gradient already there, slice by slice: the first sum's
    error, the second's, and half a step of a value of up to twice sum|terms| for each slice, of which there are fewer
    than T."""
    import torch
    m = _moe()
    rng = np.random.default_rng(T + K + N + 2)
    dz, x = _rand(rng, T, N, std=0.3), _rand(rng, T, K)
    s = m.make_linear_shape(T, K, N, flags=m.MOE_LINEAR_OVERWRITE_DW)
    acc = m.make_linear_shape(T, K, N)
    ws = torch.full((max(1, m.moe_linear_workspace_size(s)),), 0xFF, dtype=torch.uint8, device="cuda")
    dw, db = _nan(N, K, dtype=torch.float32), _nan(N, dtype=torch.float32)
    print(f"[linear wgrad] T={T} K={K} N={N}", flush=True)
    m.moe_linear_wgrad(s, dz, x, dw, db, ws, ws.numel())
    d64, x64 = dz.double(), x.double()
    dw64, bar = _h(d64.t() @ x64), _h(T * STEP * (d64.abs().t() @ x64.abs()))
    _near(_h(dw), dw64, bar, "dw")
    _near(_h(db), _h(d64.sum(0)), _h(T * STEP * d64.abs().sum(0)), "db")
    sums = []
    for _ in range(2):
        sums.append((dw.clone(), db.clone()))
        m.moe_linear_wgrad(acc, dz, x, *sums[-1], ws, ws.numel())
    _near(_h(sums[0][0]), 2 * dw64, 3 * bar, "dw added")
    assert torch.equal(sums[0][0], sums[1][0]) and torch.equal(sums[0][1], sums[1][1])
    assert torch.equal(sums[0][1], db + db)
    dw3 = _nan(N, K, dtype=torch.float32)
    m.moe_linear_wgrad(s, dz, x, dw3, None, ws, ws.numel())
    assert torch.equal(dw3, dw)


@pytest.mark.parametrize("act", ACTS[1:])
def test_dact(act):
    import torch
    m = _moe()
    rng = np.random.default_rng(7)
    for T, N in ((1, 64), (37, 192), (2000, 1088)):
        dy, z = _rand(rng, T, N), _rand(rng, T, N, std=3.0)
        s = m.make_linear_shape(T, 64, N, act=ACTS.index(act))
        dz = _nan(T, N)
        m.moe_linear_dact(s, dy, z, dz)
        want = _h(dy) * oracle.act_slope(act, _h(z))
        _near(_h(dz), want, 2.0 ** -14 * np.abs(_h(dy)) + HALF * np.abs(want), "dz")
        for alias in (dy.clone(), z.clone()):
            m.moe_linear_dact(s, alias if torch.equal(alias, dy) else dy, z if torch.equal(alias, dy) else alias, alias)
            assert torch.equal(_bits(alias), _bits(dz))


@pytest.mark.parametrize("act", ACTS)
def test_activations_far_out_and_not_finite(act):
    """x = 1 in one place and w diagonal: z is any value wanted. Tails to 2^-8 of themselves, no NaN from large values;
    an infinity or NaN stays in its row."""
    import torch
    m = _moe()
    vals = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 0.75, -0.75, 2.0, -2.0, -3.0, -4.0, -5.0, 5.0, 30.0, -30.0,
                         300.0, -300.0, 1e10, -1e10, 1e19, -1e19, 3e38, -3e38], device="cuda").bfloat16()
    for T in (3, 400):
        x = torch.zeros(T, 64, device="cuda").bfloat16()
        x[:, 0] = 1.0
        w = torch.zeros(64, 64, device="cuda").bfloat16()
        w[:len(vals), 0] = vals
        s = m.make_linear_shape(T, 64, 64, act=ACTS.index(act))
        y = _nan(T, 64)
        m.moe_linear_fwd(s, x, w, None, None, None, y)
        want = oracle.act(act, _h(vals))
        got = _h(y[T - 1, :len(vals)])
        rel = HALF + (2.0 ** -11 if act == "gelu" else 2.0 ** -14)  # gelu's tail: 2e-4 of itself to z = -5
        assert np.all(np.abs(got - want) <= rel * np.abs(want) + 1e-37), (got, want)
        slope = _nan(T, 64)
        zin = w[:, 0].repeat(T, 1).contiguous()
        eye = torch.eye(64, device="cuda").bfloat16()
        m.moe_linear_dgrad(m.make_linear_shape(T, 64, 64), torch.ones(T, 64, device="cuda").bfloat16(), eye,
                           None if act == "none" else zin, ACTS.index(act), None, slope)
        want = oracle.act_slope(act, _h(vals))
        assert np.all(np.abs(_h(slope[T - 1, :len(vals)]) - want) <= HALF * np.abs(want) + 2.0 ** -14)
        x[1, 5] = float("nan")
        w[:, 5] = 1.0
        y2 = _nan(T, 64)
        m.moe_linear_fwd(s, x, w, None, None, None, y2)
        torch.cuda.synchronize()
        keep = [i for i in range(T) if i != 1]
        assert torch.equal(_bits(y2[keep]), _bits(y[keep])) and torch.isnan(y2[1]).all()


def test_rows_behind_the_last_token():
    """A padded batch: rows past T are neither read into anything nor written."""
    import torch
    m = _moe()
    rng = np.random.default_rng(9)
    for T, K, N in ((5, 128, 192), (333, 192, 448), (5000, 128, 2048)):
        x, w, b, dz = _rand(rng, T + 70, K), _rand(rng, N, K, std=K ** -0.5), _rand(rng, N), _rand(rng, T + 70, N)
        res = _rand(rng, T + 70, N)
        s = m.make_linear_shape(T, K, N, act=m.MOE_ACT_SILU, flags=m.MOE_LINEAR_OVERWRITE_DW)
        ws = torch.empty(max(1, m.moe_linear_workspace_size(s)), dtype=torch.uint8, device="cuda")

        def all_calls():
            z, y, dx = (torch.full((T + 70, c), 7.0, device="cuda").bfloat16() for c in (N, N, K))
            dw, db = _nan(N, K, dtype=torch.float32), _nan(N, dtype=torch.float32)
            m.moe_linear_fwd(s, x, w, b, res, z, y)
            m.moe_linear_dgrad(s, dz, w, None, m.MOE_ACT_NONE, None, dx)
            m.moe_linear_wgrad(s, dz, x, dw, db, ws, ws.numel())
            torch.cuda.synchronize()
            for t in (z, y, dx):
                assert (t[T:] == 7).all()
            return z, y, dx, dw, db
        first = all_calls()
        for t in (x, dz, res):
            t[T:] = float("nan")
        for a, c in zip(first, all_calls()):
            assert torch.equal(a, c)


def test_empty_batches():
    import torch
    m = _moe()
    dw, db = torch.full((64, 128), 3.0, device="cuda"), torch.full((64,), 4.0, device="cuda")
    m.moe_linear_wgrad(m.make_linear_shape(0, 128, 64), None, None, dw, db, None, 0)
    torch.cuda.synchronize()
    assert (dw == 3).all() and (db == 4).all()
    m.moe_linear_wgrad(m.make_linear_shape(0, 128, 64, flags=m.MOE_LINEAR_OVERWRITE_DW), None, None, dw, db, None, 0)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()


def test_offsets_past_32_bits():
    """More than 2^31 elements on either side of the product, rows checked on both ends."""
    import torch
    m = _moe()
    T, K, N = 40000, 64, 65536
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(N, K, generator=gen, device="cuda") / 8).bfloat16()
    b = torch.randn(N, generator=gen, device="cuda").bfloat16()
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    print("[linear] more than 2^31 elements", flush=True)
    m.moe_linear_fwd(m.make_linear_shape(T, K, N, act=m.MOE_ACT_RELU), x, w, b, None, None, y)
    rows = [0, 17, 32767, 32768, 32769, T - 1]
    z64 = _h(x[rows]) @ _h(w).T + _h(b)
    tol = (K + 1) * STEP * (np.abs(_h(x[rows])) @ np.abs(_h(w)).T + np.abs(_h(b)))
    _near(_h(y[rows]), np.maximum(z64, 0), tol + HALF * (np.abs(z64) + tol), "y")
    dx = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    m.moe_linear_dgrad(m.make_linear_shape(T, K, N), y, w, None, m.MOE_ACT_NONE, None, dx)
    want = _h(y[rows]) @ _h(w)
    tol = N * STEP * (np.abs(_h(y[rows])) @ np.abs(_h(w)))
    _near(_h(dx[rows]), want, tol + HALF * (np.abs(want) + tol), "dx")
    s = m.make_linear_shape(T, K, N, flags=m.MOE_LINEAR_OVERWRITE_DW)
    ws = torch.empty(max(1, m.moe_linear_workspace_size(s)), dtype=torch.uint8, device="cuda")
    dw, db = _nan(N, K, dtype=torch.float32), _nan(N, dtype=torch.float32)
    m.moe_linear_wgrad(s, y, x, dw, db, ws, ws.numel())
    cols = [0, 1, 32768, N - 1]
    yc = y[:, cols].double()
    _near(_h(dw[cols]), _h(yc.t() @ x.double()), _h(T * STEP * (yc.abs().t() @ x.double().abs())), "dw")
    _near(_h(db[cols]), _h(yc.sum(0)), _h(T * STEP * yc.abs().sum(0)), "db")


def test_gelu_tail_keeps_its_digits():
    """gelu and its slope down the tail, where the values are far below any absolute error: 2^-16 of the value (the fit's
    4e-6 and the exponent's argument, off by 2 half steps of at most 85) and half a step of bf16. The slope Phi + z phi
    is a difference of up to z^2 times its size, -z phi / (z phi + Phi) >= 1 - 1 / z^2 of the terms."""
    import torch
    m = _moe()
    z = torch.linspace(-12.75, -1.5, 64 * 8, device="cuda").bfloat16().reshape(8, 64)
    z64 = _h(z)
    x = torch.zeros(8, 64, device="cuda").bfloat16()
    one = torch.ones(8, 64, device="cuda").bfloat16()
    dz = _nan(8, 64)
    m.moe_linear_dact(m.make_linear_shape(8, 64, 64, act=ACTS.index("gelu")), one, z, dz)
    want = oracle.act_slope("gelu", z64)
    phi, cdf = np.exp(-z64 ** 2 / 2) / np.sqrt(2 * np.pi), oracle.act("gelu", z64) / z64
    _near(_h(dz), want, 2.0 ** -15 * (np.abs(z64) * phi + cdf) + HALF * np.abs(want), "slope")
    for row in range(8):
        x[:, 0] = 1.0
        w = torch.zeros(64, 64, device="cuda").bfloat16()
        w[:, 0] = z[row]
        y = _nan(8, 64)
        m.moe_linear_fwd(m.make_linear_shape(8, 64, 64, act=ACTS.index("gelu")), x, w, None, None, None, y)
        want = oracle.act("gelu", z64[row])
        _near(_h(y[3]), want, 1.01 * 2.0 ** -16 * np.abs(want) + HALF * np.abs(want), "gelu")
