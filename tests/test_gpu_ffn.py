"""The dense gated feed-forward block (bf16 and 8-bit forward, gradients of
the input and of the weights) against the fp64 oracle, through the C ABI.

Tolerances, per element and derived. A product of K terms accumulated in fp32
is off by at most K 2^-23 sum|terms| (one rounding of at most a whole step a
term); a bf16 result adds half its step, 2^-8 relative. silu' is at most 1.1
and the device's sigmoid is taken to 2^-18 relative, so a = silu(g) u is off
by 1.1 |u| dg + |silu(g)| du + 2^-18 |a| + 2^-8 |a|. The second product is
compared on the a (or dh) that the first one wrote.

8-bit products: the scaled matrix instruction adds the 32 products of a block
aligned to the largest of them, and what lies below 2^-13 of it is cut off
(1 + 2^-13 keeps its second term, 1 + 2^-14 does not), so a block's sum is off
by at most 32 * 2^-13 max|product|, and max|product| is at most the product of
the two blocks' largest values. Sums over blocks are fp32 sums as above.
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -23
HALF = 2.0 ** -8   # half a bf16 step
SIG = 2.0 ** -18


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


def _ws(n):
    import torch
    return torch.full((max(1, n),), 0xFF, dtype=torch.uint8, device="cuda")


def _bits(t):
    import torch
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def _sig(z):
    return 0.5 * (1.0 + np.tanh(0.5 * z))


def _near(got, want, tol, what):
    over = np.abs(got - want) - tol
    i = np.unravel_index(np.argmax(np.where(np.isnan(over), np.inf, over)), over.shape)
    assert over[i] <= 0, f"{what}{list(i)}: {got[i]!r} is not {want[i]!r} within {tol[i]:.3e}"


def _weights(rng, d, F):
    return _rand(rng, 2 * F, d, std=d ** -0.5), _rand(rng, d, F, std=F ** -0.5)


# one token, the few-row kernels' steps, tiles with ragged rows and columns, more row tiles than a group
SHAPES = [(1, 64, 64), (1, 2048, 1408), (2, 64, 192), (15, 192, 64), (16, 128, 128), (17, 256, 320), (33, 1024, 704),
          (48, 320, 1472), (64, 512, 256), (65, 576, 128), (144, 128, 320), (145, 192, 448), (300, 1088, 576), (500, 704, 1024),
          (700, 1088, 576), (1000, 1984, 1408),
          (1300, 512, 1408)]
# enough tiles for the 256 x 256 tile in the products with N = d, in those with N = F, and several rounds of it
LARGE = [(4200, 2048, 128), (6001, 128, 1472), (9000, 320, 1088)]
# two groups of wavefronts a 128 x 128 tile in each product; a few rows more than whole rounds of the 256 x 256 tile
LARGE += [(1400, 1472, 320), (1500, 256, 1472), (65793, 256, 128), (65793, 128, 256), (65600, 256, 128)]


@pytest.mark.parametrize("T,d,F", SHAPES + LARGE)
def test_forward(T, d, F):
    import torch
    m = _moe()
    rng = np.random.default_rng(T + d + F)
    x, (wgu, wdn), add = _rand(rng, T, d), _weights(rng, d, F), _rand(rng, T, d)
    s = m.make_ffn_shape(T, d, F)
    fwd, _ = m.moe_ffn_workspace_size(s)
    h64, a64, _ = oracle.dense_ffn_fwd(_h(x), _h(wgu), _h(wdn))
    dh = d * STEP * (np.abs(_h(x)) @ np.abs(_h(wgu)).T)
    g, u = h64[:, :F], h64[:, F:]
    print(f"[ffn] T={T} d={d} F={F}", flush=True)
    h, a, y = _nan(T, 2 * F), _nan(T, F), _nan(T, d)
    m.moe_ffn_fwd(s, x, None, wgu, None, wdn, None, add, h, a, y, None, 0)
    _near(_h(h), h64, dh + HALF * (np.abs(h64) + dh), "h")
    da = 1.1 * np.abs(u) * dh[:, :F] + np.abs(g * _sig(g)) * dh[:, F:] + 1.1 * dh[:, :F] * dh[:, F:]
    da = da + (SIG + HALF) * (np.abs(a64) + da)
    _near(_h(a), a64, da, "a")
    y64 = _h(a) @ _h(wdn).T + _h(add)
    dy = (F + 1) * STEP * (np.abs(_h(a)) @ np.abs(_h(wdn)).T + np.abs(_h(add)))
    _near(_h(y), y64, dy + HALF * (np.abs(y64) + dy), "y")
    # without h and a, and with the sum in place of add: the same bits; without add
    ws = _ws(fwd)
    y2 = add.clone()
    m.moe_ffn_fwd(s, x, None, wgu, None, wdn, None, y2, None, None, y2, ws, ws.numel())
    assert torch.equal(_bits(y2), _bits(y))
    assert torch.equal(_bits(ws[:T * F * 2].view(torch.bfloat16).view(T, F)), _bits(a))
    y3 = _nan(T, d)
    m.moe_ffn_fwd(s, x, None, wgu, None, wdn, None, None, None, None, y3, ws, ws.numel())
    y64 = _h(a) @ _h(wdn).T
    _near(_h(y3), y64, dy + HALF * (np.abs(y64) + dy), "y3")


@pytest.mark.parametrize("T,d,F", SHAPES + LARGE)
def test_dgrad(T, d, F):
    import torch
    m = _moe()
    rng = np.random.default_rng(T + d + F + 1)
    dy, h, add = _rand(rng, T, d), _rand(rng, T, 2 * F), _rand(rng, T, d)
    wgu, wdn = _weights(rng, d, F)
    s = m.make_ffn_shape(T, d, F)
    print(f"[ffn dgrad] T={T} d={d} F={F}", flush=True)
    dh, dx = _nan(T, 2 * F), _nan(T, d)
    m.moe_ffn_dgrad(s, dy, h, wgu, wdn, add, dh, dx)
    da64, dh64, _ = oracle.dense_ffn_dgrad(_h(dy), _h(h), _h(wgu), _h(wdn))
    dda = d * STEP * (np.abs(_h(dy)) @ np.abs(_h(wdn)))
    g, u = _h(h)[:, :F], _h(h)[:, F:]
    sg = _sig(g)
    # |d silu| <= 1.1; the two terms of dh_gate carry the sigmoid's error each, the second with |g|
    tol_g = np.abs(u) * (1.1 * dda + np.abs(da64) * sg * (1 + np.abs(g)) * (3 * SIG))
    tol_u = np.abs(g) * sg * (dda + 2 * SIG * np.abs(da64))
    tol = np.concatenate([tol_g, tol_u], axis=1)
    _near(_h(dh), dh64, tol + HALF * (np.abs(dh64) + tol), "dh")
    dx64 = _h(dh) @ _h(wgu) + _h(add)
    tol = (2 * F + 1) * STEP * (np.abs(_h(dh)) @ np.abs(_h(wgu)) + np.abs(_h(add)))
    _near(_h(dx), dx64, tol + HALF * (np.abs(dx64) + tol), "dx")
    dx2, dh2 = add.clone(), _nan(T, 2 * F)
    m.moe_ffn_dgrad(s, dy, h, wgu, wdn, dx2, dh2, dx2)
    assert torch.equal(_bits(dx2), _bits(dx)) and torch.equal(_bits(dh2), _bits(dh))
    m.moe_ffn_dgrad(s, dy, h, wgu, wdn, None, dh2, dx2)
    dx64 = _h(dh) @ _h(wgu)
    _near(_h(dx2), dx64, tol + HALF * (np.abs(dx64) + tol), "dx2")


@pytest.mark.parametrize("T,d,F", SHAPES + [(2600, 64, 64), (5003, 128, 192), (4096, 320, 64)])
def test_wgrad(T, d, F):
    import torch
    m = _moe()
    rng = np.random.default_rng(T + d + F + 2)
    dy, x, a, dh = _rand(rng, T, d), _rand(rng, T, d), _rand(rng, T, F), _rand(rng, T, 2 * F)
    s = m.make_ffn_shape(T, d, F, m.MOE_DTYPE_BF16, m.MOE_FFN_OVERWRITE_DW)
    _, n = m.moe_ffn_workspace_size(s)
    ws = _ws(n)
    f32 = torch.float32
    dgu, ddn = _nan(2 * F, d, dtype=f32), _nan(d, F, dtype=f32)
    print(f"[ffn wgrad] T={T} d={d} F={F} ws={n}", flush=True)
    m.moe_ffn_wgrad(s, dy, x, a, dh, dgu, ddn, ws, n)
    for got, p, q in ((dgu, dh, x), (ddn, dy, a)):
        want = _h(p).T @ _h(q)
        _near(_h(got), want, T * STEP * (np.abs(_h(p)).T @ np.abs(_h(q))), "got")
    dgu2, ddn2 = dgu.clone(), ddn.clone()
    m.moe_ffn_wgrad(m.make_ffn_shape(T, d, F), dy, x, a, dh, dgu2, ddn2, ws, n)
    # accumulating: the old value joins the fp32 sum somewhere, a few more roundings
    for got, old, p, q in ((dgu2, dgu, dh, x), (ddn2, ddn, dy, a)):
        bar = (T + 16) * STEP * (np.abs(_h(p)).T @ np.abs(_h(q)) + np.abs(_h(old)))
        assert np.all(np.abs(_h(got) - 2 * _h(old)) <= bar)
    dgu3, ddn3 = torch.empty_like(dgu), torch.empty_like(ddn)
    m.moe_ffn_wgrad(s, dy, x, a, dh, dgu3, ddn3, ws, n)
    assert torch.equal(dgu3, dgu) and torch.equal(ddn3, ddn)  # fixed order: the same bits


def test_wgrad_of_no_tokens():
    import torch
    m = _moe()
    dgu, ddn = torch.full((256, 64), 2.0, device="cuda"), torch.full((64, 128), 2.0, device="cuda")
    m.moe_ffn_wgrad(m.make_ffn_shape(0, 64, 128), None, None, None, None, dgu, ddn, None, 0)
    torch.cuda.synchronize()
    assert (dgu == 2).all() and (ddn == 2).all()
    s = m.make_ffn_shape(0, 64, 128, m.MOE_DTYPE_BF16, m.MOE_FFN_OVERWRITE_DW)
    m.moe_ffn_wgrad(s, None, None, None, None, dgu, ddn, None, 0)
    torch.cuda.synchronize()
    assert (dgu == 0).all() and (ddn == 0).all()


def _mx8(t):
    import torch
    m = _moe()
    q = torch.empty(t.shape, dtype=torch.uint8, device="cuda")
    s = torch.empty(t.shape[0], t.shape[1] // 32, dtype=torch.uint8, device="cuda")
    m.moe_mx8_quantize(t.shape[0], t.shape[1], m.MOE_DTYPE_BF16, t, q, s)
    return q, s


def _block_cut(p, q):
    """32 * 2^-13 times the sum over blocks of max|p| max|q|, for every pair of rows."""
    return 2.0 ** -8 * (np.abs(p).reshape(p.shape[0], -1, 32).max(axis=2) @
                        np.abs(q).reshape(q.shape[0], -1, 32).max(axis=2).T)


def _values(q, s):
    import torch
    v = q.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)
    return v * np.repeat(np.ldexp(1.0, s.cpu().numpy().astype(np.int64) - 127), 32, axis=1)


@pytest.mark.parametrize("T,d,F", [(1, 128, 128), (1, 4096, 2816), (3, 256, 384), (16, 128, 640), (17, 512, 256),
                                   (48, 384, 1408), (64, 1024, 128), (65, 128, 256), (144, 640, 384),
                                   (145, 128, 1152), (250, 1920, 2816),
                                   (700, 1152, 640), (1300, 512, 1408), (4200, 2048, 128), (6001, 128, 1408),
                                   (9000, 384, 1152), (1500, 1536, 128), (65793, 256, 128), (65600, 256, 128)])
def test_forward_mx8(T, d, F):
    """Rows and weights of widely different block scales, so that a scale applied to a wrong block shows."""
    import torch
    m = _moe()
    rng = np.random.default_rng(T + d + F + 3)

    def scaled(t):
        e = torch.from_numpy(rng.integers(-3, 4, (t.shape[0], t.shape[1] // 32)).astype(np.float32)).cuda()
        return (t.float() * torch.exp2(e).repeat_interleave(32, dim=1)).bfloat16()

    x, add = scaled(_rand(rng, T, d)), _rand(rng, T, d)
    wgu, wdn = (scaled(w) for w in _weights(rng, d, F))
    (xq, xs), (gq, gs), (dq, ds) = _mx8(x), _mx8(wgu), _mx8(wdn)
    s = m.make_ffn_shape(T, d, F, m.MOE_DTYPE_MX8)
    n, _ = m.moe_ffn_workspace_size(s)
    ws = _ws(n)
    y = _nan(T, d)
    print(f"[ffn mx8] T={T} d={d} F={F}", flush=True)
    m.moe_ffn_fwd(s, xq, xs, gq, gs, dq, ds, add, None, None, y, ws, ws.numel())
    xv, gv, dv = _values(xq, xs), _values(gq, gs), _values(dq, ds)
    h64, a64, _ = oracle.dense_ffn_fwd(xv, gv, dv)
    dh = d * STEP * (np.abs(xv) @ np.abs(gv).T) + _block_cut(xv, gv)
    g, u = h64[:, :F], h64[:, F:]
    da = 1.1 * np.abs(u) * dh[:, :F] + np.abs(g * _sig(g)) * dh[:, F:] + 1.1 * dh[:, :F] * dh[:, F:]
    da = da + SIG * (np.abs(a64) + da)
    aq = ws[:T * F].view(T, F)
    off = -(-T * F // 256) * 256
    asc = ws[off:off + T * F // 32].view(T, F // 32)
    av = _values(aq, asc)
    S = np.ldexp(1.0, asc.cpu().numpy().astype(np.int64) - 127)
    top = np.abs(a64).reshape(T, -1, 32).max(axis=2)
    dtop = da.reshape(T, -1, 32).max(axis=2)
    fits = (top - dtop <= 448 * S) & ((top + dtop >= 448 * S / 2) | (S == 2.0 ** -127))
    assert fits.all()
    Sx = np.repeat(S, 32, axis=1)
    _near(av, a64, np.maximum(2.0 ** -4 * (np.abs(a64) + da), 2.0 ** -10 * Sx) * (1 + 1e-9) + da, "a")
    for add_t, add_v in ((add, _h(add)), (None, 0.0)):
        if add_t is None:
            m.moe_ffn_fwd(s, xq, xs, gq, gs, dq, ds, None, None, None, y, ws, ws.numel())
        y64 = av @ dv.T + add_v
        tol = (F + 1) * STEP * (np.abs(av) @ np.abs(dv).T + np.abs(add_v)) + _block_cut(av, dv)
        _near(_h(y), y64, tol + HALF * (np.abs(y64) + tol), "y")


def test_mx8_not_a_number_stays_in_its_row():
    import torch
    m = _moe()
    rng = np.random.default_rng(9)
    for T in (5, 200):
        x, (wgu, wdn) = _rand(rng, T, 256), _weights(rng, 256, 256)
        (gq, gs), (dq, ds) = _mx8(wgu), _mx8(wdn)
        s = m.make_ffn_shape(T, 256, 256, m.MOE_DTYPE_MX8)
        n, _ = m.moe_ffn_workspace_size(s)
        ys = []
        for bad in (False, True):
            if bad:
                x[3, 100] = float("inf")
            xq, xs = _mx8(x)
            y = _nan(T, 256)
            ws = _ws(n)
            m.moe_ffn_fwd(s, xq, xs, gq, gs, dq, ds, None, None, None, y, ws, n)
            ys.append(y)
        torch.cuda.synchronize()
        assert torch.isnan(ys[1][3]).all()
        keep = [i for i in range(T) if i != 3]
        assert torch.equal(_bits(ys[0][keep]), _bits(ys[1][keep]))


def test_rows_behind_the_last_token_stay():
    """Buffers made for more tokens: rows from T on keep their bytes."""
    import torch
    m = _moe()
    rng = np.random.default_rng(10)
    d, F = 192, 320
    wgu, wdn = _weights(rng, d, F)
    for T in (1, 40, 130):
        cap = T + 70
        x, dy = _rand(rng, cap, d), _rand(rng, cap, d)
        h, a, y, dh, dx = _nan(cap, 2 * F), _nan(cap, F), _nan(cap, d), _nan(cap, 2 * F), _nan(cap, d)
        s = m.make_ffn_shape(T, d, F)
        m.moe_ffn_fwd(s, x, None, wgu, None, wdn, None, None, h, a, y, None, 0)
        m.moe_ffn_dgrad(s, dy, h, wgu, wdn, None, dh, dx)
        torch.cuda.synchronize()
        for t in (h, a, y, dh, dx):
            assert torch.isfinite(t[:T].float()).all() and torch.isnan(t[T:].float()).all()
