"""Orthogonalisation and the Muon step against the fp64 oracle, through the C
ABI.

Tolerances. What the choice of types costs on a given matrix is computed, not
guessed: `oracle.orthogonalize_halves` runs the same iteration in fp64 with the
kernels' fp16 tensors, and its distance r from the formula is the sum of those
roundings. The kernels' fp32 sums decide some of the roundings the other way,
which makes another sample of the same errors, of the same size up to a few
per cent: 2 r is allowed in norm, and 40 times the root mean square (2 r over
sqrt(n)) in an element. To that come the fp32 sums themselves, of at most L
terms each (2^-23 sqrt(L), carried through slopes below 4 a step, 4^5 / 3 in
all: 2^-13 at L = 1024, and no more than that for others), and o's own rounding
to bf16, 2^-8 of each element.
"""
import math

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
U = 2.0 ** -24


def _moe():
    import token_dispatch_grouped_amd as m
    return m


def _h(t):
    return t.double().cpu().numpy()


def _gradient(rng, batch, rows, cols, uneven=1.0):
    g = rng.normal(size=(batch, rows, cols)) * np.exp(0.5 * rng.normal(size=(batch, rows, 1)))
    g = g * np.exp(0.5 * rng.normal(size=(batch, 1, cols)))
    k = min(4, rows, cols)
    return (g + uneven * rng.normal(size=(batch, rows, k)) @ rng.normal(size=(batch, k, cols))).astype(np.float32)


def _bars(u, o64):
    """(in norm, in an element) before o's own rounding."""
    r = np.linalg.norm(oracle.orthogonalize_halves(u) - o64) * 2 + 2.0 ** -13 * np.linalg.norm(o64)
    return r, 40 * r / math.sqrt(o64.size)


def _check(o, u, rounded=True):
    o64 = oracle.orthogonalize(u)
    norm, elem = _bars(u, o64)
    half = HALF if rounded else 0.0
    d = np.abs(o - o64)
    assert np.linalg.norm(d) <= norm + half * np.linalg.norm(o64), (np.linalg.norm(d), norm, np.linalg.norm(o64))
    assert np.all(d <= elem + half * (np.abs(o64) + elem)), (d.max(), elem)


def _orth(x, batch=None, out=None, dtype=None):
    import torch
    m = _moe()
    b, rows, cols = x.shape
    s = m.make_orth_shape(b if batch is None else batch, rows, cols,
                          m.MOE_DTYPE_BF16 if x.dtype == torch.bfloat16 else m.MOE_DTYPE_F32)
    ws = torch.full((m.moe_orthogonalize_workspace_size(s),), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full((b, rows, cols), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    m.moe_orthogonalize(s, x, o, ws, ws.numel())
    torch.cuda.synchronize()
    return o


# one element, vectors, sides around 64, odd ones, either side the longer, every tile shape
SHAPES = [(1, 1, 1), (2, 1, 7), (2, 9, 1), (3, 63, 65), (2, 64, 64), (2, 65, 63), (1, 127, 200), (5, 200, 129),
          (1, 333, 1001), (3, 1001, 333), (1, 700, 1300), (2, 960, 704), (1, 130, 3001), (7, 33, 31)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_orthogonalize(batch, rows, cols, bf16):
    import torch
    rng = np.random.default_rng(batch + rows + cols)
    x = torch.from_numpy(_gradient(rng, batch, rows, cols) * 1e-3).to(torch.bfloat16 if bf16 else torch.float32).cuda()
    print(f"[orth] {batch} x {rows} x {cols} bf16={bf16}", flush=True)
    o = _orth(x)
    for i in range(batch):
        _check(_h(o[i]), _h(x[i]))
    if bf16:
        y = x.clone()
        assert torch.equal(_orth(y, out=y), o)


# X X^T in 2 and 3 slices of the sum, their partial sums joined: one matrix, several, tall
@pytest.mark.parametrize("batch,rows,cols", [(1, 1500, 4200), (5, 700, 4100), (1, 6200, 1430)])
def test_long_sums_in_slices(batch, rows, cols):
    test_orthogonalize(batch, rows, cols, False)


@pytest.mark.parametrize("distinct,copies,rows,cols", [(3, 80, 256, 448), (3, 60, 520, 300), (2, 100, 512, 640), (2, 24, 900, 1024),
                                                       (2, 40, 1024, 1030)])
def test_many_matrices(distinct, copies, rows, cols):
    """Batches that fill the card, of a few distinct matrices over and over: every copy has the same bits."""
    import torch
    rng = np.random.default_rng(rows + cols)
    one = torch.from_numpy(_gradient(rng, distinct, rows, cols)).cuda()
    x = one.repeat(copies, 1, 1)
    print(f"[orth] {distinct} x {copies} of {rows} x {cols}", flush=True)
    o = _orth(x).view(copies, distinct, rows, cols)
    for i in range(distinct):
        _check(_h(o[0, i]), _h(one[i]))
    assert (o.view(torch.int16) == o[:1].view(torch.int16)).all()


def test_uneven_singular_values():
    """A few directions that hold nearly all the weight: the rest of the matrix keeps its digits."""
    import torch
    rng = np.random.default_rng(11)
    for strong in (10.0, 100.0):
        x = 0.1 * rng.normal(size=(1, 320, 512)) + strong * rng.normal(size=(1, 320, 6)) @ rng.normal(size=(1, 6, 512))
        t = torch.from_numpy(x.astype(np.float32)).cuda()
        _check(_h(_orth(t)[0]), _h(t[0]))


def test_scales_zeros_and_non_finite():
    """From the smallest to the largest fp32 numbers, a matrix of zeros, and an infinity or a NaN, which fills its own
    matrix and no other."""
    import torch
    rng = np.random.default_rng(12)
    base = torch.from_numpy(_gradient(rng, 1, 96, 160)).cuda()
    ref = _orth(base)
    for e in (-90, -10, 60, 110):
        x = base * 2.0 ** e
        assert torch.isfinite(x).all()
        got = _orth(x)
        if e >= -10:  # |U| is far above eps
            _check(_h(got[0]), _h(x[0]))
        else:  # |U| is far below eps: X starts as U / eps
            u = _h(x[0])
            assert np.linalg.norm(_h(got[0])) <= 1.1 * 3.4445 ** 5 * np.linalg.norm(u) / 1e-7 + 1e-30
    batch = base.repeat(4, 1, 1)
    batch[1] = 0
    batch[2, 5, 7] = float("inf")
    batch[3, 95, 159] = float("nan")
    o = _orth(batch)
    assert torch.equal(o[0], ref[0]) and not o[1].any() and torch.isnan(o[2]).all() and torch.isnan(o[3]).all()


def test_fewer_matrices_than_the_buffers_hold():
    import torch
    rng = np.random.default_rng(13)
    x = torch.from_numpy(_gradient(rng, 4, 70, 90)).cuda()
    o = torch.full((4, 70, 90), 7.0, device="cuda").bfloat16()
    full = _orth(x)
    _orth(x, batch=2, out=o)
    assert torch.equal(o[:2], full[:2]) and (o[2:] == 7).all()
    _orth(x, batch=0, out=o)
    assert (o[2:] == 7).all()


def test_other_coefficients_and_steps():
    import torch
    m = _moe()
    rng = np.random.default_rng(14)
    x = torch.from_numpy(_gradient(rng, 1, 100, 150)).cuda()
    for steps, coef in ((1, oracle.ORTH_COEF), (2, oracle.ORTH_COEF), (12, (1.5, -0.5, 0.0)), (8, (2.0, -1.5, 0.5))):
        s = m.make_orth_shape(1, 100, 150, m.MOE_DTYPE_F32, steps, coef)
        ws = torch.empty(m.moe_orthogonalize_workspace_size(s), dtype=torch.uint8, device="cuda")
        o = torch.empty(1, 100, 150, dtype=torch.bfloat16, device="cuda")
        m.moe_orthogonalize(s, x, o, ws, ws.numel())
        u = _h(x[0])
        o64 = oracle.orthogonalize(u, steps, coef)
        r = 2 * np.linalg.norm(oracle.orthogonalize_halves(u, steps, coef) - o64) + 2.0 ** -13 * np.linalg.norm(o64)
        assert np.linalg.norm(_h(o[0]) - o64) <= r + HALF * np.linalg.norm(o64)


def _muon(cfg, shape, p, g, mom, low):
    import torch
    m = _moe()
    ws = torch.full((m.moe_orthogonalize_workspace_size(shape),), 0xFF, dtype=torch.uint8, device="cuda")
    m.moe_muon_step(cfg, shape, p, g, mom, low, ws, ws.numel())
    torch.cuda.synchronize()


@pytest.mark.parametrize("nesterov,zero,lowp", [(True, True, True), (False, False, True), (True, False, False)])
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 5), (2, 65, 63), (3, 100, 257), (1, 640, 320), (4, 128, 192)])
def test_muon_step(batch, rows, cols, nesterov, zero, lowp):
    """Two steps. momentum: two fp32 roundings a step. param: the formula's with the update within lr * scale times
    o's bars, and the two roundings of param itself."""
    import torch
    m = _moe()
    rng = np.random.default_rng(batch + rows * 3 + cols)
    dev = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    p, mom = dev(rng.normal(0, 0.02, (batch, rows, cols))), dev(_gradient(rng, batch, rows, cols) * 1e-2)
    low = p.bfloat16() if lowp else None
    lr, mu, wd, scale, gs = 0.01, 0.95, 0.1, 0.2 * math.sqrt(max(rows, cols)), 0.5
    cfg = m.make_muon_config(lr, mu, wd, scale, gs, nesterov, zero)
    shape = m.make_orth_shape(batch, rows, cols)
    for _ in range(2):
        g = dev(_gradient(rng, batch, rows, cols) * 1e-3)
        p0, m0, g0 = _h(p), _h(mom), _h(g)
        print(f"[muon] {batch} x {rows} x {cols}", flush=True)
        _muon(cfg, shape, p, g, mom, low)
        assert (g == 0).all() if zero else np.array_equal(_h(g), g0)
        for i in range(batch):
            _, m64, _ = oracle.muon_step(p0[i], g0[i], m0[i], lr, mu, wd, scale, gs, nesterov)
            assert np.all(np.abs(_h(mom[i]) - m64) <= 2 * U * (np.abs(mu * m0[i]) + np.abs(gs * g0[i])) + 2 * U * np.abs(m64))
            # the update from the momentum that the kernel wrote, so that its rounding is not counted twice
            u = gs * g0[i] + mu * _h(mom[i]) if nesterov else _h(mom[i])
            o64 = oracle.orthogonalize(u)
            norm, elem = _bars(u, o64)
            p64 = p0[i] * (1 - lr * wd) - lr * scale * o64
            d = np.abs(_h(p[i]) - p64)
            own = 2 * U * (np.abs(p0[i]) + lr * scale * np.abs(o64)) + 2 * U * np.abs(p64)
            assert np.all(d <= lr * scale * elem + own)
            assert np.linalg.norm(d) <= lr * scale * norm + np.linalg.norm(own)
        if lowp:
            assert torch.equal(low, p.bfloat16())


def test_the_same_bits_every_time_and_with_fewer_matrices():
    import torch
    m = _moe()
    rng = np.random.default_rng(15)
    dev = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    g, mom, p = dev(_gradient(rng, 6, 200, 330)), dev(_gradient(rng, 6, 200, 330)), dev(rng.normal(0, 0.02, (6, 200, 330)))
    cfg = m.make_muon_config(0.01)
    outs = []
    for n in (6, 6):
        p1, m1, low = p.clone(), mom.clone(), torch.zeros(6, 200, 330, device="cuda").bfloat16()
        _muon(cfg, m.make_orth_shape(n, 200, 330), p1, g.clone(), m1, low)
        outs.append((p1, m1, low))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
