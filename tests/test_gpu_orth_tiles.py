"""The orthogonalisation and the Muon step on every tile of their products,
named by the record of the launches: a few distinct matrices over and over, so
that a batch fills the card and the oracle stays small. Bars: those of the
operators' own tests (test_gpu_orth.py).
"""
import math

import numpy as np
import pytest

import oracle
from tests import test_gpu_orth as base
from tests.launched import kernels

pytestmark = pytest.mark.gpu

SMALL_SYM, SMALL = "orth_tile_kernel<64, 64, 16, 64, 2, 4, ", "orth_tile_kernel<64, 128, 16, 64, 1, 4, "
PAIR, SQUARE, LARGE = "orth_tile_kernel<128, 128, 32, 64, 1, 4, ", "orth_tile_kernel<128, 128, 32, 64, 1, 2, ", "orth_wide_kernel<"

# copies of 2 matrices, rows, cols, the tile of the symmetric products, of the step: wide and tall; 4 columns and more in
# one store, or (cols % 4 != 0) each by itself; sides that leave tiles partly empty; more tiles than workgroups
CASES = [  # short sides, in both halves
    (1, 100, 257, SMALL_SYM, SMALL), (1, 257, 100, SMALL_SYM, SMALL),
    (15, 200, 300, PAIR, PAIR), (15, 300, 200, PAIR, PAIR), (10, 320, 450, PAIR, PAIR), (10, 450, 333, PAIR, PAIR),
    (40, 300, 200, PAIR, SQUARE), (15, 320, 450, PAIR, SQUARE), (15, 450, 330, PAIR, SQUARE), (40, 200, 300, PAIR, SQUARE),
    (32, 320, 448, SQUARE, SQUARE), (32, 450, 333, SQUARE, SQUARE),
    # the others
    (42, 500, 644, LARGE, LARGE), (42, 642, 500, LARGE, LARGE), (85, 640, 500, LARGE, LARGE),
    (1, 700, 780, SMALL_SYM, SMALL), (1, 778, 700, SMALL_SYM, SMALL),
    (3, 700, 780, PAIR, PAIR), (3, 770, 700, PAIR, PAIR), (4, 833, 701, PAIR, SQUARE), (4, 700, 780, PAIR, SQUARE),
    (4, 780, 700, PAIR, SQUARE), (4, 700, 778, PAIR, SQUARE), (7, 700, 780, SQUARE, LARGE), (7, 778, 700, SQUARE, LARGE),
    (9, 700, 778, SQUARE, LARGE), (21, 700, 780, LARGE, LARGE), (21, 778, 700, LARGE, LARGE), (42, 780, 700, LARGE, LARGE),
]


def _dev(a):
    import torch
    return torch.from_numpy(a.astype(np.float32)).cuda()


def _launched(call, short, sym, step, last):
    """Five times gram, polynomial and step, behind the norm and the first pass."""
    got = kernels(call)
    if got is None:
        return
    end = lambda tile, mode: tile + (f"{mode}>" if tile == LARGE else f"{mode}, {'true' if short else 'false'}>")  # noqa: E731
    want = ["orth_norm_kernel", "orth_prep_kernel"]
    for k in range(5):
        want += [end(sym, 0), end(sym, 1), end(step, last if k == 4 else 2)]
    assert len(got) == len(want) and all(g.startswith(w) for g, w in zip(got, want)), got


@pytest.mark.parametrize("copies,rows,cols,sym,step", CASES)
def test_orthogonalize(copies, rows, cols, sym, step):
    import torch
    m = base._moe()
    rng = np.random.default_rng(rows + cols)
    one = _dev(base._gradient(rng, 2, rows, cols))
    x = one.repeat(copies, 1, 1)
    s = m.make_orth_shape(2 * copies, rows, cols)
    ws = torch.full((m.moe_orthogonalize_workspace_size(s),), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    print(f"[orth] 2 x {copies} of {rows} x {cols}", flush=True)
    _launched(lambda: m.moe_orthogonalize(s, x, o, ws, ws.numel()), min(rows, cols) <= 384, sym, step, 3)
    o = o.view(copies, 2, rows, cols)
    for i in range(2):
        base._check(base._h(o[0, i]), base._h(one[i]))
    assert (o.view(torch.int16) == o[:1].view(torch.int16)).all()


@pytest.mark.parametrize("copies,rows,cols,sym,step", CASES)
def test_muon_step(copies, rows, cols, sym, step):
    """Momentum: two fp32 roundings. param: the formula's with the update within lr * scale times o's bars, and the two
    roundings of param itself; rows of a larger buffer behind the batch are left as they are."""
    import torch
    m = base._moe()
    rng = np.random.default_rng(rows * 3 + cols)
    p1, m1 = _dev(rng.normal(0, 0.02, (2, rows, cols))), _dev(base._gradient(rng, 2, rows, cols) * 1e-2)
    g1 = _dev(base._gradient(rng, 2, rows, cols) * 1e-3)
    n = 2 * copies
    spare = lambda t: torch.cat([t.repeat(copies, 1, 1), torch.full_like(t[:1], 7.0)])  # noqa: E731
    p, mom, g = spare(p1), spare(m1), spare(g1)
    low = torch.full_like(p, 7.0).bfloat16()
    lr, mu, wd, scale, gs = 0.01, 0.95, 0.1, 0.2 * math.sqrt(max(rows, cols)), 0.5
    s = m.make_orth_shape(n, rows, cols)
    ws = torch.full((m.moe_orthogonalize_workspace_size(s),), 0xFF, dtype=torch.uint8, device="cuda")
    cfg = m.make_muon_config(lr, mu, wd, scale, gs, True, True)
    print(f"[muon] 2 x {copies} of {rows} x {cols}", flush=True)
    _launched(lambda: m.moe_muon_step(cfg, s, p, g, mom, low, ws, ws.numel()), min(rows, cols) <= 384, sym, step, 4)
    for t in (p, mom, g, low):
        assert (t[n:] == 7).all()
        every = t[:n].view(copies, 2, rows, cols)
        assert torch.equal(every, every[:1].expand_as(every))
    assert not g[:n].any() and torch.equal(low[:n], p[:n].bfloat16())
    U = base.U
    for i in range(2):
        p0, m0, g0 = base._h(p1[i]), base._h(m1[i]), base._h(g1[i])
        _, m64, _ = oracle.muon_step(p0, g0, m0, lr, mu, wd, scale, gs)
        got = base._h(mom[i])
        assert np.all(np.abs(got - m64) <= 2 * U * (np.abs(mu * m0) + np.abs(gs * g0)) + 2 * U * np.abs(m64))
        u = gs * g0 + mu * got  # from the momentum that was written: its rounding is not counted twice
        o64 = oracle.orthogonalize(u)
        norm, elem = base._bars(u, o64)
        p64 = p0 * (1 - lr * wd) - lr * scale * o64
        d = np.abs(base._h(p[i]) - p64)
        own = 2 * U * (np.abs(p0) + lr * scale * np.abs(o64)) + 2 * U * np.abs(p64)
        assert np.all(d <= lr * scale * elem + own)
        assert np.linalg.norm(d) <= lr * scale * norm + np.linalg.norm(own)


@pytest.mark.parametrize("batch,rows,cols", [(6, 200, 330), (6, 330, 200), (96, 320, 448), (28, 700, 780)])
def test_the_same_bits_with_fewer_matrices(batch, rows, cols):
    """The first n matrices of larger buffers, which the same tiles take as the whole batch: the same bits, and the rest
    of every tensor untouched."""
    import torch
    m = base._moe()
    rng = np.random.default_rng(15)
    g, mom = _dev(base._gradient(rng, batch, rows, cols)), _dev(base._gradient(rng, batch, rows, cols))
    p = _dev(rng.normal(0, 0.02, (batch, rows, cols)))
    cfg = m.make_muon_config(0.01, zero_grad=True)
    ws = torch.empty(m.moe_orthogonalize_workspace_size(m.make_orth_shape(batch, rows, cols)), dtype=torch.uint8, device="cuda")
    first, names = None, None
    for n in (batch, batch - 1, batch - 2 if batch > 7 else 1, batch):
        t = [p.clone(), g.clone(), mom.clone(), torch.full_like(p, 7.0).bfloat16()]
        ws.fill_(0xFF)
        print(f"[muon] {n} of {batch} x {rows} x {cols}", flush=True)
        got = kernels(lambda: m.moe_muon_step(cfg, m.make_orth_shape(n, rows, cols), *t, ws, ws.numel()))
        first, names = first or t, names or got
        assert got == names
        for now, all_of_it, old in zip(t, first, (p, g, mom, None)):
            assert torch.equal(now[:n], all_of_it[:n])
            assert torch.equal(now[n:], old[n:]) if old is not None else (now[n:] == 7).all()
