"""Orthogonalisation of matrices whose short side is at most 384: every tensor
of the iteration in two fp16 halves, so that the result is the formula's to
fp32's own error. Seen in a Muon step from weights of zero, which writes -o in
fp32.

Tolerances, in norm, relative to the result's. The types alone cost r2 (the
oracle's iteration with them, sums exact), of which the kernels' sums make
another sample: 2 r2. The sums are fp32, of three products each instead of one,
in another order than the oracle's fp32 iteration has: four times its distance
from the formula. To both comes half a step of fp32 in the weight.
"""
import numpy as np
import pytest

import oracle
from tests import test_gpu_orth as base

pytestmark = pytest.mark.gpu


def _o(x):
    import torch
    m = base._moe()
    s = m.make_orth_shape(*x.shape)
    ws = torch.full((m.moe_orthogonalize_workspace_size(s),), 0xFF, dtype=torch.uint8, device="cuda")
    p, mom, g = torch.zeros_like(x), torch.zeros_like(x), x.clone()
    m.moe_muon_step(m.make_muon_config(1.0, 0.0, 0.0, 1.0), s, p, g, mom, None, ws, ws.numel())
    torch.cuda.synchronize()
    return -p


def _check(o, u):
    o64 = oracle.orthogonalize(u)
    bar = 2 * np.linalg.norm(oracle.orthogonalize_both_halves(u) - o64) + 4 * np.linalg.norm(oracle.orthogonalize_f32(u) - o64)
    bar = bar + 2.0 ** -24 * np.linalg.norm(o64)
    far = np.linalg.norm(o - o64)
    assert far <= bar, (far / np.linalg.norm(o64), bar / np.linalg.norm(o64))


# small, middling and square tiles, wide and tall, odd sides, the border, sums in slices (copies of 2 matrices)
@pytest.mark.parametrize("copies,rows,cols", [(1, 1, 1), (1, 3, 7), (1, 8, 8), (2, 62, 14), (1, 21, 372), (1, 40, 40), (4, 88, 141),
                                              (1, 128, 128), (1, 65, 3001), (1, 419, 328), (1, 333, 1001), (1, 384, 384),
                                              (1, 1100, 377), (15, 200, 300), (15, 300, 200), (40, 300, 200), (15, 320, 450),
                                              (32, 450, 333), (43, 384, 644), (7, 380, 8200), (7, 4100, 384)])
def test_as_near_as_fp32(copies, rows, cols):
    import torch
    rng = np.random.default_rng(rows * 7 + cols)
    x = torch.from_numpy(base._gradient(rng, 2, rows, cols)).cuda()
    print(f"[orth] short sides 2 x {copies} of {rows} x {cols}", flush=True)
    o = _o(x.repeat(copies, 1, 1)).view(copies, 2, rows, cols)
    for i in range(2):
        _check(base._h(o[0, i]), base._h(x[i]))
    assert torch.equal(o, o[:1].expand_as(o))


def test_uneven_singular_values():
    import torch
    rng = np.random.default_rng(11)
    for strong in (10.0, 100.0):
        x = 0.1 * rng.normal(size=(1, 320, 512)) + strong * rng.normal(size=(1, 320, 6)) @ rng.normal(size=(1, 6, 512))
        t = torch.from_numpy(x.astype(np.float32)).cuda()
        _check(base._h(_o(t)[0]), base._h(t[0]))
