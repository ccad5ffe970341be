"""Orthogonalisation and Muon step where the long sums of X X^T run in slices,
which the record of the launches asserts; bars as in test_gpu_orth.py."""
import numpy as np
import pytest

from tests import test_gpu_orth as base
from tests.launched import kernels

pytestmark = pytest.mark.gpu


# matrices, rows, cols: wide and tall, in 3 to 5 slices, stages that are no multiple of them, sums from 4096 on
@pytest.mark.parametrize("copies,rows,cols", [(1, 1450, 6150), (1, 6400, 1472), (9, 500, 8200), (1, 1500, 4200), (5, 4100, 700)])
@pytest.mark.parametrize("muon", [False, True])
def test_slices(copies, rows, cols, muon):
    import torch
    m = base._moe()
    rng = np.random.default_rng(rows + cols)
    x = torch.from_numpy(base._gradient(rng, 1, rows, cols)).cuda().repeat(copies, 1, 1)
    s = m.make_orth_shape(copies, rows, cols)
    ws = torch.full((m.moe_orthogonalize_workspace_size(s),), 0xFF, dtype=torch.uint8, device="cuda")
    print(f"[orth] slices {copies} x {rows} x {cols} muon={muon}", flush=True)
    if muon:  # from no momentum and weights of zero, of which -o is left
        o, mom, g = torch.zeros_like(x), torch.zeros_like(x), x.clone()
        cfg = m.make_muon_config(1.0, 0.0, 0.0, 1.0)
        got = kernels(lambda: m.moe_muon_step(cfg, s, o, g, mom, None, ws, ws.numel()))
        assert torch.equal(mom, x)
        o = -o
    else:
        o = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        got = kernels(lambda: m.moe_orthogonalize(s, x, o, ws, ws.numel()))
    assert got is None or sum(k.startswith("orth_sum_kernel") for k in got) == 5, got
    base._check(base._h(o[0]), base._h(x[0]), rounded=not muon)
    assert torch.equal(o, o[:1].expand_as(o))
