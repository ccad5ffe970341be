"""Rows of the norm whose squares pass fp32's range: |r| up to 2^127, where the
sum of squares is beyond 2^128 though rstd and y are ordinary numbers.

Tolerances: those of test_gpu_norm.py (a chain of at most d/64 + 16 additions
of terms with one rounding each, then the root, the division and two
products), and half a step of the smallest fp32 numbers, 2^-150, on rstd,
which is below 2^-126 for the longest of these rows. y carries that as a
relative 2^-150 / rstd.
"""
import numpy as np
import pytest

import oracle
from tests.test_gpu_norm import EPS, _arith, _check_mx8, _fwd, _h, _half, _moe, _round_r, _torch

pytestmark = pytest.mark.gpu


def _rows(rng, T, d, bf16):
    """Normal rows times 2^0, 2^60, 2^90 and 2^124 in turn."""
    import torch
    v = rng.normal(0, 1, (T, d)).clip(-6, 6) * np.exp2(np.array([0, 60, 90, 124])[np.arange(T) % 4])[:, None]
    return torch.from_numpy(v.astype(np.float32)).to(_torch(bf16)).cuda()


# a workgroup a row, one wavefront a row, and rows read twice
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,d", [(4, 64), (5, 4096), (2051, 512), (2060, 1088), (6, 65536)])
def test_forward_of_large_rows(T, d, bf16):
    m = _moe()
    rng = np.random.default_rng(T + d)
    x = _rows(rng, T, d, bf16)
    w = _rows(rng, 1, d, bf16)[0].contiguous()
    for res in (None, _rows(rng, T, d, bf16)):
        print(f"[norm range] T={T} d={d} bf16={bf16} residual={res is not None}", flush=True)
        r64, rstd64, y64 = oracle.rmsnorm_fwd(_h(x), _h(w), EPS, None if res is None else _h(res), _round_r(bf16))
        r, y, _, rstd = _fwd(m, x, res, w, False, bf16)
        if res is not None:
            assert np.array_equal(_h(r), r64)
        low = 2.0 ** -150 / rstd64
        assert np.all(np.abs(_h(rstd) - rstd64) <= (_arith(d) + low) * rstd64)
        rel = (_arith(d) + low)[:, None]
        assert np.all(np.abs(_h(y) - y64) <= (rel + _half(bf16)) * np.abs(y64))
        _, q, s, rstd2 = _fwd(m, x, res, w, True, bf16)
        assert np.array_equal(_h(rstd2), _h(rstd))
        _check_mx8(q, s, y64, float(rel.max()))


def test_infinite_and_nan_rows_stay_as_they_are():
    """An infinity makes its own element NaN and the others zero, as rstd is 1 / sqrt(infinity)."""
    import torch
    m = _moe()
    rng = np.random.default_rng(8)
    for T, d in ((4, 512), (2052, 512), (4, 16384)):
        x, w = _rows(rng, T, d, True), _rows(rng, 1, d, True)[0].contiguous()
        x[1, 7] = float("inf")
        x[2, 9] = float("nan")
        y, rstd = (_fwd(m, x, None, w, False, True)[i] for i in (1, 3))
        assert rstd[1] == 0 and torch.isnan(y[1, 7]) and torch.count_nonzero(torch.nan_to_num(y[1], nan=0.0)) == 0
        assert torch.isnan(rstd[2]) and torch.isnan(y[2]).all()
        assert torch.isfinite(y[0].float()).all() and torch.isfinite(y[3].float()).all() and rstd[3] > 0
