"""Layer norm of rows whose spread is no more than a few steps of their values:
one value throughout, and all but one or a few of them a step off.

Tolerances: those of the layer norm's own tests (a row's sums of at most d/64 +
16 additions, A = (d/64 + 24) 2^-24 of the spread, however far the mean is from
zero), which hold for such rows as for any other. The oracle's mean of equal
fp32 values is exact.
"""
import numpy as np
import pytest

from tests.test_gpu_layernorm import EPS, _check_fwd, _fwd, _h, _moe, _nan, _rand

pytestmark = pytest.mark.gpu

# a wavefront and a workgroup a row, in registers and from the caches; lengths whose inverse is rounded
SHAPES = [(5, 768), (7, 4160), (40, 7168), (3, 65472), (2100, 576), (2100, 1088)]


def _rows(T, d, bf16, magnitude, seed):
    import torch
    v = np.random.default_rng(seed).uniform(1, 2, (T, 1)).astype(np.float32) * np.float32(magnitude)
    v = torch.from_numpy(v).to(torch.bfloat16 if bf16 else torch.float32).cuda()
    return v.repeat(1, d).contiguous()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,d", SHAPES)
def test_rows_of_one_value(T, d, bf16):
    """n is zero and rstd 1 / sqrt(eps), at any size of the value."""
    m = _moe()
    rng = np.random.default_rng(T + d)
    w, b = _rand(rng, d, bf16=bf16), _rand(rng, d, bf16=bf16)
    for i, magnitude in enumerate((1.0, 1e4, 1e7, 1e9, 1e12, 1.5e15, 1e17, 1e19, 1e25, 1e37)):
        print(f"[ln] T={T} d={d} bf16={bf16} of {magnitude}", flush=True)
        x = _rows(T, d, bf16, magnitude, i)
        _check_fwd(_fwd(m, x, None, w, b, bf16), x, None, w, b, bf16)


@pytest.mark.parametrize("T,d", SHAPES)
def test_rows_a_step_off(T, d):
    """Some values of each fp32 row are the next number: a spread of 1 / sqrt(d) to 1/2 of a step."""
    import torch
    m = _moe()
    rng = np.random.default_rng(T + d + 1)
    w, b = _rand(rng, d, bf16=False), _rand(rng, d, bf16=False)
    for magnitude in (1.0, 1e5, 1e9, 1e15):
        for off in (1, 7, d // 2):
            print(f"[ln] T={T} d={d} of {magnitude}, {off} a step off", flush=True)
            x = _rows(T, d, False, magnitude, off)
            cols = torch.from_numpy(rng.permutation(d)[:off]).cuda()
            bits = x.view(torch.int32)
            bits[:, cols] += 1
            _check_fwd(_fwd(m, x, None, w, b, False), x, None, w, b, False)


def test_gradient_of_rows_of_one_value():
    """Through the forward's own statistics: n is zero, so dx is rstd (g - mean(g)) and dw zero. rstd to the forward's
    bar, the mean of g from d/64 + 16 additions."""
    m = _moe()
    T, d = 40, 7168
    rng = np.random.default_rng(2)
    w, dy = _rand(rng, d, bf16=False), _rand(rng, T, d, bf16=False)
    for magnitude in (1e9, 1.5e15, 1e17):
        x = _rows(T, d, False, magnitude, 3)
        _, _, mean, rstd = _fwd(m, x, None, w, None, False)
        dx, dw, db = _nan(T, d), _nan(d), _nan(d)
        s = m.make_norm_shape(T, d, m.MOE_DTYPE_F32, EPS, m.MOE_NORM_OVERWRITE_DW)
        ws = _nan(m.moe_layernorm_workspace_size(s) // 4)
        m.moe_layernorm_bwd(s, dy, x, w, mean, rstd, None, dx, dw, db, ws, 4 * ws.numel())
        g = _h(dy) * _h(w)
        want = (g - g.mean(axis=1, keepdims=True)) / np.sqrt(EPS)
        bar = (d / 64 + 40) * 2.0 ** -24 * (np.abs(g) + np.abs(g).mean(axis=1, keepdims=True)) / np.sqrt(EPS)
        assert np.all(np.abs(_h(dx) - want) <= bar) and not dw.any()
