"""The dense block where a product takes several rounds of its largest tiles
and a rest, the weight gradients of 256 x 256 tiles with the tokens in slices,
and padded batches: the operators' own tests (test_gpu_ffn.py has the bars) at
the sizes that reach these paths, which the launch records and the plan
assert.
"""
import numpy as np
import pytest

import oracle
from tests import test_gpu_ffn as base
from tests.parity_util import TOL, assert_close, to_host64
from tests.test_ffn_plan_host import SLICED
from workloads import BF16

pytestmark = pytest.mark.gpu


def _launches(call):
    import torch
    from token_dispatch_grouped_amd import _lib
    _lib.moe_profiler_reset()
    _lib.moe_profiler_enable(True)
    try:
        call()
        torch.cuda.synchronize()
        return {k: n for k, (n, _) in _lib.moe_profiler_read_all().items()}
    finally:
        _lib.moe_profiler_enable(False)
        _lib.moe_profiler_reset()


def _two_rounds_and_a_rest(T, N):
    """The 256 x 256 tiles of [T, N] are more than twice the CUs and no whole rounds."""
    import torch
    cus = torch.cuda.get_device_properties(0).multi_processor_count // 8 * 8
    tiles = -(-T // 256) * -(-N // 256)
    return tiles > 2 * cus and tiles % cus != 0


# the products with N = d: the down product (plain, with an addend, in place) and gate/up's input gradient
def test_forward_over_rounds():
    import torch
    import token_dispatch_grouped_amd as m
    T, d, F = 16700, 2048, 192
    assert _two_rounds_and_a_rest(T, d)
    x, wgu, wdn = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((T, d), (2 * F, d), (d, F)))
    h, a, y = (torch.empty(T, c, dtype=torch.bfloat16, device="cuda") for c in (2 * F, F, d))
    for add in (None, x):
        got = _launches(lambda: m.moe_ffn_fwd(m.make_ffn_shape(T, d, F), x, None, wgu, None, wdn, None, add, h, a, y,
                                              None, 0))
        assert got["ffn_down_fwd"] == 2, got
    base.test_forward(T, d, F)


@pytest.mark.parametrize("T,d,F,entry", [(16700, 2048, 192, "ffn_gateup_dgrad"), (16700, 64, 2048, "ffn_down_dgrad")])
def test_dgrad_over_rounds(T, d, F, entry):
    import torch
    import token_dispatch_grouped_amd as m
    assert _two_rounds_and_a_rest(T, max(d, F))
    dy, wgu, wdn = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((T, d), (2 * F, d), (d, F)))
    h, dh, dx = (torch.zeros(T, c, dtype=torch.bfloat16, device="cuda") for c in (2 * F, 2 * F, d))
    for add in (None, dy):
        got = _launches(lambda: m.moe_ffn_dgrad(m.make_ffn_shape(T, d, F), dy, h, wgu, wdn, add, dh, dx))
        assert got[entry] == 2, got
    base.test_dgrad(T, d, F)


@pytest.mark.parametrize("T,d,F,slices", SLICED)
def test_wgrad_of_large_tiles_in_slices(T, d, F, slices):
    """Overwriting, accumulating and repeated; the plan of each size is asserted in test_ffn_plan_host.py."""
    base.test_wgrad(T, d, F)


@pytest.mark.parametrize("T,d,F", [(77, 128, 192), (700, 1088, 576), (3011, 576, 1088)])
def test_wgrad_of_a_padded_batch(T, d, F):
    """Rows behind the last token, NaN here, are no part of the sums."""
    import torch
    import token_dispatch_grouped_amd as m
    rng = np.random.default_rng(T)
    full = [base._rand(rng, T + 70, c) for c in (d, d, F, 2 * F)]
    for t in full:
        t[T:] = float("nan")
    s = m.make_ffn_shape(T, d, F, m.MOE_DTYPE_BF16, m.MOE_FFN_OVERWRITE_DW)
    _, n = m.moe_ffn_workspace_size(s)
    got = []
    for ops in (full, [t[:T].clone() for t in full]):
        dgu, ddn = torch.empty(2 * F, d, device="cuda"), torch.empty(d, F, device="cuda")
        ws = base._ws(n)
        m.moe_ffn_wgrad(s, *ops, dgu, ddn, ws, n)
        got.append((dgu, ddn))
    for p, q in zip(*got):
        assert torch.isfinite(p).all() and torch.equal(p, q)


def test_wgrad_without_a_workspace():
    """Gradients of 512 tiles: one slice of the tokens whatever their number, nothing kept beside the gradients."""
    import torch
    import token_dispatch_grouped_amd as m
    rng = np.random.default_rng(3)
    T, d, F = 100, 65536, 128
    dy, x, a, dh = (base._rand(rng, T, c) for c in (d, d, F, 2 * F))
    s = m.make_ffn_shape(T, d, F, m.MOE_DTYPE_BF16, m.MOE_FFN_OVERWRITE_DW)
    assert m.moe_ffn_workspace_size(s)[1] == 0
    nan = float("nan")
    dgu, ddn = torch.full((2 * F, d), nan, device="cuda"), torch.full((d, F), nan, device="cuda")
    print(f"[ffn wgrad] T={T} d={d} F={F} no workspace", flush=True)
    m.moe_ffn_wgrad(s, dy, x, a, dh, dgu, ddn, None, 0)
    for got, p, q in ((dgu, dh, x), (ddn, dy, a)):
        p, q = base._h(p), base._h(q)
        base._near(base._h(got), p.T @ q, T * base.STEP * (np.abs(p).T @ np.abs(q)), "dw")
    dgu2, ddn2 = dgu.clone(), ddn.clone()
    m.moe_ffn_wgrad(m.make_ffn_shape(T, d, F), dy, x, a, dh, dgu2, ddn2, None, 0)
    # one more addition, of a sum of the same size
    assert torch.equal(dgu2, dgu + dgu) and torch.equal(ddn2, ddn + ddn)


def test_offsets_past_32_bits_in_the_large_tiles():
    """1.1 million rows of 2 x 1024 columns: the rows on both sides of the border between the large tiles' launch and
    the rest's, and rows well inside the first, all beyond 2^31 elements from the start."""
    import torch
    import token_dispatch_grouped_amd as m
    bf = torch.bfloat16
    T, d, F = 1_100_000, 64, 1024
    cus = torch.cuda.get_device_properties(0).multi_processor_count // 8 * 8
    cols = 2 * F // 256
    head = -(-T // 256) * cols // cus * cus // cols * 256
    rows = torch.tensor([2 ** 31 // (2 * F) + i for i in (0, 1, 300)] + [head - 20000] + list(range(head - 3, head + 3)) +
                        [T - 1], device="cuda")
    assert head - 20000 > 2 ** 31 // (2 * F) and head < T
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, add = (torch.randn(T, d, generator=gen, device="cuda", dtype=bf) for _ in range(2))
    wg, wd = (torch.randn(*sh, generator=gen, device="cuda", dtype=bf) * 0.05 for sh in ((2 * F, d), (d, F)))
    s = m.make_ffn_shape(T, d, F)
    h, a, y = (torch.empty(T, c, dtype=bf, device="cuda") for c in (2 * F, F, d))
    print("[offsets] forward", flush=True)
    got = _launches(lambda: m.moe_ffn_fwd(s, x, None, wg, None, wd, None, add, h, a, y, None, 0))
    assert got["ffn_gateup_fwd"] == 2, got
    tx, tadd, w64, d64 = (to_host64(t) for t in (x[rows], add[rows], wg, wd))
    h64, a64, y64 = oracle.dense_ffn_fwd(tx, w64, d64, tadd)
    for name, t, want in (("h", h, h64), ("a", a, a64), ("y", y, y64)):
        assert_close(name, to_host64(t[rows]), want, TOL[BF16])
    print("[offsets] input gradient", flush=True)
    h_rows = to_host64(h[rows])
    del a, y
    dh, dx = torch.empty_like(h), torch.empty_like(x)
    got = _launches(lambda: m.moe_ffn_dgrad(s, add, h, wg, wd, x, dh, dx))
    assert got["ffn_down_dgrad"] == 2, got
    _, dh64, dx64 = oracle.dense_ffn_dgrad(tadd, h_rows, w64, d64, tx)
    assert_close("dh", to_host64(dh[rows]), dh64, TOL[BF16])
    assert_close("dx", to_host64(dx[rows]), dx64, TOL[BF16])
