"""The event timer's entries of the dense block: one record a launch, and no
time counted in two entries."""
import pytest

pytestmark = pytest.mark.gpu


def _timed(call, calls):
    """(entries, ms between two events around the calls)"""
    import torch
    from token_dispatch_grouped_amd import _lib
    call()
    torch.cuda.synchronize()
    _lib.moe_profiler_reset()
    _lib.moe_profiler_enable(True)
    try:
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(calls):
            call()
        b.record()
        torch.cuda.synchronize()
        rec = _lib.moe_profiler_read_all()
    finally:
        _lib.moe_profiler_enable(False)
        _lib.moe_profiler_reset()
    return rec, a.elapsed_time(b)


def _bf(*shape):
    import torch
    return torch.randn(*shape, device="cuda").bfloat16() * 0.05


def test_a_product_in_two_launches_counts_two():
    """A round of the 256 x 256 tiles is 65536 rows of 256 columns: the 64 rows left over are a launch of their own."""
    import torch
    import token_dispatch_grouped_amd as m
    T, d, F = 65600, 256, 128
    x, wgu, wdn = _bf(T, d), _bf(2 * F, d), _bf(d, F)
    h, a, y, dh, dx = (torch.empty(T, c, dtype=torch.bfloat16, device="cuda") for c in (2 * F, F, d, 2 * F, d))
    s = m.make_ffn_shape(T, d, F)
    rec, _ = _timed(lambda: m.moe_ffn_fwd(s, x, None, wgu, None, wdn, None, None, h, a, y, None, 0), 3)
    assert {k: n for k, (n, _) in rec.items()} == {"ffn_gateup_fwd": 6, "ffn_down_fwd": 6}, rec
    rec, _ = _timed(lambda: m.moe_ffn_dgrad(s, y, h, wgu, wdn, None, dh, dx), 3)
    assert {k: n for k, (n, _) in rec.items()} == {"ffn_down_dgrad": 3, "ffn_gateup_dgrad": 6}, rec


def test_few_tokens_in_8_bits_count_no_time_twice():
    """The gate/up product, the quantisation of its result and the down product are three launches one after the
    other, so that their times add up to no more than the time around the calls."""
    import torch
    import token_dispatch_grouped_amd as m
    T, d, F, calls = 144, 128, 65536, 20
    u8 = torch.uint8
    ops = []
    for rows, cols in ((T, d), (2 * F, d), (d, F)):
        q = torch.empty(rows, cols, dtype=u8, device="cuda")
        sc = torch.empty(rows, cols // 32, dtype=u8, device="cuda")
        m.moe_mx8_quantize(rows, cols, m.MOE_DTYPE_BF16, _bf(rows, cols), q, sc)
        ops += [q, sc]
    s = m.make_ffn_shape(T, d, F, m.MOE_DTYPE_MX8)
    n, _ = m.moe_ffn_workspace_size(s)
    ws, y = torch.empty(n, dtype=u8, device="cuda"), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    rec, ms = _timed(lambda: m.moe_ffn_fwd(s, *ops, None, None, None, y, ws, n), calls)
    print(f"[profiler] {rec} in {ms:.3f} ms", flush=True)
    assert {k: n for k, (n, _) in rec.items()} == {"ffn_gateup_fwd": calls, "mx8_quantize": calls,
                                                   "ffn_down_fwd": calls}, rec
    # a microsecond for the events' own resolution
    assert sum(t for _, t in rec.values()) <= ms + 1e-3, (rec, ms)
