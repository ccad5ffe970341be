"""The norm and the dense block as they are used: around the expert layer
(MoeLayer with norm_eps and shared_F), as a serving step in the 8-bit form,
captured in a graph, on two streams, and with offsets past 32 bits.

Layer runs are held to the layer's own bars (max|gpu - ref| / max|ref| <= 2e-2
in bf16, 1e-4 in fp32); the operators' element-wise bars are in their own
tests. The oracle routes on the normalised rows the GPU wrote, so that no
rounding decides a selection.
"""
import numpy as np
import pytest

import oracle
from tests.parity_util import TOL, assert_close, to_device, to_host64
from workloads import BF16, F32, bf16_bits_to_f32, f32_to_bf16_bits, make_inputs, small_workload, to_f64

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _dev(a, dtype):
    return to_device(a if dtype == F32 else f32_to_bf16_bits(a), dtype)


def _draw(rng, dtype, *shape, std=1.0, mean=0.0):
    a = rng.normal(mean, std, shape).astype(np.float32)
    return a if dtype == F32 else bf16_bits_to_f32(f32_to_bf16_bits(a))


def _round(dtype):
    return (lambda v: v.astype(np.float32).astype(np.float64)) if dtype == F32 else (
        lambda v: bf16_bits_to_f32(f32_to_bf16_bits(v.astype(np.float32))).astype(np.float64))


@pytest.mark.parametrize("dtype,shared_F,residual,router", [(BF16, 192, True, True), (BF16, 320, False, False),
                                                            (BF16, 0, True, False), (F32, 0, True, True)])
def test_layer_with_norm_and_shared_block(dtype, shared_F, residual, router):
    import torch
    import token_dispatch_grouped_amd as m
    from token_dispatch_grouped_amd.layer import MoeLayer
    w = small_workload(400, 256, 8, 2, 128, dtype, "router" if router else "zipf", seed=91, micro_T=(400, 0, 257))
    inp = make_inputs(w)
    W = inp["weights"]
    rng = np.random.default_rng(92)
    nw = _draw(rng, dtype, w.d, std=0.1, mean=1.0)
    sg, sd = _draw(rng, dtype, 2 * shared_F, w.d, std=0.05), _draw(rng, dtype, w.d, shared_F, std=0.05)
    layer = MoeLayer(400, w.d, w.E, w.k, w.F, m.MOE_DTYPE_BF16 if dtype == BF16 else m.MOE_DTYPE_F32, router=router,
                     norm_eps=EPS, shared_F=shared_F)
    f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    wgu, wdn = to_device(W["w_gu"], dtype), to_device(W["w_down"], dtype)
    wr = to_device(W["w_router"], dtype) if router else None
    bias = to_device(W["bias"], F32) if router else None
    nw_d = _dev(nw, dtype)
    grads = dict(dw_gu=f32(w.E, 2 * w.F, w.d), dw_down=f32(w.E, w.d, w.F), dnorm_w=f32(w.d))
    if router:
        grads["dw_router"] = f32(w.E, w.d)
    sh = sh_w = {}
    if shared_F:
        sh_w = dict(shared_w_gu=_dev(sg, dtype), shared_w_down=_dev(sd, dtype))
        sh = dict(dshared_w_gu=f32(2 * shared_F, w.d), dshared_w_down=f32(w.d, shared_F))
    want = {k: np.zeros(tuple(v.shape)) for k, v in {**grads, **sh}.items()}
    tol = TOL[dtype]
    w64 = {k: to_f64(W[k], dtype) for k in ("w_gu", "w_down")}
    for i, mb in enumerate(inp["micro"]):
        T = w.microbatches[i]
        print(f"[block] {dtype} microbatch {i}: T={T} shared_F={shared_F} residual={residual}", flush=True)
        res = _draw(rng, dtype, T, w.d, std=2.0) if residual else None
        dres = _draw(rng, dtype, T, w.d, std=0.5) if residual else None
        x, dout = to_device(mb["x"], dtype), to_device(mb["dout"], dtype)
        lg = None if router else to_device(np.ascontiguousarray(mb["logits"]), F32)
        sv = layer.forward(T, x, wgu, wdn, logits=lg, w_router=wr, bias=bias, norm_w=nw_d,
                           residual=None if res is None else _dev(res, dtype), **sh_w)
        g = layer.backward(T, dout, wgu, wdn, grads["dw_gu"], grads["dw_down"], x=None, w_router=wr,
                           dw_router=grads.get("dw_router"), norm_w=nw_d, dnorm_w=grads["dnorm_w"],
                           norm_r=None if residual else x, dres=None if dres is None else _dev(dres, dtype), **sh_w, **sh)
        torch.cuda.synchronize()
        if T == 0:
            continue
        r, rstd, u = oracle.rmsnorm_fwd(to_f64(mb["x"], dtype), nw, EPS, res, _round(dtype))
        if residual:
            assert_close("r", to_host64(sv.norm.r), r, 0.0)
        assert_close("u", to_host64(sv.norm.y), u, tol)
        u = to_host64(sv.norm.y)
        kw = dict(w_router=to_f64(W["w_router"], dtype), bias=W["bias"].astype(np.float64)) if router else dict(
            logits=mb["logits"].astype(np.float64))
        out, saved = oracle.layer_fwd(u, w64["w_gu"], w64["w_down"], w.k, **kw)
        do = to_f64(mb["dout"], dtype)
        og = oracle.layer_bwd(do, saved, w64["w_gu"], w64["w_down"], x=u if router else None,
                              w_router=kw.get("w_router"))
        du = og["dx"]
        if shared_F:
            sh64, sa64, out = oracle.dense_ffn_fwd(u, sg, sd, out)
            _, sdh, du = oracle.dense_ffn_dgrad(do, sh64, sg, sd, du)
            a, b = oracle.dense_ffn_wgrad(do, u, sa64, sdh)
            want["dshared_w_gu"] += a
            want["dshared_w_down"] += b
        dx, dnw = oracle.rmsnorm_bwd(du, r, nw, rstd, dres)
        want["dnorm_w"] += dnw
        for k in ("dw_gu", "dw_down") + (("dw_router",) if router else ()):
            want[k] += og[k]
        assert np.array_equal(sv.topk_idx.cpu().numpy(), saved["topk_idx"])
        assert_close("out", to_host64(sv.out), out, tol)
        assert_close("dx", to_host64(g["dx"]), dx, tol)
    for k, v in {**grads, **sh}.items():
        assert_close(k, to_host64(v), want[k], tol)


def _serving(rng, T, d, F):
    """Weights and rows of a serving step in the 8-bit form, and the step."""
    import torch
    import token_dispatch_grouped_amd as m
    from token_dispatch_grouped_amd.block import GatedFfn, RmsNorm, quantize_mx8
    norm = RmsNorm(T, d, eps=EPS, mx8=True)
    ffn = GatedFfn(T, d, F, m.MOE_DTYPE_MX8)
    s = dict(x=_dev(_draw(rng, BF16, T, d), BF16), res=_dev(_draw(rng, BF16, T, d), BF16),
             nw=_dev(_draw(rng, BF16, d, std=0.1, mean=1.0), BF16),
             wg=quantize_mx8(_dev(_draw(rng, BF16, 2 * F, d, std=0.05), BF16)),
             wd=quantize_mx8(_dev(_draw(rng, BF16, d, F, std=0.05), BF16)), norm=norm, ffn=ffn,
             out=torch.empty(T, d, dtype=torch.bfloat16, device="cuda"))

    def step(n=T):
        o = norm.forward(n, s["x"], s["nw"], s["res"])
        ffn.forward(n, o.y, s["wg"], s["wd"], add=norm.r, out=s["out"])  # r + FFN(norm(r)): the stream itself
        return o
    return s, step


@pytest.mark.parametrize("T,d,F", [(1, 2048, 1408), (37, 512, 384), (300, 256, 640)])
def test_serving_step_in_8_bits(T, d, F):
    import torch
    rng = np.random.default_rng(T)
    s, step = _serving(rng, T, d, F)
    o = step()
    torch.cuda.synchronize()
    r, _, _ = oracle.rmsnorm_fwd(to_host64(s["x"]), to_host64(s["nw"]), EPS, to_host64(s["res"]), _round(BF16))
    assert_close("r", to_host64(o.r), r, 0.0)

    def quantized(a):
        q, S = oracle.mx8_quantize(a)
        return q * np.repeat(S, 32, axis=1)
    xv, gv, dv = (m.values().double().cpu().numpy() for m in (o.y, s["wg"], s["wd"]))
    _, _, y = oracle.dense_ffn_fwd(xv, gv, dv, r, quantized)
    assert_close("out", to_host64(s["out"]), y, TOL[BF16])
    # fewer rows in the same objects, and none
    s["out"].fill_(float("nan"))
    if T > 1:
        step(T - 1)
        torch.cuda.synchronize()
        assert torch.isfinite(s["out"][:T - 1].float()).all() and torch.isnan(s["out"][T - 1].float()).all()
    step(0)


def _train(rng, T, d, F):
    import torch
    from token_dispatch_grouped_amd.block import GatedFfn, RmsNorm
    norm, ffn = RmsNorm(T, d, eps=EPS), GatedFfn(T, d, F)
    b = {k: _dev(_draw(rng, BF16, T, d), BF16) for k in ("x", "res", "dy", "dres")}
    b.update(nw=_dev(_draw(rng, BF16, d, std=0.1, mean=1.0), BF16), wg=_dev(_draw(rng, BF16, 2 * F, d, std=0.05), BF16),
             wd=_dev(_draw(rng, BF16, d, F, std=0.05), BF16))
    z = dict(dnw=torch.zeros(d, device="cuda"), dwg=torch.zeros(2 * F, d, device="cuda"),
             dwd=torch.zeros(d, F, device="cuda"))

    def step():
        o = norm.forward(T, b["x"], b["nw"], b["res"])
        y = ffn.forward(T, o.y, b["wg"], b["wd"], add=o.r)
        du = ffn.dgrad(T, b["dy"], b["wg"], b["wd"])
        ffn.wgrad(T, b["dy"], o.y, z["dwg"], z["dwd"])
        dx = norm.backward(T, du, o.r, b["nw"], z["dnw"], dres=b["dres"])
        return dict(r=o.r, u=o.y, y=y, dx=dx, **z)
    return step, z


def _snap(out):
    import torch
    torch.cuda.synchronize()
    return {k: v.clone() for k, v in out.items()}


def test_graph_replays_bitwise():
    """Serving and training steps in one graph, three replays, the program's own eager work in between."""
    import torch
    rng = np.random.default_rng(5)
    step, z = _train(rng, 1500, 512, 320)
    other, _ = _train(rng, 333, 256, 192)
    few, few_step = _serving(rng, 9, 512, 256)
    many, many_step = _serving(rng, 400, 256, 256)

    def all_steps():
        few_step()
        many_step()
        return dict(step(), few=few["out"], many=many["out"])

    def poison(out):
        for k, v in out.items():
            v.zero_() if k in z else v.fill_(float("nan"))
        torch.cuda.synchronize()
    ref = _snap(all_steps())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = all_steps()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = all_steps()
    for rep in range(3):
        poison(out)
        other()
        torch.cuda.synchronize()
        g.replay()
        got = _snap(out)
        for k in ref:
            assert torch.equal(got[k], ref[k]), f"replay {rep}: {k}"


def test_two_streams_without_synchronisation():
    """Two programs with buffers of their own, interleaved on two streams, give their sequential bits."""
    import torch
    rng = np.random.default_rng(6)
    progs = [_train(rng, 900, 384, 256), _train(rng, 2500, 256, 640)]
    want = []
    for step, z in progs:
        for v in z.values():
            v.zero_()
        for _ in range(3):
            out = step()
        want.append(_snap(out))
        for v in z.values():
            v.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in progs]
    outs = [None, None]
    for _ in range(3):
        for i, (step, _) in enumerate(progs):
            with torch.cuda.stream(streams[i]):
                outs[i] = step()
    for i in range(2):
        got = _snap(outs[i])
        for k, v in want[i].items():
            assert torch.equal(got[k], v), (i, k)


def test_memory_made_for_a_call_belongs_to_its_stream():
    """The current stream is behind: it still writes into memory freed on it when a call on another stream makes its
    output, which must not be that memory."""
    import torch
    from token_dispatch_grouped_amd.block import RmsNorm, quantize_mx8
    rng = np.random.default_rng(11)
    T, d = 2048, 1024
    x, w = _dev(_draw(rng, BF16, T, d), BF16), _dev(_draw(rng, BF16, d, std=0.1, mean=1.0), BF16)
    dw = torch.zeros(d, device="cuda")
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")

    def behind(nbytes):
        """Keeps the current stream busy, then fills nbytes of memory that is freed at once."""
        b = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        for _ in range(20):
            torch.mm(busy, busy, out=busy_out)
        b.fill_(0x55)
    busy_out = torch.empty_like(busy)
    want = quantize_mx8(x)
    ref = RmsNorm(T, d)
    ref.forward(T, x, w)
    want_dx = ref.backward(T, x, x, w, dw)
    norm = RmsNorm(T, d)
    norm.forward(T, x, w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for nbytes, call in ((T * d, lambda: quantize_mx8(x, stream=side.cuda_stream)),
                         (T * d * 2, lambda: norm.backward(T, x, x, w, dw, stream=side.cuda_stream))):
        behind(nbytes)
        got = call()
        torch.cuda.synchronize()
        if isinstance(got, torch.Tensor):
            assert torch.equal(got, want_dx)
        else:
            assert torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8))
            assert torch.equal(got.scale.view(torch.uint8), want.scale.view(torch.uint8))


def test_offsets_past_32_bits():
    """2.2 billion elements in a tensor: the last rows equal the same rows computed alone."""
    import torch
    import token_dispatch_grouped_amd as m
    bf = torch.bfloat16
    T, d, n = 1_100_000, 2048, 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, d, generator=gen, device="cuda", dtype=bf)
    w = torch.randn(d, generator=gen, device="cuda", dtype=bf)

    def norm(x, mx8):
        rows = x.shape[0]
        s = m.make_norm_shape(rows, d, m.MOE_DTYPE_BF16)
        y = torch.empty(rows, d, dtype=torch.uint8 if mx8 else bf, device="cuda")
        ys = torch.empty(rows, d // 32, dtype=torch.uint8, device="cuda") if mx8 else None
        rstd = torch.empty(rows, device="cuda")
        m.moe_rmsnorm_fwd(s, x, None, w, None, y, ys, rstd)
        return y, ys, rstd
    print("[offsets] norm", flush=True)
    tail = x[-n:].clone()
    for mx8 in (False, True):
        (y, ys, rstd), (ty, tys, trstd) = norm(x, mx8), norm(tail, mx8)
        # rstd: another split of the row over threads, so another order of its sum
        assert torch.allclose(rstd[-n:], trstd, rtol=1e-5, atol=0)
        if not mx8:
            assert torch.allclose(y[-n:].float(), ty.float(), rtol=2 ** -7, atol=0)  # a bf16 step
        else:
            assert (ys[-n:].int() - tys.int()).abs().max() <= 1
            q, S = m.moe_mx8_quantize, torch.empty_like(ys)
            q(T, d, m.MOE_DTYPE_BF16, x, y, S)
            q(n, d, m.MOE_DTYPE_BF16, tail, ty, tys)
            assert torch.equal(y[-n:], ty) and torch.equal(S[-n:], tys)
    del y, ys
    print("[offsets] norm backward", flush=True)
    s = m.make_norm_shape(T, d, m.MOE_DTYPE_BF16, 1e-6, m.MOE_NORM_OVERWRITE_DW)
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(m.moe_rmsnorm_workspace_size(s), dtype=torch.uint8, device="cuda")
    m.moe_rmsnorm_bwd(s, x, x, w, rstd, None, dx, dw, ws, ws.numel())
    want, _ = oracle.rmsnorm_bwd(to_host64(tail), to_host64(tail), to_host64(w), to_host64(rstd[-n:]))
    assert_close("dx", to_host64(dx[-n:]), want, TOL[BF16])
    del x, dx, ws
    torch.cuda.empty_cache()

    d, F = 64, 1024  # h and dh: [T, 2F], 2.25 billion elements
    x, add = (torch.randn(T, d, generator=gen, device="cuda", dtype=bf) for _ in range(2))
    wg, wd = (torch.randn(*sh, generator=gen, device="cuda", dtype=bf) * 0.05 for sh in ((2 * F, d), (d, F)))
    s = m.make_ffn_shape(T, d, F, m.MOE_DTYPE_BF16, m.MOE_FFN_OVERWRITE_DW)
    h, a, y = (torch.empty(T, c, dtype=bf, device="cuda") for c in (2 * F, F, d))
    print("[offsets] block", flush=True)
    m.moe_ffn_fwd(s, x, None, wg, None, wd, None, add, h, a, y, None, 0)
    tx, tadd = to_host64(x[-n:]), to_host64(add[-n:])
    h64, a64, y64 = oracle.dense_ffn_fwd(tx, to_host64(wg), to_host64(wd), tadd)
    for name, got, want in (("h", h, h64), ("a", a, a64), ("y", y, y64)):
        assert_close(name, to_host64(got[-n:]), want, TOL[BF16])
    dh, dx = torch.empty_like(h), torch.empty_like(x)
    m.moe_ffn_dgrad(s, add, h, wg, wd, x, dh, dx)
    _, dh64, dx64 = oracle.dense_ffn_dgrad(tadd, h64, to_host64(wg), to_host64(wd), tx)
    assert_close("dh", to_host64(dh[-n:]), dh64, TOL[BF16])
    assert_close("dx", to_host64(dx[-n:]), dx64, TOL[BF16])
    # the weight gradient of rows that are zero but for the last: only that row counts
    _, nbytes = m.moe_ffn_workspace_size(s)
    ws = torch.empty(max(1, nbytes), dtype=torch.uint8, device="cuda")
    dh[:-n] = 0
    add[:-n] = 0
    dwg, dwd = torch.empty(2 * F, d, device="cuda"), torch.empty(d, F, device="cuda")
    m.moe_ffn_wgrad(s, add, x, a, dh, dwg, dwd, ws, nbytes)
    g64, d64 = oracle.dense_ffn_wgrad(tadd, tx, to_host64(a[-n:]), to_host64(dh[-n:]))
    assert_close("dw_gu", to_host64(dwg), g64, TOL[F32])
    assert_close("dw_down", to_host64(dwd), d64, TOL[F32])
