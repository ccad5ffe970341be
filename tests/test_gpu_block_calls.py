"""Calls of the norm, the quantiser, the dense block and the layer around them
that the operators' own tests do not make: the default stream by its handle,
memory made inside a capture, two host threads, empty microbatches that
overwrite, and the layer's other modes with the norm in front.
"""
import threading

import numpy as np
import pytest

import oracle
from tests.parity_util import TOL, assert_close, to_device, to_host64
from tests.test_gpu_block import EPS, _dev, _draw, _round, _snap, _train
from workloads import BF16, F32, make_inputs, small_workload, to_f64

pytestmark = pytest.mark.gpu


def test_the_default_stream_by_its_handle():
    import torch
    from token_dispatch_grouped_amd.block import GatedFfn, RmsNorm, quantize_mx8
    rng = np.random.default_rng(21)
    T, d, F = 70, 256, 192
    x, w = _dev(_draw(rng, BF16, T, d), BF16), _dev(_draw(rng, BF16, d, std=0.1, mean=1.0), BF16)
    wg, wd = _dev(_draw(rng, BF16, 2 * F, d, std=0.05), BF16), _dev(_draw(rng, BF16, d, F, std=0.05), BF16)
    got = []
    for stream in (None, 0):
        norm, ffn, dw = RmsNorm(T, d), GatedFfn(T, d, F), torch.zeros(d, device="cuda")
        o = norm.forward(T, x, w, residual=x, stream=stream)
        y = ffn.forward(T, o.y, wg, wd, add=o.r, stream=stream)
        dx = norm.backward(T, ffn.dgrad(T, y, wg, wd, stream=stream), o.r, w, dw, stream=stream)
        q = quantize_mx8(x, stream=stream)
        torch.cuda.synchronize()
        got.append([t.clone() for t in (o.r, o.y, y, dx, dw, q.q.view(torch.uint8), q.scale.view(torch.uint8))])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_a_first_backward_inside_a_capture():
    """The norm's gradient buffer is made by its first backward, here in the graph's own memory."""
    import torch
    from token_dispatch_grouped_amd.block import RmsNorm, quantize_mx8
    rng = np.random.default_rng(22)
    T, d = 300, 512
    x, w = _dev(_draw(rng, BF16, T, d), BF16), _dev(_draw(rng, BF16, d, std=0.1, mean=1.0), BF16)
    ref, dw = RmsNorm(T, d), torch.zeros(d, device="cuda")
    ref.forward(T, x, w)
    want = ref.backward(T, x, x, w, dw, overwrite=True).clone()
    want_q = quantize_mx8(x)
    norm, dw2 = RmsNorm(T, d), torch.zeros(d, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm.forward(T, x, w)
        dx = norm.backward(T, x, x, w, dw2, overwrite=True)
        q = quantize_mx8(x)
    for _ in range(3):
        for t in (dx, dw2):
            t.fill_(float("nan"))
        g.replay()
        ref.backward(T, x, x, w, dw, overwrite=True)  # the program's own work in between
        torch.cuda.synchronize()
        assert torch.equal(dx, want) and torch.equal(dw2, dw)
        assert torch.equal(q.q.view(torch.uint8), want_q.q.view(torch.uint8))
    del g
    again = norm.backward(T, x, x, w, dw2, overwrite=True)  # the buffer outlives the graph
    torch.cuda.synchronize()
    assert torch.equal(again, want)


def test_two_host_threads():
    """Two programs with buffers and streams of their own, called from two threads at once, give their own bits."""
    import torch
    rng = np.random.default_rng(23)
    progs = [_train(rng, 700, 384, 256), _train(rng, 1300, 256, 192)]
    want = []
    for step, z in progs:
        for v in z.values():
            v.zero_()
        for _ in range(5):
            out = step()
        want.append(_snap(out))
        for v in z.values():
            v.zero_()
    torch.cuda.synchronize()
    outs, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    outs[i] = progs[i][0]()
        except Exception as e:  # reported below, on the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        got = _snap(outs[i])
        for k, v in want[i].items():
            assert torch.equal(got[k], v), (i, k)


def test_empty_microbatches_overwrite_with_zeros():
    import torch
    from token_dispatch_grouped_amd.block import GatedFfn, RmsNorm
    T, d, F = 40, 128, 192
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w, wg, wd = torch.ones(T, d, **bf), torch.ones(d, **bf), torch.ones(2 * F, d, **bf), torch.ones(d, F, **bf)
    norm, ffn = RmsNorm(T, d), GatedFfn(T, d, F)
    dw, dgu, ddn = (torch.ones(*s, device="cuda") for s in ((d,), (2 * F, d), (d, F)))
    for overwrite in (False, True):
        o = norm.forward(0, x, w, residual=x)
        assert ffn.forward(0, o.y if o.y.shape[0] else x, wg, wd).shape == (0, d)
        ffn.dgrad(0, x, wg, wd)
        ffn.wgrad(0, x, x, dgu, ddn, overwrite=overwrite)
        norm.backward(0, x, x, w, dw, overwrite=overwrite)
        torch.cuda.synchronize()
        for t in (dw, dgu, ddn):
            assert (t == (0 if overwrite else 1)).all()


@pytest.mark.parametrize("dtype,mode", [(BF16, "recompute"), (BF16, "aux"), (F32, "recompute")])
def test_layer_modes_behind_the_norm(dtype, mode):
    """Recomputed activations and auxiliary losses with the norm in front: the same results as the plain layer on the
    normalised rows, and the norm's own gradient on top."""
    import torch
    import token_dispatch_grouped_amd as m
    from token_dispatch_grouped_amd.layer import MoeLayer
    w = small_workload(200, 128, 8, 2, 128, dtype, "zipf", seed=24)
    inp = make_inputs(w)
    W, mb = inp["weights"], inp["micro"][0]
    rng = np.random.default_rng(25)
    nw = _draw(rng, dtype, w.d, std=0.1, mean=1.0)
    res = _draw(rng, dtype, w.T, w.d, std=2.0)
    kw = dict(recompute=mode == "recompute", aux=(0.01, 0.001) if mode == "aux" else None)
    dt = m.MOE_DTYPE_BF16 if dtype == BF16 else m.MOE_DTYPE_F32
    layer = MoeLayer(w.T, w.d, w.E, w.k, w.F, dt, norm_eps=EPS, **kw)
    plain = MoeLayer(w.T, w.d, w.E, w.k, w.F, dt, **kw)
    x, dout, nw_d = to_device(mb["x"], dtype), to_device(mb["dout"], dtype), _dev(nw, dtype)
    wgu, wdn, lg = to_device(W["w_gu"], dtype), to_device(W["w_down"], dtype), to_device(mb["logits"], F32)
    g1, g2 = ([torch.zeros(*s, device="cuda") for s in ((w.E, 2 * w.F, w.d), (w.E, w.d, w.F))] for _ in range(2))
    dnw = torch.zeros(w.d, device="cuda")
    sv = layer.forward(w.T, x, wgu, wdn, logits=lg, norm_w=nw_d, residual=_dev(res, dtype))
    u = sv.norm.y.clone()
    got = layer.backward(w.T, dout, wgu, wdn, *g1, norm_w=nw_d, dnorm_w=dnw)
    ref_sv = plain.forward(w.T, u, wgu, wdn, logits=lg)
    ref = plain.backward(w.T, dout, wgu, wdn, *g2)
    torch.cuda.synchronize()
    assert torch.equal(sv.out, ref_sv.out) and torch.equal(got["dlogits"], ref["dlogits"])
    for a, b in zip(g1, g2):
        assert torch.equal(a, b)
    r, rstd, u64 = oracle.rmsnorm_fwd(to_f64(mb["x"], dtype), nw, EPS, res, _round(dtype))
    assert_close("u", to_host64(u), u64, TOL[dtype])
    dx, dnw64 = oracle.rmsnorm_bwd(to_host64(ref["dx"]), r, nw, rstd)
    assert_close("dx", to_host64(got["dx"]), dx, TOL[dtype])
    assert_close("dnorm_w", to_host64(dnw), dnw64, TOL[dtype])
