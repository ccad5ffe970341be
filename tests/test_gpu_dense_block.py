"""The layer norm, the dense products and the orthogonalised update as they are
used: an ungated block in the residual stream over several microbatches, its
backward pass and its weights' update; the experts' update after a layer's
backward pass; one token; captured in a graph; on two streams and from two
threads.

Chains are held to the layer's own bars (max|gpu - ref| / max|ref| <= 2e-2 in
bf16); the operators' element-wise bars are in their own tests.
"""
import threading

import numpy as np
import pytest

import oracle
from tests.parity_util import TOL, assert_close
from workloads import BF16

pytestmark = pytest.mark.gpu
EPS = 1e-5
D, F = 256, 704


def _rand(gen, *shape, std=1.0, mean=0.0):
    import torch
    return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).bfloat16()


def _h(t):
    return t.double().cpu().numpy()


class Block:
    """x -> r = x + res, r + W2 gelu(W1 LN(r) + b1) + b2, and back."""

    def __init__(self, T_max, seed=1, device="cuda"):
        import torch
        import token_dispatch_grouped_amd as m
        from token_dispatch_grouped_amd.block import LayerNorm, Linear
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.norm = LayerNorm(T_max, D, eps=EPS)
        self.up, self.down = Linear(T_max, D, F, m.MOE_ACT_GELU), Linear(T_max, F, D)
        self.p = dict(g=_rand(gen, D, std=0.1, mean=1.0), b=_rand(gen, D, std=0.1), w1=_rand(gen, F, D, std=D ** -0.5),
                      b1=_rand(gen, F, std=0.1), w2=_rand(gen, D, F, std=F ** -0.5), b2=_rand(gen, D, std=0.1))
        self.grad = {k: torch.zeros(v.shape, device="cuda") for k, v in self.p.items()}

    def step(self, T, x, res, dout, stream=None):
        p, g = self.p, self.grad
        n = self.norm.forward(T, x, p["g"], p["b"], residual=res, stream=stream)
        a = self.up.forward(T, n.y, p["w1"], p["b1"], stream=stream)
        out = self.down.forward(T, a, p["w2"], p["b2"], residual=n.r, stream=stream)
        dz1 = self.down.dgrad(T, dout, p["w2"], below=self.up, stream=stream)
        dn = self.up.dgrad(T, dz1, p["w1"], stream=stream)
        self.down.wgrad(T, dout, a, g["w2"], g["b2"], stream=stream)
        self.up.wgrad(T, dz1, n.y, g["w1"], g["b1"], stream=stream)
        dx = self.norm.backward(T, dn, n.r, p["g"], g["g"], g["b"], dres=dout, stream=stream)
        return out, dx

    def reference(self, x, res, dout):
        p = {k: _h(v) for k, v in self.p.items()}
        import torch
        round_r = lambda v: torch.from_numpy(v).float().bfloat16().double().numpy()  # noqa: E731
        r, mean, rstd, _, y = oracle.layernorm_fwd(_h(x), p["g"], p["b"], EPS, _h(res), round_r)
        z1, a = oracle.linear_fwd(y, p["w1"], p["b1"], None, "gelu")
        _, out = oracle.linear_fwd(a, p["w2"], p["b2"], r)
        dy = _h(dout)
        dz1 = oracle.linear_dgrad(dy, p["w2"], z1, "gelu")
        dw2, db2 = oracle.linear_wgrad(dy, a)
        dw1, db1 = oracle.linear_wgrad(dz1, y)
        dx, dg, db = oracle.layernorm_bwd(oracle.linear_dgrad(dz1, p["w1"]), r, p["g"], mean, rstd, dy)
        return out, dx, dict(g=dg, b=db, w1=dw1, b1=db1, w2=dw2, b2=db2)


def _batch(T, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _rand(gen, T, D), _rand(gen, T, D, std=2.0), _rand(gen, T, D, std=0.1)


def test_a_block_over_microbatches_and_its_update():
    """Gradients accumulate over microbatches, an empty one among them; then the weights are updated, and the next
    forward runs on the new ones."""
    import torch
    from token_dispatch_grouped_amd.optim import ExpertMuon
    blk = Block(700)
    opt = ExpertMuon([blk.p["w1"], blk.p["w2"]], lr=0.02, weight_decay=0.1, match_rms=0.2)
    total = {k: 0 for k in blk.grad}
    for T in (700, 0, 1, 333):
        x, res, dout = _batch(T, 10 + T)
        out, dx = blk.step(T, x, res, dout)
        if T == 0:
            continue
        out64, dx64, grads = blk.reference(x, res, dout)
        assert_close("out", _h(out), out64, TOL[BF16])
        assert_close("dx", _h(dx), dx64, TOL[BF16])
        for k in total:
            total[k] = total[k] + grads[k]
    for k in total:
        assert_close("d" + k, _h(blk.grad[k]), total[k], TOL[BF16])
    old = [_h(v) for v in opt.master]
    grads = [blk.grad["w1"], blk.grad["w2"]]
    want = [oracle.muon_step(w, _h(g) / 4, 0 * w, 0.02, 0.95, 0.1, 0.2 * np.sqrt(max(w.shape)))[0] for w, g in zip(old, grads)]
    opt.step(grads, grad_scale=0.25)
    torch.cuda.synchronize()
    for i, k in enumerate(("w1", "w2")):
        assert_close(k, _h(opt.master[i]) - old[i], want[i] - old[i], 1e-2)
        assert torch.equal(blk.p[k], opt.master[i].bfloat16()) and not blk.grad[k].any()
    x, res, dout = _batch(64, 5)
    out, _ = blk.step(64, x, res, dout)
    assert_close("out on the new weights", _h(out), blk.reference(x, res, dout)[0], TOL[BF16])


def test_one_token_at_a_time():
    """Rows one by one, as a serving loop has them, against the same rows together: the products' sums run in another
    order, so each result may fall one rounding to the other side, which the layer's bar covers."""
    import token_dispatch_grouped_amd as m
    from token_dispatch_grouped_amd.block import LayerNorm, Linear
    blk = Block(32)
    x, res, dout = _batch(32, 7)
    out, _ = blk.step(32, x, res, dout)
    out = out.clone()
    norm, up, down = LayerNorm(1, D, eps=EPS), Linear(1, D, F, m.MOE_ACT_GELU, save=False), Linear(1, F, D, save=False)
    p = blk.p
    for t in range(32):
        n = norm.forward(1, x[t:t + 1], p["g"], p["b"], residual=res[t:t + 1])
        stream = n.r.clone()
        y = down.forward(1, up.forward(1, n.y, p["w1"], p["b1"]), p["w2"], p["b2"], residual=stream, out=stream)
        assert y.data_ptr() == stream.data_ptr()
        assert_close(f"token {t}", _h(y[0]), _h(out[t]), TOL[BF16])


def test_the_experts_update_after_a_layers_backward():
    import torch
    import token_dispatch_grouped_amd as m
    from token_dispatch_grouped_amd.layer import MoeLayer
    from token_dispatch_grouped_amd.optim import ExpertMuon
    from tests.parity_util import to_device
    from workloads import make_inputs, small_workload
    w = small_workload(400, 128, 8, 2, 192, BF16, "zipf", seed=23, n_empty=1)
    inp = make_inputs(w)
    mb, W = inp["micro"][0], inp["weights"]
    layer = MoeLayer(w.T, w.d, w.E, w.k, w.F, m.MOE_DTYPE_BF16)
    wgu, wdn = to_device(W["w_gu"], BF16), to_device(W["w_down"], BF16)
    x, dout, lg = to_device(mb["x"], BF16), to_device(mb["dout"], BF16), to_device(mb["logits"], "f32")
    dgu, ddn = torch.zeros(w.E, 2 * w.F, w.d, device="cuda"), torch.zeros(w.E, w.d, w.F, device="cuda")
    layer.forward(w.T, x, wgu, wdn, logits=lg)
    layer.backward(w.T, dout, wgu, wdn, dgu, ddn)
    opt = ExpertMuon([wgu, wdn], lr=0.05, momentum=0.9, nesterov=False, parts=[2, 1])
    old = [_h(v) for v in opt.master]
    grads = [_h(dgu), _h(ddn)]
    opt.step([dgu, ddn])
    torch.cuda.synchronize()
    for i, (rows, cols) in enumerate(((w.F, w.d), (w.d, w.F))):
        scale = np.sqrt(max(1.0, rows / cols))
        p, g, new = (v.reshape(-1, rows, cols) for v in (old[i], grads[i], _h(opt.master[i])))
        for e in range(p.shape[0]):
            want = oracle.muon_step(p[e], g[e], 0 * g[e], 0.05, 0.9, 0.0, scale, nesterov=False)[0]
            assert_close(f"{i}.{e}", new[e] - p[e], want - p[e], 1e-2)  # an expert without tokens: exactly zero
    assert torch.equal(wgu, opt.master[0].bfloat16()) and torch.equal(wdn, opt.master[1].bfloat16())
    assert not dgu.any() and not ddn.any()


def _state(blk, opt):
    return [blk.grad[k] for k in blk.grad] + opt.master + opt.momenta + [blk.p["w1"], blk.p["w2"]]


def test_captured_and_replayed():
    """A training step of the block and its update as one graph, replayed with other eager work between: every replay has
    the bits of the eager step."""
    import torch
    from token_dispatch_grouped_amd.optim import ExpertMuon
    T = 333
    x, res, dout = _batch(T, 3)

    def fresh():
        blk = Block(T)
        return blk, ExpertMuon([blk.p["w1"], blk.p["w2"]], lr=0.02)

    def step(blk, opt):
        out, dx = blk.step(T, x, res, dout)
        opt.step([blk.grad["w1"], blk.grad["w2"]])
        return out, dx

    blk, opt = fresh()
    eager = []
    for _ in range(3):
        out, dx = step(blk, opt)
        torch.cuda.synchronize()
        eager.append([v.clone() for v in [out, dx] + _state(blk, opt)])
    blk, opt = fresh()
    other, _ = fresh()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):  # the first backward happens in here
        out, dx = step(blk, opt)
    for i in range(3):
        out.fill_(float("nan"))
        dx.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([out, dx] + _state(blk, opt), eager[i]):
            assert torch.equal(a, b)
        other.step(T, x, res, dout)
        torch.cuda.synchronize()


def test_two_streams_and_two_threads():
    import torch
    from token_dispatch_grouped_amd.optim import ExpertMuon, Orthogonalizer
    T = 333
    data = [_batch(T, 31), _batch(T, 32)]

    def run(i, stream):
        with torch.cuda.stream(stream):
            blk = Block(T, seed=i)
            opt = ExpertMuon([blk.p["w1"], blk.p["w2"]], lr=0.02)
            orth = Orthogonalizer(1, F, D)
            for _ in range(3):
                out, dx = blk.step(T, *data[i])
                o = orth.forward(1, blk.grad["w1"].view(1, F, D))
                opt.step([blk.grad["w1"], blk.grad["w2"]])
            return [v.clone() for v in [out, dx, o] + _state(blk, opt)]

    want = [run(i, torch.cuda.current_stream()) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [run(i, streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    threaded = [None, None]

    def work(i):
        threaded[i] = run(i, streams[i])
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, threaded):
        for u, v, w in zip(a, b, c):
            assert torch.equal(u, v) and torch.equal(u, w)


def test_another_stream_by_its_handle():
    """Calls ordered on a stream that is not the current one, buffers they make included."""
    import torch
    T = 200
    x, res, dout = _batch(T, 41)
    blk = Block(T)
    want = [v.clone() for v in blk.step(T, x, res, dout)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    blk2 = Block(T)
    torch.cuda.synchronize()
    got = blk2.step(T, x, res, dout, stream=side.cuda_stream)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_the_event_timer_has_one_record_a_launch():
    import torch
    import token_dispatch_grouped_amd as m
    from token_dispatch_grouped_amd import _lib

    def records(call, calls=3):
        call()
        torch.cuda.synchronize()
        _lib.moe_profiler_reset()
        _lib.moe_profiler_enable(True)
        try:
            for _ in range(calls):
                call()
            torch.cuda.synchronize()
            return {k: n for k, (n, _) in _lib.moe_profiler_read_all().items()}
        finally:
            _lib.moe_profiler_enable(False)
            _lib.moe_profiler_reset()

    # sums of X X^T in slices and their join
    x = torch.randn(1, 1500, 4200, device="cuda")
    s = m.make_orth_shape(1, 1500, 4200)
    ws = torch.empty(m.moe_orthogonalize_workspace_size(s), dtype=torch.uint8, device="cuda")
    o = torch.empty(1, 1500, 4200, dtype=torch.bfloat16, device="cuda")
    rec = records(lambda: m.moe_orthogonalize(s, x, o, ws, ws.numel()))
    assert rec == {"orth_norm": 3, "orth_prep": 3, "orth_gram": 15, "orth_gram_sum": 15, "orth_poly": 15, "orth_step": 12,
                   "orth_last": 3}, rec
    # a bias gradient in a pass of its own
    T, K, N = 300, 64, 64
    dz, x = (torch.randn(T, c, device="cuda").bfloat16() for c in (N, K))
    dw, db = torch.zeros(N, K, device="cuda"), torch.zeros(N, device="cuda")
    s = m.make_linear_shape(T, K, N)
    ws = torch.empty(m.moe_linear_workspace_size(s), dtype=torch.uint8, device="cuda")
    rec = records(lambda: m.moe_linear_wgrad(s, dz, x, dw, db, ws, ws.numel()))
    assert rec["linear_wgrad"] == rec["linear_db"] == rec["linear_db_reduce"] == 3, rec
