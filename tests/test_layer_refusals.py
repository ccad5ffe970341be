"""A layer with the norm in front and the shared block beside it refuses a
wrong tensor before it calls anything (CPU only, the library's calls counted):
the weight gradients accumulate, so a refusal halfway would leave a part of
the step in them.
"""
import contextlib

import pytest

torch = pytest.importorskip("torch")
from token_dispatch_grouped_amd import _lib  # noqa: E402
from token_dispatch_grouped_amd import block  # noqa: E402
from token_dispatch_grouped_amd.layer import MoeLayer  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
T, D, E, K, F, SF = 8, 128, 4, 2, 128, 64


def t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in dir(_lib):
        if name.startswith("moe_") and callable(getattr(_lib, name)) and not name.endswith(("_size", "_shape", "_config")):
            monkeypatch.setattr(_lib, name, lambda *a, _n=name, **k: made.append(_n))
    monkeypatch.setattr(block, "_on", lambda device: contextlib.nullcontext())
    return made


def _weights():
    return dict(norm_w=t(D), shared_w_gu=t(2 * SF, D), shared_w_down=t(D, SF))


def _grads():
    return dict(dnorm_w=t(D, dtype=F32), dshared_w_gu=t(2 * SF, D, dtype=F32), dshared_w_down=t(D, SF, dtype=F32))


W = (t(E, 2 * F, D), t(E, D, F))
DW = (t(E, 2 * F, D, dtype=F32), t(E, D, F, dtype=F32))


@pytest.mark.parametrize("bad", [dict(norm_w=t(D, dtype=F32)), dict(residual=t(T, 64)), dict(shared_w_gu=t(SF, D)),
                                 dict(shared_w_down=t(SF, D)), dict(x=t(T - 1, D)), dict(x=t(T, D, dtype=F32))])
def test_forward(calls, bad):
    full = MoeLayer(T, D, E, K, F, norm_eps=1e-6, shared_F=SF, device="cpu")
    args = {**dict(x=t(T, D)), **_weights(), **bad}
    with pytest.raises(ValueError, match=next(iter(bad)).replace("norm_w", "weight").replace("shared_", "")):
        full.forward(T, args.pop("x"), *W, logits=t(T, E, dtype=F32), **args)
    assert calls == []


@pytest.mark.parametrize("bad", [dict(dout=t(T, D, dtype=F32)), dict(dnorm_w=t(D)), dict(dnorm_w=t(64, dtype=F32)),
                                 dict(norm_w=t(64)), dict(dres=t(T - 1, D)), dict(shared_w_gu=t(SF, D)),
                                 dict(dshared_w_gu=t(2 * SF, D)), dict(dshared_w_down=t(SF, D, dtype=F32)),
                                 dict(norm_r=t(T, D, dtype=F32))])
def test_backward(calls, bad):
    full = MoeLayer(T, D, E, K, F, norm_eps=1e-6, shared_F=SF, device="cpu")
    args = {**dict(dout=t(T, D), norm_r=t(T, D)), **_weights(), **_grads(), **bad}
    with pytest.raises(ValueError):
        full.backward(T, args.pop("dout"), *W, *DW, **args)
    assert calls == []


def test_backward_without_the_norm_checks_x(calls):
    beside = MoeLayer(T, D, E, K, F, shared_F=SF, device="cpu")
    args = {k: v for k, v in {**_weights(), **_grads()}.items() if "norm" not in k}
    with pytest.raises(ValueError, match="x"):
        beside.backward(T, t(T, D), *W, *DW, x=t(T, 64), **args)
    assert calls == []


def test_right_tensors_are_taken(calls):
    full = MoeLayer(T, D, E, K, F, norm_eps=1e-6, shared_F=SF, device="cpu")
    full.forward(T, t(T, D), *W, logits=t(T, E, dtype=F32), **_weights(), residual=t(T, D))
    assert calls[0] == "moe_rmsnorm_fwd" and calls[-1] == "moe_ffn_fwd"
    del calls[:]
    full.backward(T, t(T, D), *W, *DW, **_weights(), **_grads(), dres=t(T, D))
    assert calls[-3:] == ["moe_ffn_dgrad", "moe_ffn_wgrad", "moe_rmsnorm_bwd"]


def test_buffers_that_a_step_writes_before_it_reads_them(calls):
    """One layer for every depth: the gradient buffer of the step before is written by the routed experts' backward
    before the shared block reads dout and the norm reads dres, and out before the shared block reads x."""
    full = MoeLayer(T, D, E, K, F, norm_eps=1e-6, shared_F=SF, device="cpu")
    full.norm_summed = True
    both = {**_weights(), **_grads()}
    for word, args in (("dout", dict(dout=full.dx)), ("dout", dict(dout=full.dx[1:T])), ("dres", dict(dout=t(T, D), dres=full.dx))):
        T1 = min(T, args["dout"].shape[0])
        with pytest.raises(ValueError, match=word):
            full.backward(T1, args.pop("dout"), *W, *DW, **both, **args)
    full.norm_summed = False
    with pytest.raises(ValueError, match="norm_r"):  # the forward wrote its out over it
        full.backward(T, t(T, D), *W, *DW, norm_r=full.out, **both)
    normed = MoeLayer(T, D, E, K, F, norm_eps=1e-6, device="cpu")
    normed.norm_summed = True
    only = {k: v for k, v in both.items() if "shared" not in k}
    with pytest.raises(ValueError, match="dres"):
        normed.backward(T, t(T, D), *W, *DW, dres=normed.dx, **only)
    beside = MoeLayer(T, D, E, K, F, shared_F=SF, device="cpu")
    w = {k: v for k, v in _weights().items() if "norm" not in k}
    g = {k: v for k, v in _grads().items() if "norm" not in k}
    with pytest.raises(ValueError, match="x"):
        beside.forward(T, beside.out, *W, logits=t(T, E, dtype=F32), **w)
    with pytest.raises(ValueError, match="dout"):
        beside.backward(T, beside.dx, *W, *DW, x=t(T, D), **w, **g)
    with pytest.raises(ValueError, match="x"):
        beside.backward(T, t(T, D), *W, *DW, x=beside.out, **w, **g)
    assert calls == []
    # read before they are written: taken
    normed.backward(T, normed.dx, *W, *DW, dres=t(T, D), **only)
    full.forward(T, full.out, *W, logits=t(T, E, dtype=F32), residual=full.norm.r, **_weights())
    plain = MoeLayer(T, D, E, K, F, device="cpu")
    plain.forward(T, plain.out, *W, logits=t(T, E, dtype=F32))
    plain.backward(T, plain.dx, *W, *DW)


def test_block_buffers_that_the_weight_gradient_reads_later(calls):
    f = block.GatedFfn(T, D, SF, device="cpu")
    wg, wd = t(2 * SF, D), t(D, SF)
    with pytest.raises(ValueError, match="x"):
        f.forward(T, f.y, wg, wd)
    with pytest.raises(ValueError, match="dy"):
        f.dgrad(T, f.dx, wg, wd)
    x = t(T, D)
    with pytest.raises(ValueError, match="x"):
        f.forward(T, x, wg, wd, out=x)
    with pytest.raises(ValueError, match="dy"):
        f.dgrad(T, x, wg, wd, out=x)
    assert calls == []
    f.forward(T, x, wg, wd, add=f.y)
    f.dgrad(T, x, wg, wd, add=f.dx)
    two = t(2 * T, D)
    f.forward(T, two[:T], wg, wd, out=two[T:])  # side by side
    serving = block.GatedFfn(T, D, SF, save=False, device="cpu")
    serving.forward(T, serving.y, wg, wd)  # no weight gradient follows
    n = block.RmsNorm(T, D, device="cpu")
    n.dx = t(T, D)
    n.backward(T, x, x, t(D), t(D, dtype=F32), dres=n.dx)  # in place, as the library allows
