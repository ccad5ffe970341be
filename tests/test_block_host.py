"""RmsNorm, GatedFfn and MoeLayer's norm and shared block refuse wrong tensors
before anything is called (CPU only)."""
import pytest

torch = pytest.importorskip("torch")
import token_dispatch_grouped_amd as moe  # noqa: E402
from token_dispatch_grouped_amd import block  # noqa: E402
from token_dispatch_grouped_amd.layer import MoeLayer  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def test_norm_checks():
    n = block.RmsNorm(8, 128, device="cpu")
    x, w = t(8, 128), t(128)
    for bad in (t(8, 128, dtype=F32), t(7, 128), t(8, 64), t(128, 8).t(), t(2, 8, 128), None, 3):
        with pytest.raises(ValueError, match="x"):
            n.forward(8, bad, w)
    with pytest.raises(ValueError, match="weight"):
        n.forward(8, x, t(128, dtype=F32))
    with pytest.raises(ValueError, match="residual"):
        n.forward(8, x, w, residual=t(6, 128))
    for T in (-1, 9):
        with pytest.raises(ValueError, match="T ="):
            n.forward(T, x, w)
    with pytest.raises(ValueError, match="dw"):
        n.backward(8, x, x, w, t(128))
    with pytest.raises(ValueError, match="dres"):
        n.backward(8, x, x, w, t(128, dtype=F32), dres=t(8, 64))
    with pytest.raises(moe.MoeError):
        block.RmsNorm(8, 100, device="cpu")


def test_ffn_checks():
    f = block.GatedFfn(8, 128, 256, device="cpu")
    x, wg, wd = t(8, 128), t(512, 128), t(128, 256)
    for args, word in (((8, t(8, 64), wg, wd), "x"), ((8, x, t(256, 128), wd), "w_gu"), ((8, x, wg, t(256, 128)), "w_down"),
                       ((9, x, wg, wd), "T =")):
        with pytest.raises(ValueError, match=word):
            f.forward(*args)
    with pytest.raises(ValueError, match="add"):
        f.forward(8, x, wg, wd, add=t(8, 128, dtype=F32))
    with pytest.raises(ValueError, match="out"):
        f.forward(8, x, wg, wd, out=t(4, 128))
    with pytest.raises(ValueError, match="dw_gu"):
        f.wgrad(8, x, x, t(512, 128), t(128, 256, dtype=F32))
    for g in (block.GatedFfn(8, 128, 256, save=False, device="cpu"),
              block.GatedFfn(8, 128, 256, moe.MOE_DTYPE_MX8, device="cpu")):
        with pytest.raises(ValueError, match="backward"):
            g.dgrad(8, x, wg, wd)
        with pytest.raises(ValueError, match="backward"):
            g.wgrad(8, x, x, t(512, 128, dtype=F32), t(128, 256, dtype=F32))
    with pytest.raises(ValueError, match="Mx8"):
        g.forward(8, x, wg, wd)
    m = block.empty_mx8(8, 128, "cpu")
    with pytest.raises(ValueError, match="w_gu.q"):
        g.forward(8, m, m, m)
    with pytest.raises(ValueError, match="scale"):
        block._check_mx8("x", block.Mx8(m.q, m.scale.view(torch.uint8)), 8, (128,), torch.device("cpu"))
    with pytest.raises(moe.MoeError):
        block.GatedFfn(8, 128, 192, moe.MOE_DTYPE_MX8, device="cpu")


def test_quantize_checks():
    for bad in (t(4, 128, dtype=torch.float16), t(128), t(128, 4).t(), None):
        with pytest.raises(ValueError):
            block.quantize_mx8(bad)
    with pytest.raises(ValueError, match="out"):
        block.quantize_mx8(t(4, 128), out=block.empty_mx8(4, 64, "cpu"))


def test_layer_checks():
    with pytest.raises(ValueError, match="recompute"):
        MoeLayer(8, 128, 4, 2, 128, recompute=True, shared_F=128, device="cpu")
    with pytest.raises(ValueError, match="BF16"):
        MoeLayer(8, 128, 4, 2, 128, dtype=moe.MOE_DTYPE_F32, shared_F=128, device="cpu")
    x, w = t(8, 128), t(1)
    plain = MoeLayer(8, 128, 4, 2, 128, device="cpu")
    for kw in (dict(norm_w=t(128)), dict(residual=x), dict(shared_w_gu=w, shared_w_down=w)):
        with pytest.raises(ValueError):
            plain.forward(8, x, w, w, **kw)
    with pytest.raises(ValueError):
        plain.backward(8, x, w, w, w, w, dres=x)
    full = MoeLayer(8, 128, 4, 2, 128, norm_eps=1e-6, shared_F=64, device="cpu")
    for kw in (dict(), dict(norm_w=t(128)), dict(norm_w=t(128), shared_w_gu=w), dict(shared_w_gu=w, shared_w_down=w)):
        with pytest.raises(ValueError):
            full.forward(8, x, w, w, **kw)
    grads = dict(norm_w=w, dnorm_w=w, shared_w_gu=w, shared_w_down=w, dshared_w_gu=w, dshared_w_down=w)
    with pytest.raises(ValueError, match="norm_r"):  # the last forward had no residual
        full.backward(8, x, w, w, w, w, **grads)
    full.norm_summed = True
    with pytest.raises(ValueError, match="norm_r"):
        full.backward(8, x, w, w, w, w, norm_r=x, **grads)
