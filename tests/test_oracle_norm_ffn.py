"""Pins of the norm, block-form and dense feed-forward oracles (CPU only)."""
import numpy as np
import pytest

import oracle


def _num_grad(f, v, h=1e-6):
    g = np.zeros_like(v)
    it = np.nditer(v, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = v[i]
        v[i] = old + h
        hi = f()
        v[i] = old - h
        lo = f()
        v[i] = old
        g[i] = (hi - lo) / (2 * h)
    return g


@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_gradient_against_differences(residual):
    rng = np.random.default_rng(1)
    x, w, dy = rng.normal(size=(3, 8)), rng.normal(1, 0.2, 8), rng.normal(size=(3, 8))
    res = rng.normal(size=(3, 8)) if residual else None
    dres = rng.normal(size=(3, 8)) if residual else None
    eps = 1e-3

    def loss():
        r, _, y = oracle.rmsnorm_fwd(x, w, eps, res)
        return np.sum(y * dy) + (np.sum(r * dres) if residual else 0.0)

    r, rstd, _ = oracle.rmsnorm_fwd(x, w, eps, res)
    dx, dw = oracle.rmsnorm_bwd(dy, r, w, rstd, dres)
    # central differences at h = 1e-6: truncation ~ h^2, rounding ~ 2^-53 / h = 1e-10
    np.testing.assert_allclose(dx, _num_grad(loss, x), atol=1e-7)
    np.testing.assert_allclose(dw, _num_grad(loss, w), atol=1e-7)
    if residual:
        np.testing.assert_allclose(dx, _num_grad(loss, res), atol=1e-7)


def test_rmsnorm_by_hand():
    # row (3, 4), eps 0.5: mean square 12.5, rstd = 1 / sqrt(13)
    r, rstd, y = oracle.rmsnorm_fwd(np.array([[1.0, 4.0]]), np.array([2.0, -1.0]), 0.5, np.array([[2.0, 0.0]]))
    assert r.tolist() == [[3.0, 4.0]] and rstd[0] == pytest.approx(13 ** -0.5)
    assert y[0].tolist() == pytest.approx([6 * 13 ** -0.5, -4 * 13 ** -0.5])


def test_mx8_by_hand():
    v = np.zeros((1, 160))
    v[0, :32] = 448.0            # exactly the largest: S = 1
    v[0, 32:64] = 448.5          # just over: S = 2, 224.25 -> 224
    v[0, 64], v[0, 65] = 1.75, 0.0625   # S = 2^-8: 448 and 16
    v[0, 66] = 2.0 ** -18        # 2^-10 of a unit: below half of the smallest step 2^-9, a tie to even -> 0
    v[0, 96] = 1e-45             # a fp32 denormal: S = 2^-127
    q, S = oracle.mx8_quantize(v)
    assert S[0].tolist() == [1.0, 2.0, 2.0 ** -8, 2.0 ** -127, 2.0 ** -127]
    assert q[0, 0] == 448 and q[0, 32] == 224 and q[0, 64] == 448 and q[0, 65] == 16 and q[0, 66] == 0
    assert q[0, 128:].tolist() == [0.0] * 32


def test_mx8_rounding_against_torch():
    torch = pytest.importorskip("torch")
    v = np.concatenate([np.linspace(-448, 448, 40001), np.linspace(-0.05, 0.05, 20001)]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.mx8_round(v), want)


def test_dense_ffn_gradient_against_differences():
    rng = np.random.default_rng(2)
    T, d, F = 3, 5, 4
    x, wg, wd = rng.normal(size=(T, d)), rng.normal(size=(2 * F, d)), rng.normal(size=(d, F))
    add, dy = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss():
        return np.sum(oracle.dense_ffn_fwd(x, wg, wd, add)[2] * dy)

    h, a, _ = oracle.dense_ffn_fwd(x, wg, wd, add)
    _, dh, dx = oracle.dense_ffn_dgrad(dy, h, wg, wd)
    dw_gu, dw_down = oracle.dense_ffn_wgrad(dy, x, a, dh)
    np.testing.assert_allclose(dx, _num_grad(loss, x), atol=1e-7)
    np.testing.assert_allclose(dw_gu, _num_grad(loss, wg), atol=1e-7)
    np.testing.assert_allclose(dw_down, _num_grad(loss, wd), atol=1e-7)
    np.testing.assert_allclose(dy, _num_grad(loss, add), atol=1e-7)


def test_dense_ffn_is_one_expert_of_the_layer():
    """The block equals the routed layer with one expert that takes every token with weight one."""
    rng = np.random.default_rng(3)
    T, d, F = 6, 8, 4
    x, wg, wd = rng.normal(size=(T, d)), rng.normal(size=(2 * F, d)), rng.normal(size=(d, F))
    out, _ = oracle.layer_fwd(x, wg[None], wd[None], 1, logits=np.zeros((T, 1)))
    np.testing.assert_allclose(oracle.dense_ffn_fwd(x, wg, wd)[2], out, rtol=1e-12)
