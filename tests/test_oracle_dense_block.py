"""Pins of the layer norm, dense product and orthogonalisation oracles (CPU
only): central differences, torch's float64 forms, matrices of known singular
values."""
import numpy as np
import pytest

import oracle


def _num_grad(f, v, h=1e-6):
    g = np.zeros_like(v)
    for i in np.ndindex(*v.shape):
        old = v[i]
        v[i] = old + h
        hi = f()
        v[i] = old - h
        lo = f()
        v[i] = old
        g[i] = (hi - lo) / (2 * h)
    return g


@pytest.mark.parametrize("residual", [False, True])
def test_layernorm_gradient_against_differences(residual):
    rng = np.random.default_rng(1)
    x, w, b = rng.normal(0.5, 1, (3, 8)), rng.normal(1, 0.2, 8), rng.normal(size=8)
    dy = rng.normal(size=(3, 8))
    res, dres = (rng.normal(size=(3, 8)), rng.normal(size=(3, 8))) if residual else (None, None)

    def loss():
        r, _, _, _, y = oracle.layernorm_fwd(x, w, b, 1e-3, res)
        return np.sum(y * dy) + (np.sum(r * dres) if residual else 0.0)

    r, mean, rstd, _, _ = oracle.layernorm_fwd(x, w, b, 1e-3, res)
    dx, dw, db = oracle.layernorm_bwd(dy, r, w, mean, rstd, dres)
    # h = 1e-6: truncation ~ h^2, rounding ~ 2^-53 / h = 1e-10
    for got, v in ((dx, x), (dw, w), (db, b)):
        np.testing.assert_allclose(got, _num_grad(loss, v), atol=1e-7)


def test_layernorm_against_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    x, w, b = rng.normal(3, 2, (5, 64)), rng.normal(size=64), rng.normal(size=64)
    y = torch.nn.functional.layer_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    np.testing.assert_allclose(oracle.layernorm_fwd(x, w, b, 1e-5)[4], y.numpy(), atol=1e-13)


@pytest.mark.parametrize("name", oracle.ACTS)
def test_activations_against_torch_and_differences(name):
    torch = pytest.importorskip("torch")
    F = torch.nn.functional
    z = np.concatenate([np.linspace(-12, 12, 401), [1e-3, -1e-3]]) + 1e-4
    t = torch.from_numpy(z)
    want = {"none": t, "relu": F.relu(t), "gelu": F.gelu(t), "gelu_tanh": F.gelu(t, approximate="tanh"), "silu": F.silu(t)}
    np.testing.assert_allclose(oracle.act(name, z), want[name].numpy(), atol=1e-14, rtol=1e-12)
    h = 1e-6
    diff = (oracle.act(name, z + h) - oracle.act(name, z - h)) / (2 * h)
    np.testing.assert_allclose(oracle.act_slope(name, z), diff, atol=2e-8)


@pytest.mark.parametrize("name", oracle.ACTS)
def test_chain_of_two_products_against_differences(name):
    """dx of the upper product, with the lower activation's slope, is the dz of the lower one."""
    rng = np.random.default_rng(3)
    x, w1, b1 = rng.normal(size=(4, 3)), rng.normal(size=(5, 3)), rng.normal(size=5)
    w2, b2, res, dy = rng.normal(size=(2, 5)), rng.normal(size=2), rng.normal(size=(4, 2)), rng.normal(size=(4, 2))

    def loss():
        z, a = oracle.linear_fwd(x, w1, b1, None, name)
        return np.sum(oracle.linear_fwd(a, w2, b2, res)[1] * dy)

    z1, a = oracle.linear_fwd(x, w1, b1, None, name)
    dz1 = oracle.linear_dgrad(dy, w2, z1, name)
    dw1, db1 = oracle.linear_wgrad(dz1, x)
    dw2, db2 = oracle.linear_wgrad(dy, a)
    for got, v in ((oracle.linear_dgrad(dz1, w1), x), (dw1, w1), (db1, b1), (dw2, w2), (db2, b2), (dy, res)):
        np.testing.assert_allclose(got, _num_grad(loss, v), atol=1e-7)


def _with_singular_values(rng, m, n, s):
    u, _ = np.linalg.qr(rng.normal(size=(m, len(s))))
    v, _ = np.linalg.qr(rng.normal(size=(n, len(s))))
    return (u * s) @ v.T, u, v


@pytest.mark.parametrize("m,n", [(6, 9), (9, 6), (7, 7), (1, 5), (5, 1)])
def test_orthogonalisation_maps_the_singular_values(m, n):
    """U diag(s) V^T goes to U diag(p(...p(s / |s|))) V^T."""
    rng = np.random.default_rng(4)
    s = np.exp(rng.normal(0, 1, min(m, n)))
    u_mat, u, v = _with_singular_values(rng, m, n, s)
    a, b, c = oracle.ORTH_COEF
    q = s / np.linalg.norm(s)
    for _ in range(5):
        q = a * q + b * q ** 3 + c * q ** 5
    np.testing.assert_allclose(oracle.orthogonalize(u_mat, eps=0.0), (u * q) @ v.T, atol=1e-11)
    assert np.all(q < 1.21)


def test_orthogonalisation_of_scaled_zero_and_orthogonal_matrices():
    rng = np.random.default_rng(5)
    x = rng.normal(size=(8, 20))
    np.testing.assert_allclose(oracle.orthogonalize(x * 1e6, eps=0.0), oracle.orthogonalize(x, eps=0.0), atol=1e-12)
    assert not oracle.orthogonalize(np.zeros((3, 4))).any()
    # the cubic iteration converges to the polar factor
    u, _, vt = np.linalg.svd(x, full_matrices=False)
    np.testing.assert_allclose(oracle.orthogonalize(x, steps=40, coef=(1.5, -0.5, 0.0)), u @ vt, atol=1e-10)


def test_the_halves_are_the_iteration_up_to_rounding():
    """Close to the formula, on matrices of even and of very uneven singular values, and the formula itself where fp16
    holds everything: the identity, whose iterates are multiples of it."""
    rng = np.random.default_rng(6)
    even = rng.normal(size=(96, 160))
    uneven = 0.1 * even + rng.normal(size=(96, 4)) * 10 @ rng.normal(size=(4, 160))
    for u in (even, uneven, even.T):
        want = oracle.orthogonalize(u)
        assert np.linalg.norm(oracle.orthogonalize_halves(u) - want) <= 2e-3 * np.linalg.norm(want)
    # s_k times the identity: A comes from the high half alone, which is off by up to 2^-11 of X, so A by 2^-10 and the
    # step by 2^-10 (|b| s^3 + 2 |c| s^5), which the slopes of the later steps carry on; the last step has |a + b s^2 + c
    # s^4| times the high half's own 2^-11 s beside it
    a, b, c = oracle.ORTH_COEF
    s, bar = 0.125, 0.0
    for _ in range(5):
        bar = bar * abs(a + 3 * b * s ** 2 + 5 * c * s ** 4) + 2.0 ** -10 * (abs(b) * s ** 3 + 2 * abs(c) * s ** 5)
        s = a * s + b * s ** 3 + c * s ** 5
    d = oracle.orthogonalize_halves(np.eye(64, 128)) - oracle.orthogonalize(np.eye(64, 128))
    bar += 2.0 ** -11 * abs(s)
    assert np.abs(d).max() <= bar + 2.0 ** -19  # X itself to 22 bits before that


def test_muon_step_by_hand():
    """A 1 x 1 weight: o = p(...p(sign)) alone, momentum and decay as written."""
    a, b, c = oracle.ORTH_COEF
    q = 1.0
    for _ in range(5):
        q = a * q + b * q ** 3 + c * q ** 5
    p, m, o = oracle.muon_step([[2.0]], [[-0.5]], [[0.3]], lr=0.1, mu=0.9, weight_decay=0.5, scale=2.0, grad_scale=2.0,
                               nesterov=True, eps=0.0)
    assert m[0, 0] == pytest.approx(0.9 * 0.3 - 1.0)
    assert o[0, 0] == pytest.approx(-q) and p[0, 0] == pytest.approx(2.0 * 0.95 + 0.2 * q)
    # plain momentum may point the other way
    assert oracle.muon_step([[2.0]], [[-0.1]], [[1.0]], lr=0.1, mu=0.9, nesterov=False, eps=0.0)[2][0, 0] == pytest.approx(q)
