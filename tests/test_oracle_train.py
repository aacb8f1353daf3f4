"""Pins of the training oracle: every gradient against central differences
of the float64 forward functions and against torch's float64 autograd."""

import numpy as np
import pytest

import oracle

H = 1e-5
# A central difference of a smooth function is off by H^2 f'''/6 plus the
# rounding of f over 2 H: with |f| and its derivatives of order 10 that is
# 1e-9 + 10 * 2^-53 / 1e-5 = 1e-9 + 1e-10.
TOL = 1e-7


def _difference(fn, a):
    """d fn() / d a by central differences, a changed in place."""
    out = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + H
        hi = fn()
        a[i] = keep - H
        lo = fn()
        a[i] = keep
        out[i] = (hi - lo) / (2 * H)
    return out


@pytest.mark.parametrize("n,d", [(1, 1), (1, 7), (4, 5)])
def test_layer_norm_grad(n, d):
    rng = np.random.default_rng(n * 10 + d)
    x, dy = rng.standard_normal((n, d)) + 0.5, rng.standard_normal((n, d))
    w, b = rng.standard_normal(d), rng.standard_normal(d)
    y, mean, rstd = oracle.layer_norm(x, w, b, 1e-2)
    dx, dw, db = oracle.layer_norm_grad(dy, x, w, mean, rstd)
    loss = lambda: float((oracle.layer_norm(x, w, b, 1e-2)[0] * dy).sum())  # noqa: E731
    np.testing.assert_allclose(dx, _difference(loss, x), atol=TOL * 10, rtol=TOL)
    np.testing.assert_allclose(dw, _difference(loss, w), atol=TOL, rtol=TOL)
    np.testing.assert_allclose(db, _difference(loss, b), atol=TOL, rtol=TOL)
    torch = pytest.importorskip("torch")
    t = torch.tensor(x, requires_grad=True)
    ty = torch.nn.functional.layer_norm(t, (d,), torch.tensor(w), torch.tensor(b), 1e-2)
    ty.backward(torch.tensor(dy))
    np.testing.assert_allclose(y, ty.detach().numpy(), atol=1e-12)
    np.testing.assert_allclose(dx, t.grad.numpy(), atol=1e-11)


def _layer(seed, n, d, E, k, f, skip=()):
    """Small routed batch; experts in `skip` get no row."""
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((n, E))
    z[:, list(skip)] = -50.0
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k]
    return rng, z, idx, oracle.dispatch(idx, E)


@pytest.mark.parametrize("k,renorm", [(1, False), (2, True), (3, True), (2, False)])
def test_whole_layer_gradients(k, renorm):
    """The gradients chained as a training step chains them: the loss sum(y dy)
    + the auxiliary loss, differentiated through experts, weights and router."""
    n, d, E, f, alpha = 5, 4, 4, 3, 0.3
    rng, z0, _, _ = _layer(k, n, d, E, k, f)
    x, wg, bias = rng.standard_normal((n, d)), rng.standard_normal((E, d)), rng.standard_normal(E)
    bias[3] = -30.0  # expert 3 has no rows
    w1, w3, w2 = (rng.standard_normal(s) for s in ((E, f, d), (E, f, d), (E, d, f)))
    dy = rng.standard_normal((n, d))
    z = x @ wg.T + bias
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k]
    frac = np.bincount(idx[:, 0], minlength=E) / n
    dp = oracle.dispatch(idx, E)

    def loss():
        z = x @ wg.T + bias
        w, p = oracle.router_weights(z, idx, renorm)
        y = np.zeros((n, d))
        for t in range(n):
            for j in range(k):
                e = idx[t, j]
                y[t] += w[t, j] * oracle.swiglu_expert(x[t:t + 1], w1[e], w3[e], w2[e])[0]
        return float((y * dy).sum() + alpha * E * (frac * p.mean(axis=0)).sum())

    w, _ = oracle.router_weights(z, idx, renorm)
    perm, inv, offsets = dp["perm"], dp["inv"].reshape(n, k), dp["offsets"]
    h, g, u = oracle.expert_up(x, perm, offsets, w1, w3)
    da, dw1, dw3, dw2, dtw = oracle.grouped_ffn_grad(dy, x, perm, inv, w, offsets, w1, w3, w2, g, u)
    dz, dx, dwg, dbias = oracle.router_grad(z, idx, w, dtw, frac, alpha, renorm, x, wg, da, inv)
    for got, var in ((dx, x), (dwg, wg), (dbias, bias), (dw1, w1), (dw3, w3), (dw2, w2)):
        # (values of order 10 to 100 under this loss)
        np.testing.assert_allclose(got, _difference(loss, var), atol=100 * TOL, rtol=1e-6)
    assert not dw1[3].any() and not dw2[3].any()


def test_pile_rows_without_a_combine():
    rng = np.random.default_rng(3)
    R, d, f = 6, 4, 3
    offsets = np.array([0, 2, 2, 5])  # an empty expert, and a row behind the last pile
    a, dy = rng.standard_normal((R, d)), rng.standard_normal((R, d))
    w1, w3, w2 = (rng.standard_normal(s) for s in ((3, f, d), (3, f, d), (3, d, f)))
    h, g, u = oracle.expert_up(a, None, offsets, w1, w3)
    da, dw1, dw3, dw2, dtw = oracle.grouped_ffn_grad(dy, a, None, None, None, offsets, w1, w3, w2, g, u)
    assert dtw is None and np.isnan(da[5]).all() and np.isnan(h[5]).all()

    def loss():
        s = 0.0
        for e in range(3):
            r = slice(offsets[e], offsets[e + 1])
            s += (oracle.swiglu_expert(a[r], w1[e], w3[e], w2[e]) * dy[r]).sum()
        return float(s)

    np.testing.assert_allclose(da[:5], _difference(loss, a)[:5], atol=10 * TOL, rtol=1e-6)
    for got, var in ((dw1, w1), (dw3, w3), (dw2, w2)):
        np.testing.assert_allclose(got, _difference(loss, var), atol=10 * TOL, rtol=1e-6)


def test_pairs_outside_the_experts_have_no_gradient():
    rng = np.random.default_rng(5)
    n, E, k, d = 4, 3, 2, 5
    z, x, wg = rng.standard_normal((n, E)), rng.standard_normal((n, d)), rng.standard_normal((E, d))
    idx = np.array([[0, 1], [2, -1], [7, 1], [-1, 9]])
    w, dw = rng.random((n, k)), rng.standard_normal((n, k))
    dz, dx, dwg, dbias = oracle.router_grad(z, idx, w, dw, None, 0.0, True, x, wg)
    assert not dz[3].any() and np.isfinite(dz).all()
    other = dw.copy()
    other[1, 1] = other[2, 0] = other[3] = 1e6
    np.testing.assert_array_equal(dz, oracle.router_grad(z, idx, w, other, None, 0.0, True, x, wg)[0])


def test_the_same_expert_twice_adds_up():
    z = np.array([[0.3, -0.2, 0.1]])
    idx = np.array([[1, 1]])
    w, p = oracle.router_weights(z, idx, True)
    dw = np.array([[0.7, -0.4]])
    dz = oracle.router_grad(z, idx, w, dw, None, 0.0, True, np.ones((1, 2)), np.ones((3, 2)))[0]
    np.testing.assert_allclose(dz, 0.0, atol=1e-15)  # both weights stay 1/2
    w, p = oracle.router_weights(z, idx, False)
    dz = oracle.router_grad(z, idx, w, dw, None, 0.0, False, np.ones((1, 2)), np.ones((3, 2)))[0]
    want = p[0, 1] * (dw.sum()) * (np.eye(3)[1] - p[0])
    np.testing.assert_allclose(dz[0], want, atol=1e-15)
