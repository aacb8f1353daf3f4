"""Pins of the training oracle: the gradients of a whole step against torch's
float64 autograd through a layer that shares no code with the oracle."""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")


def _layer(x, p, k, renorm, alpha, eps):
    """Norm, router, experts and combine, every expert on every token, the
    chosen ones picked by their weights; (y, the auxiliary loss)."""
    E = p["wg"].shape[0]
    xn = torch.nn.functional.layer_norm(x, (x.shape[1],), p["norm_weight"], p["norm_bias"], eps)
    prob = torch.softmax(torch.nn.functional.linear(xn, p["wg"], p["bias"]), dim=1)
    top, idx = torch.topk(prob, k, dim=1)
    w = top / top.sum(dim=1, keepdim=True) if renorm else top
    silu = torch.nn.functional.silu
    out = [(silu(xn @ p["w1"][e].T) * (xn @ p["w3"][e].T)) @ p["w2"][e].T for e in range(E)]
    y = sum((w * (idx == e)).sum(dim=1, keepdim=True) * out[e] for e in range(E))
    f = torch.bincount(idx[:, 0], minlength=E).double() / len(x)  # a count: no gradient
    return y, alpha * E * (f * prob.mean(dim=0)).sum()


# n, d, E, k, f
SHAPES = [(1, 1, 1, 1, 1), (9, 6, 4, 1, 5), (9, 6, 4, 2, 5), (17, 8, 6, 3, 7), (5, 4, 3, 3, 2)]


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("n,d,E,k,f", SHAPES)
def test_step_gradients(n, d, E, k, f, renorm):
    alpha, eps = 0.3, 1e-2
    rng = np.random.default_rng(100 * n + 10 * E + k)
    sizes = dict(x=(n, d), norm_weight=(d,), norm_bias=(d,), wg=(E, d), bias=(E,), w1=(E, f, d), w3=(E, f, d),
                 w2=(E, d, f))
    v = {name: rng.standard_normal(size) for name, size in sizes.items()}
    if E > 1:
        v["bias"][E - 1] = -30.0 if k < E else 0.0  # where it may be, an expert without a token
    dy = rng.standard_normal((n, d))

    t = {name: torch.tensor(a, requires_grad=True) for name, a in v.items()}
    y, aux = _layer(t["x"], t, k, renorm, alpha, eps)
    ((y * torch.tensor(dy)).sum() + aux).backward()

    xn, mean, rstd = oracle.layer_norm(v["x"], v["norm_weight"], v["norm_bias"], eps)
    z = xn @ v["wg"].T + v["bias"]
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k]
    w, _ = oracle.router_weights(z, idx, renorm)
    dp = oracle.dispatch(idx, E)
    perm, inv, offsets = dp["perm"], dp["inv"].reshape(n, k), dp["offsets"]
    frac = np.bincount(idx[:, 0], minlength=E) / n
    h, g, u = oracle.expert_up(xn, perm, offsets, v["w1"], v["w3"])
    got = {}
    da, got["w1"], got["w3"], got["w2"], dw = oracle.grouped_ffn_grad(
        dy, xn, perm, inv, w, offsets, v["w1"], v["w3"], v["w2"], g, u)
    _, dxn, got["wg"], got["bias"] = oracle.router_grad(z, idx, w, dw, frac, alpha, renorm, xn, v["wg"], da, inv)
    got["x"], got["norm_weight"], got["norm_bias"] = oracle.layer_norm_grad(dxn, v["x"], v["norm_weight"], mean, rstd)
    for name in sizes:
        want = t[name].grad.numpy()
        # Two float64 evaluations of one expression: sums of at most n k d f < 2^12
        # products, six operators deep, of values that cancel by up to 1e3.
        np.testing.assert_allclose(got[name], want, rtol=0, atol=2.0 ** -53 * 2 ** 12 * 6 * 1e3 * max(1, np.abs(want).max()),
                                   err_msg=name)


@pytest.mark.parametrize("n,d", [(1, 1), (3, 9)])
def test_ffn_without_a_combine(n, d):
    """The dense block: pile rows in, pile rows out, one expert."""
    f = 4
    rng = np.random.default_rng(n)
    a, dy = rng.standard_normal((n, d)), rng.standard_normal((n, d))
    w1, w3, w2 = (rng.standard_normal(s) for s in ((1, f, d), (1, f, d), (1, d, f)))
    offsets = np.array([0, n])
    _, g, u = oracle.expert_up(a, None, offsets, w1, w3)
    da, dw1, dw3, dw2, _ = oracle.grouped_ffn_grad(dy, a, None, None, None, offsets, w1, w3, w2, g, u)
    ta, t1, t3, t2 = (torch.tensor(x, requires_grad=True) for x in (a, w1[0], w3[0], w2[0]))
    y = (torch.nn.functional.silu(ta @ t1.T) * (ta @ t3.T)) @ t2.T
    y.backward(torch.tensor(dy))
    for got, t in ((da, ta), (dw1[0], t1), (dw3[0], t3), (dw2[0], t2)):
        np.testing.assert_allclose(got, t.grad.numpy(), rtol=0, atol=1e-12)
