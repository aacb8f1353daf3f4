"""GPU parity of moe_router_backward with the float64 oracle.

Tolerances (derived, not measured); U = 2^-24, half = half a step of the
stored type.  dlogits: a softmax probability is off by (E + 32) U at most
(its sum of E terms, the exponent and the division), D by (k + 2) U of
sum |w dw|; a few roundings join them.  dx and dW_g: a float32 sum of E + k
(or n) terms, and with bf16 rows each product's dlogits is off by 2^-16 (it
enters as a bf16 value and a bf16 rest), then one rounding."""

import numpy as np
import pytest

import oracle
from tests.gpu_support import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SPLIT = {"bf16": 2.0 ** -16, "f32": 0.0}

# n, d, E, k
SHAPES = {
    "bf16": [(1, 8, 1, 1), (1, 264, 8, 2), (3, 72, 5, 1), (33, 256, 8, 2), (70, 520, 33, 4), (300, 136, 64, 3),
             (65, 136, 65, 8), (600, 264, 128, 4), (40, 72, 300, 32), (17, 64, 1024, 1), (4100, 264, 8, 2)],
    "f32": [(1, 1, 1, 1), (6, 3, 4, 1), (33, 65, 5, 2), (129, 64, 64, 4), (70, 33, 130, 8), (3000, 20, 7, 2)],
}
CASES = [(t,) + s for t in SHAPES for s in SHAPES[t]]


def _t(a, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)


def _f64(t):
    return t.double().cpu().numpy()


def _batch(dtype, n, d, E, k, renorm, seed=0):
    import torch

    rng = np.random.default_rng(seed + n + d + E)
    z = _t(2 * rng.standard_normal((n, E)), "f32")
    idx = np.argsort(-_f64(z), axis=1, kind="stable")[:, :k].astype(np.int32)
    w, _ = oracle.router_weights(_f64(z), idx, renorm)
    order = np.argsort(idx.reshape(-1), kind="stable")
    inv = np.empty(n * k, np.int32)
    inv[order] = np.arange(n * k)
    return dict(z=z, idx=torch.from_numpy(idx).cuda(), w=_t(w, "f32"), dw=_t(rng.standard_normal((n, k)), "f32"),
                f=_t(np.bincount(idx[:, 0], minlength=E) / n, "f32"), x=_t(rng.standard_normal((n, d)), dtype),
                wg=_t(rng.standard_normal((E, d)) / d ** 0.5, dtype), da=_t(rng.standard_normal((n * k, d)), dtype),
                inv=torch.from_numpy(inv.reshape(n, k)).cuda())


def _run(b, dtype, shape, alpha=0.5, aux=True, rows=True, bias=True, stream=None):
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    n, d, E, k = shape[:4]

    def out(count, dt):
        return torch.full((count + 8,), 7.0, dtype=dt, device="cuda")

    dz, dx, dwg, db = (out(n * E, torch.float32), out(n * d, b["x"].dtype), out(E * d, b["x"].dtype),
                       out(E, torch.float32))
    nb = B.moe_router_backward_workspace_bytes(shape)
    ws = torch.full((nb + 256,), 255, dtype=torch.uint8, device="cuda")
    B.moe_router_backward(shape, b["z"], b["idx"], b["w"], b["dw"], b["f"] if aux else None, alpha, b["x"], dtype,
                          b["wg"], b["da"] if rows else None, b["inv"] if rows else None, dz, dx, dwg,
                          db if bias else None, ws, nb, stream)
    torch.cuda.synchronize()
    for t, count in ((dz, n * E), (dx, n * d), (dwg, E * d), (db, E)):
        assert (t[count:] == 7).all()
    assert (ws[nb:] == 255).all() and (bias or (db == 7).all())
    return dz[:-8].view(n, E), dx[:-8].view(n, d), dwg[:-8].view(E, d), db[:-8]


def _check(name, got, ref, tol):
    assert np.isfinite(got).all(), name
    worst = float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-300), initial=0.0))
    say(f"    {name}: largest error / tolerance {worst:.3f}")
    assert worst <= 1.0, name


def _verify(b, got, dtype, shape, renorm, alpha=0.5, aux=True, rows=True):
    n, d, E, k = shape[:4]
    h = {key: _f64(t) if t.is_floating_point() else t.cpu().numpy() for key, t in b.items()}
    args = (h["z"], h["idx"], h["w"], h["dw"], h["f"] if aux else None, alpha, renorm, h["x"], h["wg"])
    dz, dx, dwg, db = oracle.router_grad(*args, *((h["da"], h["inv"]) if rows else ()))
    ok = (h["idx"] >= 0) & (h["idx"] < E)
    aw = np.where(ok, np.abs(h["w"] * h["dw"]), 0.0)
    D = aw.sum(axis=1, keepdims=True)
    p = np.exp(h["z"] - h["z"].max(axis=1, keepdims=True))
    p = p / p.sum(axis=1, keepdims=True)
    mag = np.zeros((n, E))
    for j in range(k):
        t = np.nonzero(ok[:, j])[0]
        e = h["idx"][t, j]
        if renorm:
            np.add.at(mag, (t, e), aw[t, j] + np.abs(h["w"][t, j]) * D[t, 0])
        else:
            np.add.at(mag, (t, e), p[t, e] * np.abs(h["dw"][t, j]))
    if not renorm:
        mag += p * D
    if aux:
        mag += alpha * E / n * p * (np.abs(h["f"]) + (p * np.abs(h["f"])).sum(axis=1, keepdims=True))
    ez = (E + 3 * k + 64) * U * mag
    _check("dlogits", _f64(got[0]), dz, ez)
    az = np.abs(dz) + ez
    tx = (ez + (SPLIT[dtype] + (2 * E + k + 16) * U) * az) @ np.abs(h["wg"])
    if rows:
        for j in range(k):
            r = h["inv"][:, j]
            good = (r >= 0) & (r < n * k)
            tx[good] += (E + k + 16) * U * np.abs(h["da"][r[good]])
    _check("dx", _f64(got[1]), dx, HALF[dtype] * np.abs(dx) * (1 + 2 ** -8) + tx)
    tw = (ez + (SPLIT[dtype] + (2 * n + 64) * U) * az).T @ np.abs(h["x"])
    _check("dwg", _f64(got[2]), dwg, HALF[dtype] * np.abs(dwg) * (1 + 2 ** -8) + tw)
    _check("dbias", _f64(got[3]), db, (ez + (n / 64 + 96) * U * az).sum(axis=0))


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("dtype,n,d,E,k", CASES)
def test_gradient(dtype, n, d, E, k, renorm):
    import torch

    say(f"[router grad] {dtype} n={n} d={d} E={E} k={k} renorm={renorm}")
    shape = (n, d, E, k, 8, renorm)
    b = _batch(dtype, n, d, E, k, renorm)
    got = _run(b, dtype, shape)
    _verify(b, got, dtype, shape, renorm)
    for p, q in zip(got, _run(b, dtype, shape)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_options(dtype):
    import torch

    say(f"[router grad, options] {dtype}")
    n, d, E, k = 50, 72, 9, 2
    b = _batch(dtype, n, d, E, k, True)
    shape = (n, d, E, k, 8)  # the default rule renormalises for k > 1
    for aux in (True, False):
        for rows in (True, False):
            got = _run(b, dtype, shape, aux=aux, rows=rows)
            _verify(b, got, dtype, shape, True, aux=aux, rows=rows)
    no_bias = _run(b, dtype, shape, aux=False, rows=False, bias=False)
    for p, q in zip(got[:3], no_bias[:3]):
        assert torch.equal(p, q)
    one = _batch(dtype, n, d, E, 1, False)
    _verify(one, _run(one, dtype, (n, d, E, 1, 8)), dtype, (n, d, E, 1), False)  # k = 1: raw


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_ids_outside_and_repeated(dtype, renorm):
    say(f"[router grad, ids] {dtype} renorm={renorm}")
    n, d, E, k = 40, 64, 6, 3
    b = _batch(dtype, n, d, E, k, renorm)
    b["idx"][::3, 1] = E
    b["idx"][1::4, 0] = -1
    b["idx"][2::5, 2] = b["idx"][2::5, 0]
    b["inv"][::3, 1] = -1
    b["inv"][1::4, 0] = n * k
    shape = (n, d, E, k, 8, renorm)
    _verify(b, _run(b, dtype, shape), dtype, shape, renorm)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_logits(dtype):
    """Experts masked with -inf have probability 0 and no gradient; a token
    with every expert masked has none at all, whatever its weights hold; a NaN
    logit spoils its own token's rows, and W_g's gradient with them."""
    import torch

    say(f"[router grad, masks] {dtype}")
    n, d, E, k = 30, 64, 8, 2
    for renorm in (0, 1):
        b = _batch(dtype, n, d, E, k, renorm)
        b["z"][:, 5] = -float("inf")
        idx = torch.argsort(-b["z"], dim=1, stable=True)[:, :k].to(torch.int32)
        b["idx"] = idx.contiguous()
        w, _ = oracle.router_weights(_f64(b["z"]), idx.cpu().numpy(), renorm)
        b["w"] = _t(w, "f32")
        shape = (n, d, E, k, 8, renorm)
        got = _run(b, dtype, shape)
        assert not _f64(got[0])[:, 5].any()
        _verify(b, got, dtype, shape, renorm)
        b["z"][3] = -float("inf")
        b["w"][3] = float("nan")
        dz, dx, dwg, db = _run(b, dtype, shape)
        assert not dz[3].any() and torch.isfinite(dwg).all() and torch.isfinite(dx).all()
        keep = [t for t in range(n) if t != 3]
        assert torch.equal(dz[keep], got[0][keep]) and torch.equal(dx[keep], got[1][keep])
        b["z"][4, 0] = float("nan")
        dz, dx, _, _ = _run(b, dtype, shape)
        assert torch.isnan(dz[4]).all()
        keep = [t for t in range(n) if t not in (3, 4)]
        assert torch.equal(dz[keep], got[0][keep]) and torch.equal(dx[keep], got[1][keep])


def test_gradient_against_differences():
    """The auxiliary loss and a loss on the weights, from the library's own
    router, against dlogits' effect along W_g and the bias."""
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    say("[router grad, differences]")
    n, d, E, k, alpha = 48, 16, 6, 2, 0.7
    rng = np.random.default_rng(2)
    wg = _t(rng.standard_normal((E, d)), "f32")
    bias, dw = _t(rng.standard_normal(E), "f32"), _t(rng.standard_normal((n, k)), "f32")
    # tokens whose three best logits are 0.15 apart, so that a step of 2^-10 per
    # element (at most 2^-10 * 16 * 4 in a logit) changes no choice
    many = _t(rng.standard_normal((4000, d)), "f32")
    top = -np.sort(-(_f64(many) @ _f64(wg).T + _f64(bias)), axis=1)[:, :3]
    x = many[np.nonzero((-np.diff(top, axis=1)).min(axis=1) > 0.15)[0][:n]].contiguous()
    shape = (n, d, E, k, 8)
    nb = B.moe_router_stats_workspace_bytes(shape)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def forward(wg, bias):
        z, idx = torch.empty(n, E, device="cuda"), torch.empty(n, k, dtype=torch.int32, device="cuda")
        w = torch.empty(n, k, device="cuda")
        B.moe_router_topk(shape, x, "f32", wg, bias, z, idx, w)
        P, f, loss = torch.empty(E, device="cuda"), torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
        B.moe_router_stats(shape, z, idx, alpha, P, f, loss, ws, nb)
        torch.cuda.synchronize()
        return z, idx, w, f, float((w.double() * dw.double()).sum()) + float(loss)

    z, idx, w, f, _ = forward(wg, bias)
    b = dict(z=z, idx=idx, w=w, dw=dw, f=f, x=x, wg=wg, da=None, inv=None)
    dz, dx, dwg, db = _run(b, "f32", shape, alpha=alpha, rows=False)
    h = 2.0 ** -10
    for var, grad, at in ((wg, dwg, 0), (bias, db, 1)):
        v = _t(np.sign(rng.standard_normal(tuple(var.shape))), "f32") * h
        args = [(wg + v, bias), (wg - v, bias)] if at == 0 else [(wg, bias + v), (wg, bias - v)]
        hi, lo = forward(*args[0]), forward(*args[1])
        assert torch.equal(hi[1], idx) and torch.equal(lo[1], idx)  # no token changes its experts
        want = float((grad.double() * 2 * v.double()).sum())
        # float32 sums of n k terms of size 1; third order: each logit moves by at
        # most h sqrt(d) 4, whose cube is 2^-25 n k / 6 of the weights' size 1
        tol = (n * k * (E + d + 64) * U) * 4 + n * k * (4 * h * d ** 0.5) ** 3
        got = hi[4] - lo[4]
        say(f"    {got:.6e} against {want:.6e}, tolerance {tol:.1e}")
        assert abs(got - want) <= tol
