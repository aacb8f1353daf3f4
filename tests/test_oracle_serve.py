"""The oracle of the MXFP4 encoder, the few-token layer and the norms around a
block, against something other than itself (no GPU)."""

import numpy as np
import pytest
import torch

import oracle
from oracle import serve_oracle as S


def test_mxfp4_encoder_against_exhaustive_search():
    rng = np.random.default_rng(1)
    mags = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    values = np.concatenate([mags, -mags])
    x = rng.standard_normal((40, 64)) * np.exp2(rng.integers(-60, 60, (40, 1)))
    x[3, :32] = 0.0
    x[4, :32] = np.arange(32) * 0.25  # ties of every border, top value 7.75
    x[5, 1:32] = 0.0                  # one value alone
    q, s = S.encode_mxfp4(x)
    got = oracle.decode_mxfp4(q, s)
    for i in range(40):
        for b in range(2):
            v = x[i, 32 * b: 32 * b + 32]
            top = np.abs(v).max()
            if top == 0:
                assert s[i, b] == 0 and (q[i, 16 * b: 16 * b + 16] == 0).all()
                continue
            # the scale: the largest power of two X with 4 * 2^X <= top
            X = max(X for X in range(-127, 127) if 4.0 * 2.0 ** X <= top)
            assert s[i, b] == X + 127
            near = np.abs(v[:, None] / 2.0 ** X - values).min(axis=1)
            r = got[i, 32 * b: 32 * b + 32]
            clipped = np.abs(v) > 6 * 2.0 ** X
            assert np.array_equal(np.abs(r / 2.0 ** X - v / 2.0 ** X)[~clipped], near[~clipped])
            assert (np.abs(r[clipped]) == 6 * 2.0 ** X).all() and (np.sign(r) * np.sign(v) >= 0).all()
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    row = got[4, :32]
    for v, want in ((.25, 0), (.75, 1), (1.25, 1), (1.75, 2), (2.5, 2), (3.5, 4), (5, 4)):
        assert row[int(v * 4)] == want, v


def test_mxfp4_encoder_edges():
    x = np.zeros((5, 32))
    x[0, 3], x[1, 4], x[2, 5] = np.inf, np.nan, 2.0 ** -149
    x[3, 0] = (2 - 2.0 ** -23) * 2.0 ** 127
    x[4, :2] = 2.0 ** -126, -2.0 ** -127
    q, s = S.encode_mxfp4(x)
    assert s[0, 0] == s[1, 0] == 255 and (q[:2] == 0).all()
    assert np.isnan(oracle.decode_mxfp4(q[:2], s[:2])).all()
    assert s[2, 0] == 0 and (q[2] == 0).all()
    assert s[3, 0] == 252 and q[3, 0] == 7
    assert s[4, 0] == 0 and list(oracle.decode_mxfp4(q, s)[4, :2]) == [2.0 ** -126, -2.0 ** -127]


def test_few_layer_is_the_dense_layer():
    rng = np.random.default_rng(2)
    n, d, E, k, f = 5, 24, 6, 3, 40
    L = dict(n=n, d=d, E=E, k=k, d_ff=f, renorm=True, x_dtype="f32", w_dtype="f32",
             x=rng.standard_normal((n, d)).astype(np.float32), wg=rng.standard_normal((E, d)).astype(np.float32),
             bias=rng.standard_normal(E).astype(np.float32),
             **{key: rng.standard_normal((E, *shape)).astype(np.float32)
                for key, shape in (("w1", (f, d)), ("w3", (f, d)), ("w2", (d, f)))})
    ref = oracle.forward(L, k)
    got = S.few_layer(*(np.asarray(L[key], np.float64) for key in ("x", "wg", "bias", "w1", "w3", "w2")), k, True)
    assert np.array_equal(got["idx"], ref["idx"])
    np.testing.assert_allclose(got["y"], ref["y"], rtol=1e-12, atol=1e-12)


def _norms(rng, d, kinds):
    return [None if kind is None else dict(kind=kind, weight=1 + .3 * rng.standard_normal(d),
                                           bias=rng.standard_normal(d) if kind == "layer" else None, eps=1e-5)
            for kind in kinds]


@pytest.mark.parametrize("kinds", [("layer", "rms"), ("rms", "layer"), (None, "layer"), ("layer", None), (None, None)])
@pytest.mark.parametrize("gated", [False, True])
def test_block_norm_gradient(kinds, gated):
    rng = np.random.default_rng(3)
    n, d, scale = 4, 9, 1.3
    x, z, dh, du = (rng.standard_normal((n, d)) for _ in range(4))
    gate = rng.standard_normal(d) if gated else None
    post, pre = _norms(rng, d, kinds)
    fwd = S.block_norm(x, z, scale, gate, post, pre)
    got = S.block_norm_grad(dh, du, z, fwd["h"], scale, gate, post, pre, fwd["stats"])

    # torch's autograd, with torch's own layer norm
    leaf = lambda a: None if a is None else torch.tensor(a, requires_grad=True)
    tx, tz, tg = leaf(x), leaf(z), leaf(gate)
    tp = [None if v is None else (leaf(v["weight"]), leaf(v["bias"])) for v in (post, pre)]

    def norm(v, kind, p):
        if kind is None:
            return v
        if kind == "layer":
            return torch.nn.functional.layer_norm(v, (d,), p[0], p[1], 1e-5)
        return torch.nn.functional.rms_norm(v, (d,), p[0], 1e-5)

    v = norm(tz, kinds[0], tp[0])
    h = scale * tx + (v if tg is None else v * tg)
    loss = (h * torch.tensor(dh)).sum()
    if pre:
        loss = loss + (norm(h, kinds[1], tp[1]) * torch.tensor(du)).sum()
    loss.backward()
    want = dict(dx=tx.grad, dz=tz.grad)
    if gated:
        want["dgate"] = tg.grad
    for name, p in (("post", tp[0]), ("pre", tp[1])):
        if p:
            want[f"d{name}_weight"] = p[0].grad
            if p[1] is not None:
                want[f"d{name}_bias"] = p[1].grad
    for key, ref in want.items():
        np.testing.assert_allclose(got[key], ref.numpy(), rtol=1e-9, atol=1e-9, err_msg=key)

    # and central differences of the forward function
    def f(x_, z_):
        o = S.block_norm(x_, z_, scale, gate, post, pre)
        return (o["h"] * dh).sum() + ((o["u"] * du).sum() if pre else 0.0)

    for name, a in (("dx", x), ("dz", z)):
        for i in ((0, 0), (2, 5), (3, 8)):
            lo, hi = a.copy(), a.copy()
            lo[i] -= 1e-6
            hi[i] += 1e-6
            diff = (f(hi, z) - f(lo, z) if name == "dx" else f(x, hi) - f(x, lo)) / 2e-6
            assert abs(diff - got[name][i]) < 1e-6 * max(1.0, abs(diff))
