"""The MXFP4 encoder, the few-token layer, the norms around it and the MXFP4
product run together as a decode step, and the norms around a layer that is
trained: against the float64 oracles, and captured in graphs."""

import numpy as np
import pytest

import oracle
from oracle import serve_oracle as S
from tests.gpu_support import say

pytestmark = pytest.mark.gpu


def _norm(rng, d, kind):
    import torch

    vec = lambda c: torch.from_numpy((c + 0.2 * rng.standard_normal(d)).astype(np.float32)).cuda()
    return dict(kind=kind, weight=vec(1.0), bias=vec(0.0) if kind == "layer" else None, eps=1e-5)


def _f64(t):
    return t.double().cpu().numpy()


def _norm64(v):
    return dict(kind=v["kind"], weight=_f64(v["weight"]), bias=None if v["bias"] is None else _f64(v["bias"]),
                eps=v["eps"])


def _block(n, d, E, k, f, m, seed):
    import torch
    from mixture_experts_layer_wave_amd.device import DecodeBlock

    rng = np.random.default_rng(seed)
    bf = lambda *s, scale=1.0: torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).cuda().bfloat16()
    blk = DecodeBlock(n, bf(E, d, scale=d ** -0.5), bf(E, f, d, scale=d ** -0.5), bf(E, f, d, scale=d ** -0.5),
                      bf(E, d, f, scale=f ** -0.5), k, scale=1.0, gate=None, post=_norm(rng, d, "rms"),
                      pre=_norm(rng, d, "layer"), head=bf(m, d, scale=d ** -0.5))
    blk.h.copy_(bf(n, d))
    blk.u.copy_(bf(n, d))
    return blk


def _dec(q, s):
    q, s = q.cpu().numpy(), s.cpu().numpy()
    return oracle.decode_mxfp4(q.reshape(-1, q.shape[-1]), s.reshape(-1, s.shape[-1])).reshape(*q.shape[:-1], -1)


@pytest.mark.parametrize("n,d,E,k,f,m", [(1, 256, 16, 4, 320, 1000), (7, 128, 8, 2, 192, 333), (16, 64, 4, 1, 96, 50)])
def test_decode_steps(n, d, E, k, f, m):
    import torch

    say(f"[decode block] n {n} d {d} E {E} k {k} f {f} m {m}")
    blk = _block(n, d, E, k, f, m, 5 + n)
    w = {key: _dec(blk.experts["w" + key], blk.experts["s" + key]) for key in "132"}
    head = _dec(*blk.head)
    for step in range(3):
        h0, u0 = _f64(blk.h), _f64(blk.u)
        blk.step()
        torch.cuda.synchronize()
        r = S.few_layer(u0, _f64(blk.wg), None, w["1"], w["3"], w["2"], k, k > 1)
        assert np.array_equal(blk.idx.cpu().numpy(), r["idx"])
        # each stage from the one before it as stored: z is off by a rounding of the hidden
        # (2^-8 of each, over |w2|) and its own
        wh = np.zeros((n, d))
        for t in range(n):
            for j in range(k):
                wh[t] += r["w"][t, j] * np.abs(w["2"][r["idx"][t, j]]) @ np.abs(r["h"][t, j])
        z = _f64(blk.z)
        assert (np.abs(z - r["y"]) <= 2.0 ** -8 * np.abs(r["y"]) + (2.0 ** -8 + 2.0 ** -13) * wh).all()
        b = S.block_norm(h0, z, 1.0, None, _norm64(blk.post), _norm64(blk.pre))
        # one rounding each; float32 before (2^-14 of the rows' size covers sums of 256 and their norms)
        slack = 2.0 ** -14 * (1 + np.abs(b["h"]).max(axis=1, keepdims=True))
        assert (np.abs(_f64(blk.h) - b["h"]) <= 2.0 ** -8 * np.abs(b["h"]) + slack).all()
        assert (np.abs(_f64(blk.u) - b["u"]) <= 2.0 ** -8 * np.abs(b["u"]) + 4 * slack).all()
        u = _f64(blk.u)
        assert (np.abs(_f64(blk.logits) - u @ head.T) <= (d / 32 + 64) * 2.0 ** -24 * (np.abs(u) @ np.abs(head).T)).all()


def test_decode_graph_of_several_blocks():
    """Four blocks in one graph with one workspace between them, replayed with
    eager steps in between."""
    import torch

    blks = [_block(3, 128, 8, 2, 160, 200, 40 + i) for i in range(4)]
    for b in blks[1:]:
        b.h, b.u = blks[0].h, blks[0].u
        b.ws = blks[0].ws
    h0, u0 = blks[0].h.clone(), blks[0].u.clone()

    def run():
        for b in blks:
            b.step()

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(3):
        blks[0].h.copy_(h0 * (rep + 1))
        blks[0].u.copy_(u0)
        run()
        torch.cuda.synchronize()
        want = [t.clone() for b in blks for t in (b.h, b.u, b.z, b.logits, b.idx)]
        blks[0].h.copy_(h0 * (rep + 1))
        blks[0].u.copy_(u0)
        blks[0].ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((t for b in blks for t in (b.h, b.u, b.z, b.logits, b.idx)), want))


def test_training_step_with_norms_around_the_layer():
    """h, u = norms(x0, z0); y = layer(u); h2 = h + post(y): the gradient of a
    weighted sum of h2 through both norms and the trained layer, against
    differences of the library's own forward pass (float32)."""
    import torch
    from mixture_experts_layer_wave_amd import binding as B
    from mixture_experts_layer_wave_amd import workloads as W
    from mixture_experts_layer_wave_amd.device import TrainingLayer

    wl = W.Workload("around", 24, 40, 4, 2, 56, "f32", "f32", 91, 92)
    L = TrainingLayer(W.make_layer(wl, use_fixture=False, cache=False), alpha=0.0)
    n, d = L.n, L.d
    rng = np.random.default_rng(8)
    vec = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()
    x0, z0, r = vec(n, d), vec(n, d), vec(n, d)
    gate = 1 + 0.1 * vec(d)
    n1, n2, n3 = _norm(rng, d, "rms"), _norm(rng, d, "rms"), _norm(rng, d, "layer")
    h, h2 = torch.empty_like(x0), torch.empty_like(x0)
    s1, s2 = torch.empty((4, n), device="cuda"), torch.empty((4, n), device="cuda")

    def forward():
        B.moe_block_norm(n, d, x0, z0, "f32", 1.0, gate, n1, n2, h, L.x, s1)
        y = L.forward_train()
        B.moe_block_norm(n, d, h, y, "f32", 0.5, None, n3, None, h2, None, s2)
        return float((h2.double() * r.double()).sum())

    forward()
    e = lambda: torch.empty_like(x0)
    dh, dy, dx, dz = e(), e(), e(), e()
    p = [torch.empty(d, device="cuda") for _ in range(6)]
    nb = B.moe_block_norm_backward_workspace_bytes(n, d)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    B.moe_block_norm_backward(n, d, r, None, L.y, h2, "f32", 0.5, None, n3, None, s2, dh, dy, None, p[0], p[1], None,
                              None, ws, nb)
    g = L.backward(dy)
    B.moe_block_norm_backward(n, d, dh, g["x"], z0, h, "f32", 1.0, gate, n1, n2, s1, dx, dz, p[2], p[3], None, p[4],
                              None, ws, nb)
    torch.cuda.synchronize()
    idx = L.idx.clone()
    for leaf, grad in ((x0, dx), (z0, dz), (gate, p[2]), (n1["weight"], p[3]), (n2["weight"], p[4]),
                       (n3["weight"], p[0]), (n3["bias"], p[1]), (L.w["w1"], g["w1"])):
        v = torch.randn(leaf.shape, generator=torch.Generator().manual_seed(3)).cuda()
        keep, eps = leaf.clone(), 2.0 ** -9
        leaf.copy_(keep + eps * v)
        hi = forward()
        same = torch.equal(L.idx, idx)
        leaf.copy_(keep - eps * v)
        lo = forward()
        same = same and torch.equal(L.idx, idx)
        leaf.copy_(keep)
        if not same:
            continue  # a step across a routing border has no difference quotient
        want = float((grad.double() * v.double()).sum())
        # eps^2 of the curvature, and float32 rounding of about 1000 terms over eps
        assert abs((hi - lo) / (2 * eps) - want) <= 1e-2 * abs(want) + 5e-2
