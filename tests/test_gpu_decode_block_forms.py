"""DecodeBlock with the forms of norms that it may lack: without a norm in
front of the next block, h itself is the layer's input, the head's input and,
without a head, the result.

Tolerances (derived, not measured), from each stage's stored input: the layer
rounds its hidden and its output once (2^-8 each of bf16, 2^-13 for the
float32 steps in between), the residual update its row once, the head sums in
float32.  Choices: a logit is off by a float32 sum of d terms."""

import numpy as np
import pytest

from oracle import serve_oracle as S
from tests.gpu_support import say
from tests.test_gpu_decode_block import _dec, _f64, _norm, _norm64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _layer(u, wg, w, idx, renorm):
    """(y, its magnitudes' sum) of the layer for given choices, float64."""
    z = u @ wg.T
    e = np.exp(z - z.max(axis=1, keepdims=True))
    p = np.take_along_axis(e / e.sum(axis=1, keepdims=True), idx, axis=1)
    p = p / p.sum(axis=1, keepdims=True) if renorm else p
    y, size = np.zeros_like(u), np.zeros_like(u)
    for t in range(len(u)):
        for j, at in enumerate(idx[t]):
            g, v = w["1"][at] @ u[t], w["3"][at] @ u[t]
            h = g / (1 + np.exp(-g)) * v
            y[t] += p[t, j] * (w["2"][at] @ h)
            size[t] += p[t, j] * (np.abs(w["2"][at]) @ np.abs(h))
    return y, size


def _check_choices(u, wg, idx):
    """The choices are the k largest logits, largest first, up to their rounding."""
    z = u @ wg.T
    ez = 2 * (u.shape[1] / 32 + 64) * U * (np.abs(u) @ np.abs(wg).T).max(axis=1)
    for t in range(len(u)):
        assert len(set(idx[t])) == len(idx[t]) and (np.diff(z[t, idx[t]]) <= ez[t]).all()
        assert np.delete(z[t], idx[t]).max(initial=-np.inf) <= z[t, idx[t]].min() + ez[t]


@pytest.mark.parametrize("post", ["rms", "layer", None])
@pytest.mark.parametrize("m", [None, 200])
@pytest.mark.parametrize("n", [1, 4, 5, 16])
def test_steps_without_a_norm_in_front(n, m, post):
    import torch
    from mixture_experts_layer_wave_amd.device import DecodeBlock

    d, E, k, f = 128, 8, 2, 192
    say(f"[decode block, no norm in front] n {n} head {m} post {post}")
    rng = np.random.default_rng(70 + n)
    bf = lambda *s, scale=1.0: torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).cuda().bfloat16()
    gate = torch.from_numpy((0.5 + 0.1 * rng.standard_normal(d)).astype(np.float32)).cuda()
    blk = DecodeBlock(n, bf(E, d, scale=d ** -0.5), bf(E, f, d, scale=d ** -0.5), bf(E, f, d, scale=d ** -0.5),
                      bf(E, d, f, scale=f ** -0.5), k, scale=0.75, gate=gate,
                      post=None if post is None else _norm(rng, d, post), pre=None,
                      head=None if m is None else bf(m, d, scale=d ** -0.5))
    blk.u.zero_()
    blk.h.copy_(bf(n, d))
    w = {key: _dec(blk.experts["w" + key], blk.experts["s" + key]) for key in "132"}
    wg = _f64(blk.wg)
    for step in range(3):
        h0 = _f64(blk.h)
        out = blk.step()
        torch.cuda.synchronize()
        idx = blk.idx.cpu().numpy()
        _check_choices(h0, wg, idx)
        y, size = _layer(h0, wg, w, idx, True)
        z = _f64(blk.z)
        assert (np.abs(z - y) <= 2.0 ** -8 * np.abs(y) + (2.0 ** -8 + 2.0 ** -13) * size).all(), step
        b = S.block_norm(h0, z, 0.75, _f64(gate), None if post is None else _norm64(blk.post), None)
        slack = 2.0 ** -14 * (1 + np.abs(b["h"]).max(axis=1, keepdims=True))
        assert (np.abs(_f64(blk.h) - b["h"]) <= 2.0 ** -8 * np.abs(b["h"]) + slack).all()
        if m is None:
            assert torch.equal(out, blk.h)
        else:
            h, head = _f64(blk.h), _dec(*blk.head)
            assert (np.abs(_f64(out) - h @ head.T) <= (d / 32 + 64) * U * (np.abs(h) @ np.abs(head).T)).all()


def test_no_norm_in_front_in_a_graph():
    """Three blocks in a row over one h, captured and replayed."""
    import torch
    from mixture_experts_layer_wave_amd.device import DecodeBlock

    n, d, E, k, f = 3, 64, 4, 2, 96
    rng = np.random.default_rng(5)
    bf = lambda *s, scale=1.0: torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).cuda().bfloat16()
    blks = [DecodeBlock(n, bf(E, d, scale=d ** -0.5), bf(E, f, d, scale=d ** -0.5), bf(E, f, d, scale=d ** -0.5),
                        bf(E, d, f, scale=f ** -0.5), k, post=_norm(rng, d, "rms")) for _ in range(3)]
    for b in blks:
        b.u.zero_()
        b.h = blks[0].h
    h0 = bf(n, d)

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
        run()
        torch.cuda.synchronize()
        want = [t.clone() for b in blks for t in (b.h, b.z, b.idx)]
        # (the layer reads what the block before it left)
        y, size = _layer(_f64(h0 * (rep + 1)), _f64(blks[0].wg),
                         {key: _dec(blks[0].experts["w" + key], blks[0].experts["s" + key]) for key in "132"},
                         blks[0].idx.cpu().numpy(), True)
        assert (np.abs(_f64(blks[0].z) - y) <= 2.0 ** -8 * np.abs(y) + (2.0 ** -8 + 2.0 ** -13) * size).all()
        blks[0].h.copy_(h0 * (rep + 1))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((t for b in blks for t in (b.h, b.z, b.idx)), want))
