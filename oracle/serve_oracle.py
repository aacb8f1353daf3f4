"""Float64 CPU oracle of the MXFP4 encoder, the layer for a few tokens and the
norms around a block (TEST INFRASTRUCTURE).

Each function is written from its formula in plain numpy float64 and shares
no code with the HIP library.  Pinned by ``tests/test_oracle_serve.py``:
the encoder by exhaustive search over the format's values, the norms'
gradient by central differences and by torch's float64 autograd, the layer
by the dense oracle.
"""

from __future__ import annotations

import numpy as np

from .moe_oracle import router_logits, softmax_rows, topk_select, topk_weights
from .train_oracle import sigmoid

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode_mxfp4(x):
    """(codes [rows][cols/2], scales [rows][cols/32]) of the rows of x: the
    shared exponent floor(log2 amax) - 2 (at least -127), each element to the
    nearest magnitude, ties to the even code, at most 6; a block with an
    infinity or a NaN has scale code 255 and codes 0."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    top = np.abs(b).max(axis=2)
    _, e = np.frexp(top)  # top = m 2^e, m in [1/2, 1)
    X = np.where(top > 0, np.maximum(e - 1 - 2, -127), -127)
    v = np.abs(b) / np.exp2(X.astype(np.float64))[:, :, None]
    dist = np.abs(v[..., None] - E2M1)
    best = dist.min(axis=3, keepdims=True)
    # of two magnitudes as near as each other, the one with the even code
    code = np.where(dist == best, np.arange(8) + 8 * (np.arange(8) % 2), 99).min(axis=3) % 8
    code = np.where(v >= 6.0, 7, code) | (np.signbit(b) << 3)
    code = np.where(bad[:, :, None], 0, code).reshape(rows, cols // 2, 2).astype(np.uint8)
    return code[..., 0] | (code[..., 1] << 4), np.where(bad, 255, X + 127).astype(np.uint8)


def few_layer(x, wg, bias, w1, w3, w2, k, renorm):
    """Every intermediate of the layer on float64 matrices (w1 [E][f][d], ..):
    z, idx, w, g and u [n][k][f], h = silu(g) u, y."""
    n, d = x.shape
    z = router_logits(x, wg, bias)
    idx = topk_select(z, k)
    w = topk_weights(softmax_rows(z), idx, renorm)
    f = w1.shape[1]
    g, u, y = np.zeros((n, k, f)), np.zeros((n, k, f)), np.zeros((n, d))
    for t in range(n):
        for j in range(k):
            e = idx[t, j]
            g[t, j], u[t, j] = w1[e] @ x[t], w3[e] @ x[t]
    h = g * sigmoid(g) * u
    for t in range(n):
        for j in range(k):
            y[t] += w[t, j] * (w2[idx[t, j]] @ h[t, j])
    return dict(z=z, idx=idx, w=w, g=g, u=u, h=h, y=y)


def row_norm(v, norm):
    """(norm(v), mean, rstd); norm: dict(kind, weight, bias or None, eps)."""
    v = np.asarray(v, np.float64)
    mean = v.mean(axis=1) if norm["kind"] == "layer" else np.zeros(len(v))
    c = v - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + norm["eps"])
    y = c * rstd[:, None] * norm["weight"]
    return (y if norm["bias"] is None else y + norm["bias"]), mean, rstd


def row_norm_grad(dy, v, mean, rstd, norm):
    """(dv, dweight, dbias)"""
    xh = (v - mean[:, None]) * rstd[:, None]
    t = dy * norm["weight"]
    dv = t - xh * (t * xh).mean(axis=1, keepdims=True)
    if norm["kind"] == "layer":
        dv = dv - t.mean(axis=1, keepdims=True)
    return rstd[:, None] * dv, (dy * xh).sum(axis=0), dy.sum(axis=0)


def block_norm(x, z, scale, gate, post, pre):
    """dict(h, u, stats): h = scale x + gate post(z), u = pre(h)."""
    stats = np.zeros((4, len(x)))
    v = z
    if post:
        v, stats[0], stats[1] = row_norm(z, post)
    h = scale * x + (v if gate is None else v * gate)
    u = None
    if pre:
        u, stats[2], stats[3] = row_norm(h, pre)
    return dict(h=h, u=u, stats=stats)


def block_norm_grad(dh, du, z, h, scale, gate, post, pre, stats):
    """Gradients of block_norm, with h and stats as the forward pass kept
    them: dict(D, dx, dz, dgate, dpost_weight, dpost_bias, dpre_weight,
    dpre_bias); D is the whole gradient with respect to h."""
    out = {}
    D = np.zeros_like(du if dh is None else dh) if dh is None else np.asarray(dh, np.float64)
    if pre:
        dv, out["dpre_weight"], out["dpre_bias"] = row_norm_grad(du, h, stats[2], stats[3], pre)
        D = D + dv
    into = D if gate is None else D * gate
    v = z
    if post:
        out["dz"], out["dpost_weight"], out["dpost_bias"] = row_norm_grad(into, z, stats[0], stats[1], post)
        v = (z - stats[0][:, None]) * stats[1][:, None] * post["weight"]
        v = v if post["bias"] is None else v + post["bias"]
    else:
        out["dz"] = into
    if gate is not None:
        out["dgate"] = (D * v).sum(axis=0)
    out.update(D=D, dx=scale * D)
    return out
