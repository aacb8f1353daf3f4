"""Float64 CPU oracle of the training operators (TEST INFRASTRUCTURE).

Layer norm, the gated expert FFN with its kept pre-activations, and their
gradients and the router's, each written from its formula in plain numpy
float64.  It shares no code with the HIP library.  Every gradient here is
pinned by central differences of the forward functions
(``tests/test_oracle_train.py``) and by torch's float64 autograd through an
independent layer (``tests/test_oracle_train_autograd.py``).

Sources: "How Mixture of Experts Scales Model Parameters"
(zhangchitc.github.io), sections "Routing", "Top-K", "The forward pass:
dispatch, then combine" and "Load balancing", for what is differentiated.
The page holds f_i constant in the auxiliary loss (a count has no gradient).
"""

from __future__ import annotations

import numpy as np


def layer_norm(x, w, b=None, eps=1e-5):
    """(y, mean, rstd) of the rows of x [n][d]."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    y = c * rstd[:, None] * w
    return (y if b is None else y + b), mean, rstd


def layer_norm_grad(dy, x, w, mean, rstd):
    """(dx, dweight, dbias); mean and rstd as the forward pass gave them."""
    xh = (np.asarray(x, np.float64) - mean[:, None]) * rstd[:, None]
    t = dy * w
    dx = rstd[:, None] * (t - t.mean(axis=1, keepdims=True) - xh * (t * xh).mean(axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), np.asarray(dy, np.float64).sum(axis=0)


def sigmoid(g):
    g = np.asarray(g, np.float64)
    return np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))


def expert_up(a, perm, offsets, w1, w3):
    """(h, g, u) of every pile row: g = a W1^T, u = a W3^T, h = silu(g) u.
    Rows outside the piles are NaN (not written)."""
    R = len(perm) if perm is not None else len(a)
    f = w1.shape[1]
    g, u = np.full((R, f), np.nan), np.full((R, f), np.nan)
    for e in range(len(offsets) - 1):
        r = np.arange(offsets[e], offsets[e + 1])
        rows = a[perm[r]] if perm is not None else a[r]
        g[r], u[r] = rows @ w1[e].T, rows @ w3[e].T
    return g * sigmoid(g) * u, g, u


def row_weights(inv, topk_w, R):
    """Combine weight of each pile row (0 for rows that no pair points at)."""
    w = np.zeros(R)
    for t in range(inv.shape[0]):
        for j in range(inv.shape[1]):
            if 0 <= inv[t, j] < R:
                w[inv[t, j]] = topk_w[t, j]
    return w


def grouped_ffn_grad(dy, a, perm, inv, topk_w, offsets, w1, w3, w2, g, u):
    """(da_perm, dw1, dw3, dw2, dtopk_w) of

        y[t] = sum_j topk_w[t][j] yp[inv[t][j]],  yp[r] = (silu(g_r) u_r) W2_e^T,
        g_r = a[perm[r]] W1_e^T,  u_r = a[perm[r]] W3_e^T

    with the pre-activations g, u given.  perm = inv = topk_w = None: a and
    dy are pile rows and y = yp (dtopk_w is None).  Rows of da_perm outside
    the piles are NaN (not written); their pairs' dtopk_w is 0."""
    R = g.shape[0]
    wr = row_weights(inv, topk_w, R) if perm is not None else np.ones(R)
    da = np.full((R, w1.shape[2]), np.nan)
    dw1, dw3, dw2 = np.zeros(w1.shape), np.zeros(w3.shape), np.zeros(w2.shape)
    drow = np.zeros(R)
    for e in range(len(offsets) - 1):
        r = np.arange(offsets[e], offsets[e + 1])
        src = perm[r] if perm is not None else r
        x, d, ge, ue = a[src], dy[src], g[r], u[r]
        s = sigmoid(ge)
        h = ge * s * ue
        dh = d @ w2[e]
        drow[r] = (dh * h).sum(axis=1)
        dh = dh * wr[r, None]
        dg = dh * ue * s * (1.0 + ge * (1.0 - s))
        du = dh * ge * s
        da[r] = dg @ w1[e] + du @ w3[e]
        dw1[e], dw3[e] = dg.T @ x, du.T @ x
        dw2[e] = (d * wr[r, None]).T @ h
    dw = None
    if perm is not None:
        ok = (inv >= 0) & (inv < R)
        dw = np.where(ok, drow[np.where(ok, inv, 0)], 0.0)
    return da, dw1, dw3, dw2, dw


def router_weights(z, idx, renorm):
    """Combine weights of the chosen experts, as a function of the logits."""
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p = p / p.sum(axis=1, keepdims=True)
    w = np.take_along_axis(p, idx, axis=1)
    return (w / w.sum(axis=1, keepdims=True) if renorm else w), p


def router_grad(z, idx, topk_w, dtopk_w, f, alpha, renorm, x, wg, da_perm=None, inv=None):
    """(dlogits, dx, dwg, dbias).  The loss depends on the logits through the
    combine weights of the chosen experts (ids outside [0, E) have no pile
    and no gradient) and, with f given, through alpha E sum_i f_i P_i, f
    constant.  dx also adds the experts' input gradients of each token."""
    n, E = z.shape
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p = p / p.sum(axis=1, keepdims=True)
    ok = (idx >= 0) & (idx < E)
    w, dw = np.where(ok, topk_w, 0.0), np.where(ok, dtopk_w, 0.0)
    D = (w * dw).sum(axis=1, keepdims=True)
    dz = np.zeros((n, E))
    for t in range(n):
        for j in range(idx.shape[1]):
            if ok[t, j]:
                if renorm:
                    dz[t, idx[t, j]] += w[t, j] * (dw[t, j] - D[t, 0])
                else:
                    dz[t, idx[t, j]] += p[t, idx[t, j]] * dw[t, j]
        if not renorm:
            dz[t] -= p[t] * D[t, 0]
    if f is not None:
        dz = dz + alpha * E / n * p * (f - (p * f).sum(axis=1, keepdims=True))
    dx = dz @ wg
    if da_perm is not None:
        for j in range(inv.shape[1]):
            r = inv[:, j]
            good = (r >= 0) & (r < len(da_perm))
            dx[good] += da_perm[r[good]]
    return dz, dx, dz.T @ x, dz.sum(axis=0)
