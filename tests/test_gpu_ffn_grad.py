"""GPU parity of moe_expert_up_save and moe_grouped_ffn_backward with the
float64 oracle, element by element.

Tolerances (derived, not measured).  half = half a step of the stored type
(2^-8 of the value for bf16, 2^-24 for float32), U = 2^-24.  A float32 sum of
K products is off by at most (K + 32) U of the sum of their magnitudes (32
for the few operations around it).  The gradient's intermediates dg, du and
w silu(g) u carry that error of their own product plus one rounding to the
stored type, and each output adds its own sum and its own rounding.  silu and
silu' are at most 1.1 in slope, and their hardware exponent and reciprocal
are off by a few U.  The bounds are worst cases, so the relative 2-norm is
held too: two independent roundings of at most `half` each have a root mean
square of half sqrt(2 / 3) at most, float32 sums a few hundred U."""

import numpy as np
import pytest

import oracle
from tests.gpu_support import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
NORM = {"bf16": 2.0 ** -8 * (2 / 3) ** 0.5, "f32": 256 * U}

# silu and silu' below float32's range.  1 / (1 + e^-g) is 0 as soon as e^-g
# overflows or its reciprocal is subnormal, that is from e^-g > 2^126 on, g <
# -87.33; the true silu(g) = g / (1 + e^-g) and silu'(g) = s (1 + g (1 - s))
# there are at most 87.34 e^-87.33 = 87.34 * 2^-126 < 2^-119 in size, and
# smaller further down.  So each is off by at most 2^-119 there.
TINY = 2.0 ** -119

# n, d, E, k, d_ff, skew of the routing (large: most experts get no row)
SHAPES = {
    "bf16": [(1, 8, 1, 1, 8, 0), (1, 64, 4, 2, 72, 0), (3, 136, 5, 2, 200, 0), (300, 136, 5, 2, 200, 0),
             (70, 64, 1, 1, 72, 0), (50, 64, 6, 6, 64, 0), (40, 64, 300, 8, 32, 0), (700, 320, 8, 2, 448, 2),
             (257, 512, 3, 1, 776, 0), (520, 264, 2, 2, 520, 0), (1200, 72, 16, 2, 264, 6)],
    "f32": [(1, 1, 1, 1, 1, 0), (2, 3, 2, 2, 5, 0), (33, 12, 5, 2, 20, 0), (100, 65, 3, 2, 97, 0),
            (301, 70, 7, 3, 131, 4), (65, 64, 70, 1, 64, 0)],
}
CASES = [(t,) + s for t in SHAPES for s in SHAPES[t]]


def _t(a, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)


def _f64(t):
    return t.double().cpu().numpy()


class Batch:
    """A routed batch on the GPU, its dispatch by the library, and float64
    copies of what is stored."""

    def __init__(self, dtype, n, d, E, k, f, skew, seed=0, bad=0.0):
        import torch
        from mixture_experts_layer_wave_amd import binding as B

        rng = np.random.default_rng(seed + 7 * n + d + E)
        self.dtype, self.n, self.d, self.E, self.k, self.f, self.R = dtype, n, d, E, k, f, n * k
        self.shape = (n, d, E, k, f)
        z = rng.standard_normal((n, E)) - skew * np.log1p(np.arange(E))
        idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
        if bad:
            idx[rng.random((n, k)) < bad] = E + 3
        self.idx = torch.from_numpy(idx).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.counts, self.offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        self.perm, self.inv = torch.empty(self.R, **i32), torch.empty((n, k), **i32)
        B.moe_dispatch(self.shape, self.idx, self.counts, self.offsets, self.perm, self.inv)
        self.w = _t(0.1 + rng.random((n, k)), "f32")
        self.x, self.dy = _t(rng.standard_normal((n, d)), dtype), _t(rng.standard_normal((n, d)), dtype)
        self.w1, self.w3 = (_t(rng.standard_normal((E, f, d)) / d ** 0.5, dtype) for _ in range(2))
        self.w2 = _t(rng.standard_normal((E, d, f)) / f ** 0.5, dtype)
        self.host = {key: _f64(getattr(self, key)) for key in ("w", "x", "dy", "w1", "w3", "w2")}
        for key in ("perm", "inv", "offsets"):
            self.host[key] = getattr(self, key).cpu().numpy()
        self.live = int(self.host["offsets"][E])

    def weights(self, **kw):
        return dict(dtype=self.dtype, w1=self.w1, w3=self.w3, w2=self.w2, **kw)

    def rows(self, cols):
        """An output [R + 1][cols] of sevens."""
        import torch

        return torch.full((self.R + 1, cols), 7.0, dtype=self.x.dtype, device="cuda")

    def up(self, a=None, perm=True, weights=None):
        import torch
        from mixture_experts_layer_wave_amd import binding as B

        h, g, u = (self.rows(self.f) for _ in range(3))
        B.moe_expert_up_save(self.shape, self.x if a is None else a, self.dtype, self.perm if perm else None,
                             self.offsets, weights or self.weights(), h, g, u)
        torch.cuda.synchronize()
        for t in (h, g, u):
            assert (t[self.live:] == 7).all()  # rows behind the last pile are left as they were
        return h, g, u

    def back(self, g, u, a=None, dy=None, perm=True, weights=None):
        import torch
        from mixture_experts_layer_wave_amd import binding as B

        nb = B.moe_grouped_ffn_backward_workspace_bytes(self.shape, self.dtype)
        ws = torch.full((nb + 256,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns, and a guard
        da = self.rows(self.d)
        dw = [torch.full((m.numel() + 8,), 7.0, dtype=m.dtype, device="cuda") for m in (self.w1, self.w3, self.w2)]
        if weights:  # a slot table: gradients are by logical expert
            dw = [torch.full((self.E * self.d * self.f + 8,), 7.0, dtype=self.x.dtype, device="cuda")
                  for _ in range(3)]
        dtw = torch.full((self.R + 4,), 7.0, device="cuda")
        B.moe_grouped_ffn_backward(
            self.shape, self.dy if dy is None else dy, self.x if a is None else a, self.dtype,
            self.perm if perm else None, self.inv if perm else None, self.w if perm else None, self.offsets,
            weights or self.weights(), g, u, da, *dw, dtw if perm else None, ws, nb)
        torch.cuda.synchronize()
        assert (ws[nb:] == 255).all() and (da[self.live:] == 7).all() and (dtw[self.R:] == 7).all()
        for m in dw:
            assert (m[-8:] == 7).all()
        E, d, f = self.E, self.d, self.f
        return (da, dw[0][:-8].view(E, f, d), dw[1][:-8].view(E, f, d), dw[2][:-8].view(E, d, f),
                dtw[:self.R].view(self.n, self.k) if perm else None)


def check(name, got, ref, tol, dtype):
    assert np.isfinite(got).all(), name
    err = np.abs(got - ref)
    worst = float(np.max(err / np.maximum(tol, 1e-300), initial=0.0))
    norm = float(np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300)) if err.size else 0.0
    say(f"    {name}: largest error / tolerance {worst:.3f}, relative norm {norm:.2e}")
    assert worst <= 1.0, name
    assert norm <= NORM[dtype] or not np.linalg.norm(ref), name


def check_up(b, got, a, perm):
    H = b.host
    half, src = HALF[b.dtype], (H["perm"] if perm else np.arange(b.R))
    hr, gr, ur = oracle.expert_up(a, src, H["offsets"], H["w1"], H["w3"])
    ga, ua = np.zeros_like(gr), np.zeros_like(ur)
    for e in range(b.E):
        r = np.arange(H["offsets"][e], H["offsets"][e + 1])
        ga[r], ua[r] = np.abs(a[src[r]]) @ np.abs(H["w1"][e]).T, np.abs(a[src[r]]) @ np.abs(H["w3"][e]).T
    L = slice(0, b.live)
    acc = (b.d + 32) * U
    hr, gr, ur, ga, ua = hr[L], gr[L], ur[L], ga[L], ua[L]
    check("g", _f64(got[1])[L], gr, half * np.abs(gr) + acc * ga, b.dtype)
    check("u", _f64(got[2])[L], ur, half * np.abs(ur) + acc * ua, b.dtype)
    silu = np.abs(gr * oracle.train_oracle.sigmoid(gr))
    check("h", _f64(got[0])[L], hr, half * np.abs(hr) + acc * (1.1 * ga * np.abs(ur) + silu * ua) +
          acc * acc * ga * ua, b.dtype)


def check_back(b, got, g, u, a, dy, perm, w=None):
    """w: weights [E] to use in the oracle (a slot table resolved)."""
    H = b.host
    w1, w3, w2 = w or (H["w1"], H["w3"], H["w2"])
    g64, u64 = _f64(g)[:b.R], _f64(u)[:b.R]
    pi = (H["perm"], H["inv"], H["w"]) if perm else (None, None, None)
    da, dw1, dw3, dw2, dtw = oracle.grouped_ffn_grad(dy, a, *pi, H["offsets"], w1, w3, w2, g64, u64)
    half = HALF[b.dtype]
    wr = oracle.row_weights(H["inv"], H["w"], b.R) if perm else np.ones(b.R)
    ida, idw = np.zeros_like(da), np.zeros(b.R)
    t1, t3, t2 = np.zeros_like(dw1), np.zeros_like(dw3), np.zeros_like(dw2)
    for e in range(b.E):
        r = np.arange(H["offsets"][e], H["offsets"][e + 1])
        src = H["perm"][r] if perm else r
        x, dd, W = np.abs(a[src]), dy[src], np.abs(wr[r, None])
        ge, ue = g64[r], u64[r]
        s = oracle.train_oracle.sigmoid(ge)
        silu, h = ge * s, np.abs(ge * s * ue)
        dh = dd @ w2[e]
        mag = np.abs(dd) @ np.abs(w2[e])
        dg, du = np.abs(W * dh * ue * s * (1 + ge * (1 - s))), np.abs(W * dh * silu)
        acc = (b.d + 32) * U
        eg = half * dg + acc * W * mag * np.abs(ue) * 1.1 + TINY * W * mag * np.abs(ue)
        eu = half * du + acc * W * mag * np.abs(silu) + TINY * W * mag
        eh = (half + 32 * U) * W * h + TINY * W * np.abs(ue)
        K = (2 * b.f + 32) * U
        ida[r] = (eg + K * (dg + eg)) @ np.abs(w1[e]) + (eu + K * (du + eu)) @ np.abs(w3[e])
        idw[r] = ((b.d + b.f + 64) * U * mag * h).sum(axis=1)
        K = (len(r) + 32) * U
        t1[e], t3[e] = (eg + K * (dg + eg)).T @ x, (eu + K * (du + eu)).T @ x
        t2[e] = np.abs(dd).T @ (eh + K * (W * h + eh))
    L = slice(0, b.live)
    check("da", _f64(got[0])[L], da[L], half * np.abs(da[L]) + ida[L], b.dtype)
    for name, o, ref, t in (("dw1", got[1], dw1, t1), ("dw3", got[2], dw3, t3), ("dw2", got[3], dw2, t2)):
        check(name, _f64(o), ref, (half + U) * np.abs(ref) + t, b.dtype)
    if perm:
        ok = (H["inv"] >= 0) & (H["inv"] < b.R)
        tol = np.where(ok, idw[np.where(ok, H["inv"], 0)], 0.0)
        check("dtopk_w", _f64(got[4]), dtw, tol, "f32")
    empty = np.diff(H["offsets"]) == 0
    for o in got[1:4]:
        assert not _f64(o)[empty].any()


@pytest.mark.parametrize("dtype,n,d,E,k,f,skew", CASES)
def test_up_and_gradient(dtype, n, d, E, k, f, skew):
    import torch

    say(f"[ffn grad] {dtype} n={n} d={d} E={E} k={k} d_ff={f}")
    b = Batch(dtype, n, d, E, k, f, skew)
    up = b.up()
    check_up(b, up, b.host["x"], True)
    got = b.back(up[1], up[2])
    check_back(b, got, up[1], up[2], b.host["x"], b.host["dy"], True)
    # the same calls again give the same bits
    for p, q in zip(up + got, b.up() + b.back(up[1], up[2])):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype,n,d,E,k,f,skew", [
    ("bf16", 300, 136, 5, 2, 200, 3), ("bf16", 1, 64, 3, 1, 64, 0), ("bf16", 600, 256, 1, 1, 512, 0),
    ("f32", 90, 33, 4, 2, 61, 3), ("f32", 130, 64, 1, 1, 100, 0)])
def test_pile_rows_without_a_combine(dtype, n, d, E, k, f, skew):
    """perm = NULL: a and dy are pile rows; with E = 1 the dense block."""
    import torch

    say(f"[ffn grad, pile rows] {dtype} n={n} E={E}")
    b = Batch(dtype, n, d, E, k, f, skew, seed=5)
    rng = np.random.default_rng(n)
    a, dy = _t(rng.standard_normal((b.R, d)), dtype), _t(rng.standard_normal((b.R, d)), dtype)
    up = b.up(a=a, perm=False)
    check_up(b, up, _f64(a), False)
    got = b.back(up[1], up[2], a=a, dy=dy, perm=False)
    check_back(b, got, up[1], up[2], _f64(a), _f64(dy), False)
    if E == 1:  # the forward pass that keeps nothing gives the same hidden
        from mixture_experts_layer_wave_amd import binding as B

        if dtype == "bf16":
            h = b.rows(f)
            B.moe_expert_up(b.shape, a, dtype, None, b.offsets, b.weights(), h)
            torch.cuda.synchronize()
            assert torch.equal(h, up[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [0.3, 1.0])
def test_pairs_outside_the_experts(dtype, bad):
    """Pairs with ids outside [0, E) have no pile row: their dtopk_w is 0, the
    rows behind the last pile stay as they were, and with no pair left every
    weight gradient is zero."""
    say(f"[ffn grad, pairs without a pile] {dtype} {bad}")
    b = Batch(dtype, 120, 72, 6, 3, 88, 0, seed=9, bad=bad)
    up = b.up()
    got = b.back(up[1], up[2])
    if bad < 1:
        check_back(b, got, up[1], up[2], b.host["x"], b.host["dy"], True)
    else:
        assert b.live == 0 and all(not _f64(o).any() for o in got[1:])
    gone = b.host["inv"] < 0
    assert gone.any() and not _f64(got[4])[gone].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slot_table(dtype):
    """Weights read through a slot table (entries out of range are clamped);
    gradients by logical expert."""
    import torch

    say(f"[ffn grad, slots] {dtype}")
    b = Batch(dtype, 90, 64, 4, 2, 96, 0, seed=11)
    table = torch.tensor([2, 9, 0, 2], dtype=torch.int32, device="cuda")
    use = [2, 3, 0, 2]
    weights = b.weights(slot=table, n_slots=4)
    plain = [b.host[key][use] for key in ("w1", "w3", "w2")]
    up = b.up(weights=weights)
    got = b.back(up[1], up[2], weights=weights)
    check_back(b, got, up[1], up[2], b.host["x"], b.host["dy"], True, w=plain)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_pre_activations(dtype):
    """Pre-activations at which exp overflows or underflows give the limits of
    silu and silu': 0 below, g and 1 above."""
    say(f"[ffn grad, extreme pre-activations] {dtype}")
    b = Batch(dtype, 64, 64, 2, 1, 64, 0, seed=13)
    g, u = b.rows(b.f), b.rows(b.f)
    u[:b.R] = 1.0
    values = [-1e4, -200.0, -90.0, -30.0, 0.0, 30.0, 90.0, 200.0]
    for j in range(b.f):
        g[:b.R, j] = values[j % len(values)]
    got = b.back(g, u)
    check_back(b, got, g, u, b.host["x"], b.host["dy"], True)


@pytest.mark.parametrize("dtype,n,d,E,k,f,skew", [
    ("bf16", 2100, 256, 2, 2, 2000, 1),  # one block per CU, da's sum over K in ranges
    ("bf16", 8000, 1288, 1, 1, 1288, 0),  # the same, da in one range
    ("f32", 1300, 40, 2, 2, 72, 2)])  # a pile longer than the tokens a block holds at once
def test_long_piles(dtype, n, d, E, k, f, skew):
    say(f"[ffn grad, long piles] {dtype} n={n} d={d} E={E} d_ff={f}")
    b = Batch(dtype, n, d, E, k, f, skew, seed=19)
    up = b.up()
    check_up(b, up, b.host["x"], True)
    check_back(b, b.back(up[1], up[2]), up[1], up[2], b.host["x"], b.host["dy"], True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_token_twice_in_one_pile(dtype):
    """Two slots of a token with the same expert are two pile rows, each with
    its own weight and its own gradient of it."""
    from mixture_experts_layer_wave_amd import binding as B

    say(f"[ffn grad, repeated ids] {dtype}")
    b = Batch(dtype, 90, 72, 4, 3, 88, 0, seed=23)
    b.idx[::2, 2] = b.idx[::2, 0]
    B.moe_dispatch(b.shape, b.idx, b.counts, b.offsets, b.perm, b.inv)
    for key in ("perm", "inv", "offsets"):
        b.host[key] = getattr(b, key).cpu().numpy()
    up = b.up()
    check_up(b, up, b.host["x"], True)
    check_back(b, b.back(up[1], up[2]), up[1], up[2], b.host["x"], b.host["dy"], True)


def test_weights_past_32_bit_offsets():
    """300 experts of 2704 x 2704: the last ones' weights and gradients lie
    more than 2^32 bytes and 2^31 elements in."""
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    say("[ffn grad, offsets past 32 bits]")
    n, d, E, f = 5, 2704, 300, 2704
    bf = dict(dtype=torch.bfloat16, device="cuda")
    small = Batch("bf16", n, d, 3, 1, f, 0, seed=29)
    where = [0, 150, 299]
    big = [torch.zeros(E, *m.shape[1:], **bf) for m in (small.w1, small.w3, small.w2)]
    for m, t in zip(big, (small.w1, small.w3, small.w2)):
        m[where] = t
    out = [torch.full_like(m, 7.0) for m in big]
    shape = (n, d, E, 1, f)
    idx = torch.tensor(where, dtype=torch.int32, device="cuda")[small.idx.long()].to(torch.int32).contiguous()
    counts, offsets = (torch.empty(E + i, dtype=torch.int32, device="cuda") for i in (0, 1))
    B.moe_dispatch(shape, idx, counts, offsets, small.perm, small.inv)
    weights = dict(dtype="bf16", w1=big[0], w3=big[1], w2=big[2])
    h, g, u = (small.rows(f) for _ in range(3))
    B.moe_expert_up_save(shape, small.x, "bf16", small.perm, offsets, weights, h, g, u)
    da, dtw = small.rows(d), torch.empty(n, 1, device="cuda")
    nb = B.moe_grouped_ffn_backward_workspace_bytes(shape, "bf16")
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    B.moe_grouped_ffn_backward(shape, small.dy, small.x, "bf16", small.perm, small.inv, small.w, offsets, weights, g,
                               u, da, *out, dtw, ws, nb)
    torch.cuda.synchronize()
    check_up(small, (h, g, u), small.host["x"], True)
    got = (da, *(m[where] for m in out), dtw)
    check_back(small, got, g, u, small.host["x"], small.host["dy"], True)
    rest = torch.ones(E, dtype=torch.bool, device="cuda")
    rest[where] = False
    for m in out:
        assert not m[rest].any()


def test_gradient_against_differences():
    """d/d step of the loss sum(y dy), with y from the library's own float32
    forward pass (up, down, combine), along a random direction of every input."""
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    say("[ffn grad, differences]")
    n, d, E, k, f = 40, 24, 4, 2, 36
    b = Batch("f32", n, d, E, k, f, 0, seed=17)
    _, g, u = b.up()
    da, dw1, dw3, dw2, dtw = b.back(g, u)
    dx = torch.zeros(n, d, device="cuda", dtype=torch.float64)
    for j in range(k):
        dx += da[b.inv[:, j].long()].double()

    def loss(x, w1, w3, w2, w):
        h = torch.empty(b.R, f, device="cuda")
        yp, y = torch.empty(b.R, d, device="cuda"), torch.empty(n, d, device="cuda")
        ws = dict(dtype="f32", w1=w1, w3=w3, w2=w2)
        B.moe_expert_up(b.shape, x, "f32", b.perm, b.offsets, ws, h)
        B.moe_expert_down(b.shape, h, b.offsets, ws, yp)
        B.moe_combine(b.shape, yp, "f32", b.inv, w, y, "f32")
        torch.cuda.synchronize()
        return y.double(), float((y.double().abs() * b.dy.double().abs()).sum())

    at = [b.x, b.w1, b.w3, b.w2, b.w]
    for i, (var, grad) in enumerate(zip(at, (dx, dw1, dw3, dw2, dtw))):
        rng = np.random.default_rng(i)
        v = _t(np.sign(rng.standard_normal(tuple(var.shape))), "f32") * 2.0 ** -7
        yp, size = loss(*[t + v if j == i else t for j, t in enumerate(at)])
        ym, _ = loss(*[t - v if j == i else t for j, t in enumerate(at)])
        got = float(((yp - ym) * b.dy.double()).sum())
        step = ((var + v).double() - (var - v).double())
        want = float((grad.double() * step).sum())
        # the forward's float32 rounding, (d + f + 64) U of the terms' size, where the
        # terms of y are up to sqrt(f) times y; and the third-order term: a
        # relative step s = 2^-7 per element leaves s^2 of the difference's size
        # of order sum |grad| |step|
        tol = 4 * (d + f + 64) * U * size * f ** 0.5 + 2.0 ** -14 * 8 * float((grad.double() * step).abs().sum())
        say(f"    input {i}: {got:.6e} against {want:.6e}, tolerance {tol:.1e}")
        assert abs(got - want) <= tol
