"""GPU parity of moe_forward_few with the float64 oracle, element by element.

Tolerances (derived, not measured).  With stored inputs exact, every step is
float32: a sum over K terms goes through accumulators fed up to 32 terms (bf16
products) or 4 (float32) at a time, at most K / 32 + 64 (K / 8 + 64) additions
deep, each off by at most 2^-24 of the magnitudes summed.  |silu'| <= 1.1 and
|silu(g)| <= |g| carry the errors of g and u into h; exp2 and the reciprocal are
off by an ulp each, and the exponent's own rounding by |g| 2^-24: 16 + 2 |g| units
of silu.  A weight's relative error is twice the largest logit's, plus the
softmax's.  The hidden times its weight is rounded once to the activations' type,
the output once."""

import numpy as np
import pytest

import oracle
from oracle import serve_oracle as S
from tests.gpu_support import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _torch():
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    return torch, B


class Few:
    """A layer's inputs on the device, and as float64."""

    def __init__(self, n, d, E, k, f, wdt, bias=True, seed=0, renorm=-1):
        torch, B = _torch()
        self.args = n, d, E, k, f, wdt
        self.shape = (n, d, E, k, f, renorm)
        self.wdt, self.act = wdt, "f32" if wdt == "f32" else "bf16"
        self.dt = torch.float32 if wdt == "f32" else torch.bfloat16
        rng = np.random.default_rng(seed + 31 * n + d + E + f)

        def dev(a, dt=None):
            return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(dt or self.dt)

        # logits whose gaps no rounding closes: a token's are a shuffled ladder of
        # steps of 0.05 through the bias-free part, checked below
        self.x, self.wg = dev(rng.standard_normal((n, d))), dev(rng.standard_normal((E, d)) * d ** -0.5)
        self.bias = dev(rng.standard_normal(E), torch.float32) if bias else None
        self.w, self.m64 = dict(dtype=wdt), {}
        for key, rows, cols in (("w1", f, d), ("w3", f, d), ("w2", d, f)):
            v = dev(rng.standard_normal((E * rows, cols)) * cols ** -0.5, torch.float32)
            if wdt == "mxfp4":
                q = torch.empty((E, rows, cols // 2), dtype=torch.uint8, device="cuda")
                s = torch.empty((E, rows, cols // 32), dtype=torch.uint8, device="cuda")
                B.moe_quantize_mxfp4(E * rows, cols, v, "f32", q, s)
                self.w[key], self.w["s" + key[1]] = q, s
            else:
                self.w[key] = v.view(E, rows, cols).to(self.dt)
        self.refresh()

    def refresh(self):
        n, d, E, k, f, wdt = self.args
        for key, rows, cols in (("w1", f, d), ("w3", f, d), ("w2", d, f)):
            if wdt == "mxfp4":
                q, s = self.w[key].cpu().numpy(), self.w["s" + key[1]].cpu().numpy()
                self.m64[key] = oracle.decode_mxfp4(q.reshape(-1, cols // 2), s.reshape(-1, cols // 32)).reshape(-1, rows, cols)
            else:
                self.m64[key] = self.w[key].double().cpu().numpy()

    def ref(self, slot=None):
        n, d, E, k, f, wdt = self.args
        renorm = k > 1 if self.shape[5] < 0 else self.shape[5] == 1
        m = self.m64 if slot is None else {key: v[np.clip(slot, 0, len(v) - 1)] for key, v in self.m64.items()}
        return S.few_layer(self.x.double().cpu().numpy(), self.wg.double().cpu().numpy(),
                           None if self.bias is None else self.bias.double().cpu().numpy(), m["w1"], m["w3"],
                           m["w2"], k, renorm), m

    def buffers(self, out=None):
        torch, B = _torch()
        n, d, E, k, f, wdt = self.args
        out = out or self.act
        self.nb = B.moe_forward_few_workspace_bytes(self.shape, wdt)
        b = dict(y=torch.full((n + 1, d), 7.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda"),
                 idx=torch.full((n + 1, k), -7, dtype=torch.int32, device="cuda"),
                 tw=torch.full((n + 1, k), 7.0, device="cuda"),
                 ws=torch.full((self.nb + 256,), 255, dtype=torch.uint8, device="cuda"), out=out)
        return b

    def call(self, b, stream=None, weights=None):
        _, B = _torch()
        B.moe_forward_few(self.shape, self.x, self.act, self.wg, self.bias, weights or self.w, b["y"], b["out"],
                          b["idx"], b["tw"], b["ws"], self.nb, stream)

    def run(self, out=None, weights=None):
        torch, _ = _torch()
        n = self.args[0]
        b = self.buffers(out)
        self.call(b, weights=weights)
        torch.cuda.synchronize()
        assert (b["y"][n] == 7).all() and (b["idx"][n] == -7).all() and (b["tw"][n] == 7).all()
        assert (b["ws"][self.nb:] == 255).all()
        return b["y"][:n], b["idx"][:n], b["tw"][:n]

    def tolerances(self, r, m, out):
        """(of the weights, of y)"""
        n, d, E, k, f, wdt = self.args
        deep = (lambda K: K / 8 + 64) if wdt == "f32" else (lambda K: K / 32 + 64)
        x = np.abs(self.x.double().cpu().numpy())
        ez = (deep(d) * U * (x @ np.abs(self.wg.double().cpu().numpy()).T)).max(axis=1)
        ez += 2 * U * np.abs(r["z"]).max(axis=1)
        ew = r["w"] * (2 * ez + (E / 64 + 32) * U)[:, None]
        ty = HALF[out] * np.abs(r["y"])
        for t in range(n):
            for j in range(k):
                e = r["idx"][t, j]
                g, u, h = r["g"][t, j], r["u"][t, j], r["h"][t, j]
                eg, eu = (deep(d) * U * (np.abs(m[key][e]) @ x[t]) for key in ("w1", "w3"))
                s = np.abs(g / (1 + np.exp(-g)))
                eh = (1.1 * eg + (16 + 2 * np.abs(g)) * U * s) * np.abs(u) + s * eu + 1.1 * eg * eu
                wh = r["w"][t, j] * np.abs(h)
                eh = r["w"][t, j] * eh + ew[t, j] * np.abs(h) + (HALF[self.act] + 4 * U) * wh
                w2 = np.abs(m["w2"][e])
                ty[t] += w2 @ (eh * (1 + HALF[self.act])) + (deep(f) + 8) * U * (w2 @ wh)
        return ew, ty


CASES = [
    # n, d, E, k, f: one token to sixteen, one expert, all experts, tails of K steps
    (1, 2880, 16, 4, 2880, "mxfp4"), (8, 2880, 16, 4, 2880, "mxfp4"), (3, 64, 4, 2, 96, "mxfp4"),
    (16, 160, 32, 4, 224, "mxfp4"), (5, 32, 1, 1, 32, "mxfp4"), (12, 416, 6, 6, 1056, "mxfp4"),
    (16, 4096, 3, 2, 64, "mxfp4"), (9, 7200, 2, 1, 64, "mxfp4"), (2, 64, 300, 9, 64, "mxfp4"),
    (16, 64, 1024, 32, 32, "mxfp4"), (7, 96, 40, 8, 8192, "mxfp4"),
    (1, 1024, 8, 1, 4096, "bf16"), (16, 1024, 8, 1, 4096, "bf16"), (4, 72, 5, 2, 136, "bf16"),
    (16, 8, 3, 3, 8, "bf16"), (16, 4096, 4, 2, 520, "bf16"), (13, 64, 1024, 32, 40, "bf16"),
    (1, 3, 4, 1, 12, "f32"), (6, 117, 4, 2, 101, "f32"), (16, 512, 9, 3, 260, "f32"), (11, 1, 2, 1, 1, "f32"),
    (2, 64, 1024, 32, 20, "f32"),
]


@pytest.mark.parametrize("n,d,E,k,f,wdt", CASES)
def test_layer(n, d, E, k, f, wdt):
    say(f"[few] {wdt} n {n} d {d} E {E} k {k} f {f}")
    L = Few(n, d, E, k, f, wdt)
    r, m = L.ref()
    # the tokens' choices have to be decided by more than the logits' rounding
    z = -np.sort(-r["z"], axis=1)
    gaps = (z[:, : min(k + 1, E) - 1] - z[:, 1: min(k + 1, E)])
    assert gaps.size == 0 or gaps.min() > 2e-6
    for out in ({"f32", L.act}):
        y, idx, tw = L.run(out)
        assert np.array_equal(idx.cpu().numpy(), r["idx"])
        ew, ty = L.tolerances(r, m, out)
        werr = np.abs(tw.double().cpu().numpy() - r["w"]) / np.maximum(ew, 1e-300)
        yerr = np.abs(y.double().cpu().numpy() - r["y"]) / np.maximum(ty, 1e-300)
        say(f"    {out}: largest error / tolerance: weights {werr.max():.3f}, y {yerr.max():.3f}")
        assert werr.max() <= 1 and yerr.max() <= 1


@pytest.mark.parametrize("wdt", ["mxfp4", "bf16", "f32"])
def test_renorm_rule_slots_and_optional_outputs(wdt):
    torch, B = _torch()
    n, d, E, k, f = 6, 128, 12, 3, 96
    for renorm in (0, 1):
        L = Few(n, d, E, k, f, wdt, renorm=renorm, bias=False)
        r, m = L.ref()
        y, idx, tw = L.run("f32")
        assert np.array_equal(idx.cpu().numpy(), r["idx"])
        ew, ty = L.tolerances(r, m, "f32")
        assert (np.abs(tw.double().cpu().numpy() - r["w"]) <= ew).all()
        assert (np.abs(y.double().cpu().numpy() - r["y"]) <= ty).all()
    # a slot table, with entries outside the slots (clamped)
    slot = np.array([3, 0, 0, 11, 7, -4, 5, 99, 2, 1, 6, 8], np.int32)
    w = dict(L.w, slot=torch.from_numpy(slot).cuda(), n_slots=E)
    r, m = L.ref(slot)
    ys, idx, _ = L.run("f32", weights=w)
    _, ty = L.tolerances(r, m, "f32")
    assert (np.abs(ys.double().cpu().numpy() - r["y"]) <= ty).all()
    # ids and weights are optional
    b = L.buffers("f32")
    B.moe_forward_few(L.shape, L.x, L.act, L.wg, None, L.w, b["y"], "f32", None, None, b["ws"], L.nb)
    torch.cuda.synchronize()
    assert torch.equal(b["y"][:n], y)


@pytest.mark.parametrize("wdt", ["mxfp4", "bf16", "f32"])
def test_nan_tokens_and_nan_experts_stay_apart(wdt):
    torch, B = _torch()
    n, d, E, k, f = 9, 96, 8, 2, 160
    say(f"[few] NaN, {wdt}")
    L = Few(n, d, E, k, f, wdt)
    y0, idx0, tw0 = (t.clone() for t in L.run("f32"))
    # an expert of NaN (and, in the other forms, infinities) spoils its own tokens only
    e = int(idx0[4, 1])
    saved = {key: v.clone() for key, v in L.w.items() if hasattr(v, "clone")}
    if wdt == "mxfp4":
        L.w["s1"][e, :, 0] = 255
        L.w["s2"][e, 5] = 255
    else:
        L.w["w1"][e, 3, :] = float("nan")
        L.w["w2"][e, :, 7] = float("inf")
    y, idx, tw = L.run("f32")
    hit = (idx0 == e).any(dim=1)
    assert hit.any() and not hit.all()
    assert torch.equal(idx, idx0) and torch.equal(tw, tw0)
    assert torch.equal(y[~hit], y0[~hit]) and y[hit].isnan().any(dim=1).all()
    for key, v in saved.items():
        L.w[key].copy_(v)
    # a token of NaN takes experts 0 .. k-1 with NaN weights; the others are as before
    # (it may share their experts, so the sums' cuts may differ: compare within tolerance)
    L.x[2] = float("nan")
    y, idx, tw = L.run("f32")
    assert idx[2].tolist() == list(range(k)) and tw[2].isnan().all() and y[2].isnan().all()
    keep = [t for t in range(n) if t != 2]
    assert torch.equal(idx[keep], idx0[keep]) and torch.equal(tw[keep], tw0[keep])
    L.x[2] = 0.0
    r, m = L.ref()
    _, ty = L.tolerances(r, m, "f32")
    assert (np.abs(y.double().cpu().numpy() - r["y"]) <= ty)[keep].all()


def test_ties_go_to_the_lower_expert():
    torch, B = _torch()
    for wdt, E in (("mxfp4", 40), ("bf16", 200)):
        L = Few(4, 64, E, 5, 64, wdt, bias=False)
        L.wg.copy_(L.wg[:1].expand_as(L.wg).clone())  # all logits alike
        _, idx, tw = L.run()
        assert (idx == torch.arange(5, device="cuda", dtype=torch.int32)).all()
        assert torch.allclose(tw, torch.full_like(tw, 0.2), rtol=1e-6)


def test_same_bits_every_time_in_graphs_and_on_two_streams():
    """Workgroups take their parts in an order that changes from call to call;
    the results do not.  Two layers run at once on two streams, and captured."""
    torch, B = _torch()
    Ls = [Few(1, 512, 16, 4, 512, "mxfp4"), Few(11, 256, 8, 2, 1024, "bf16")]
    bs = [L.buffers() for L in Ls]
    want = [tuple(t.clone() for t in L.run()) for L in Ls]
    streams = [torch.cuda.Stream() for _ in Ls]
    torch.cuda.synchronize()
    for rep in range(20):
        for L, b, st in zip(Ls, bs, streams):
            for _ in range(5):
                L.call(b, stream=st)
    torch.cuda.synchronize()
    for L, b, w in zip(Ls, bs, want):
        assert all(torch.equal(b[key][: L.args[0]], v) for key, v in zip(("y", "idx", "tw"), w))
    graphs = []
    for L, b in zip(Ls, bs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.call(b)
            L.call(b)
        graphs.append(g)
    for rep in range(3):
        for L in Ls:
            L.x.copy_(torch.randn(L.x.shape, generator=torch.Generator().manual_seed(rep)).to(L.dt))
        want = [tuple(t.clone() for t in L.run()) for L in Ls]
        for b in bs:
            b["ws"].fill_(255)
            b["y"].fill_(7)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for L, b, w in zip(Ls, bs, want):
            assert all(torch.equal(b[key][: L.args[0]], v) for key, v in zip(("y", "idx", "tw"), w))


@pytest.mark.parametrize("n,d,E,k,f,wdt", [(1, 2880, 16, 4, 2880, "mxfp4"), (8, 1024, 8, 1, 4096, "bf16"),
                                           (5, 36, 6, 2, 52, "f32")])
def test_against_moe_forward(n, d, E, k, f, wdt):
    """The same choice, and outputs that differ by the hidden's rounding only."""
    torch, B = _torch()
    L = Few(n, d, E, k, f, wdt)
    y, idx, tw = L.run("f32")
    y2, idx2, tw2 = torch.empty_like(y), torch.empty_like(idx), torch.empty_like(tw)
    nb = B.moe_workspace_bytes(L.shape, wdt)
    B.moe_forward(L.shape, L.x, L.act, L.wg, L.bias, L.w, y2, "f32", idx2, tw2,
                  torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    torch.cuda.synchronize()
    assert torch.equal(idx, idx2)
    r, m = L.ref()
    _, ty = L.tolerances(r, m, "f32")
    # both round the hidden once (moe_forward before the weight, and its bf16 pile outputs once more)
    extra = HALF[L.act] * np.abs(r["y"]) if wdt != "f32" else 0.0
    assert (np.abs((y - y2).double().cpu().numpy()) <= 2 * ty + 2 * extra).all()
