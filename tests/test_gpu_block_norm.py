"""GPU parity of moe_block_norm and its gradient with the float64 oracle.

Tolerances (derived, not measured).  Outputs are rounded once (half a step:
2^-8 bf16, 2^-24 float32).  Before that all arithmetic is float32: a row's sum
adds at most 32 elements per thread, then 6 lane steps and 16 wave sums, under
64 additions deep, each off by at most 2^-24 of the magnitudes summed; 96 * 2^-24
covers those with the products, square root and division around them.  u is
taken from h before its rounding, so h's float32 error alone goes through the
second norm: directly, through the mean, and through the variance.  A column
sum over n rows is at most n / 256 + 96 additions deep."""

import numpy as np
import pytest

from oracle import serve_oracle as S
from tests.gpu_support import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
A = 96 * U
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SIZES = {
    "bf16": [(1, 8), (3, 16), (7, 136), (65, 512), (33, 520), (2, 2048), (1, 2880), (300, 4096), (5, 4104),
             (9, 8192), (3, 8200), (2, 16384), (3000, 64), (1300, 1024)],
    "f32": [(1, 1), (2, 3), (5, 17), (6, 64), (7, 65), (9, 255), (4, 257), (33, 1021), (5, 1024), (3, 2047),
            (9, 2049), (3, 4097), (2, 8193), (2, 16383), (1, 16384), (3000, 33), (1300, 500)],
}
FORMS = [("layer", "layer", True), ("rms", "layer", False), ("layer", "rms", True), (None, "rms", True),
         ("rms", None, True), (None, "layer", False), (None, None, True), (None, None, False)]


def _tensor(a, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)


def _f64(t):
    return t.double().cpu().numpy()


def _norm64(v):
    return None if v is None else dict(kind=v["kind"], weight=_f64(v["weight"]),
                                       bias=None if v["bias"] is None else _f64(v["bias"]), eps=v["eps"])


class Case:
    scale = 1.25

    def __init__(self, dtype, n, d, form, seed=0, bias=True):
        rng = np.random.default_rng(1000 * n + d + seed)
        self.dtype, self.n, self.d = dtype, n, d
        self.x = _tensor(rng.standard_normal((n, d)) + 2.0 * rng.standard_normal((n, 1)), dtype)
        self.z = _tensor(rng.standard_normal((n, d)), dtype)
        self.dh, self.du = (_tensor(rng.standard_normal((n, d)), dtype) for _ in range(2))
        vec = lambda c: _tensor(c + 0.3 * rng.standard_normal(d), "f32")
        norm = lambda kind: None if kind is None else dict(
            kind=kind, weight=vec(1.0), bias=vec(0.0) if bias and kind == "layer" else None, eps=1e-5)
        self.post, self.pre = norm(form[0]), norm(form[1])
        self.gate = vec(0.5) if form[2] else None

    def forward(self, stats=True, stream=None, h=None, u=None):
        import torch
        from mixture_experts_layer_wave_amd import binding as B

        n, d = self.n, self.d
        full = lambda *s: torch.full(s, 7.0, dtype=self.x.dtype, device="cuda")
        hh, uu = (full(n + 1, d) if h is None else h), (full(n + 1, d) if u is None else u)
        st = torch.full((4 * n + 4,), 7.0, device="cuda")
        B.moe_block_norm(n, d, self.x, self.z, self.dtype, self.scale, self.gate, self.post, self.pre, hh,
                         uu if self.pre else None, st if stats else None, stream)
        torch.cuda.synchronize()
        assert (st[4 * n:] == 7).all()
        if h is None:
            assert (hh[n] == 7).all()
        if u is None:
            assert (uu[n] == 7).all() and (self.pre is not None or (uu == 7).all())
        return hh[:n], uu[:n], st[: 4 * n].view(4, n)

    def backward(self, h, stats, dh="own", dx=None, dz=None, want=True):
        import torch
        from mixture_experts_layer_wave_amd import binding as B

        n, d = self.n, self.d
        full = lambda: torch.full((n + 1, d), 7.0, dtype=self.x.dtype, device="cuda")
        dxx, dzz = (full() if dx is None else dx), (full() if dz is None else dz)
        par = {key: torch.full((d + 1,), 7.0, device="cuda") for key in
               ("dgate", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias")}
        give = dict(dgate=self.gate is not None, dpost_weight=self.post, dpost_bias=self.post, dpre_weight=self.pre,
                    dpre_bias=self.pre)
        nb = B.moe_block_norm_backward_workspace_bytes(n, d)
        ws = torch.full((nb + 256,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns, and a guard
        B.moe_block_norm_backward(n, d, self.dh if isinstance(dh, str) else dh, self.du if self.pre else None, self.z, h, self.dtype,
                                  self.scale, self.gate, self.post, self.pre, stats, dxx, dzz,
                                  *(par[key] if give[key] and want else None for key in par), ws, nb)
        torch.cuda.synchronize()
        assert (ws[nb:] == 255).all()
        if dx is None:
            assert (dxx[n] == 7).all()
        if dz is None:
            assert (dzz[n] == 7).all()
        out = dict(dx=dxx[:n], dz=dzz[:n])
        for key, v in par.items():
            assert v[d] == 7
            if give[key] and want:
                out[key] = v[:d]
            else:
                assert (v == 7).all()
        return out


def _check(name, got, ref, tol):
    assert np.isfinite(got).all(), name
    worst = float(np.max((np.abs(got - ref) / np.maximum(tol, 1e-300)), initial=0.0))
    say(f"    {name}: largest error / tolerance {worst:.3f}")
    assert worst <= 1.0, name


def _norm_tol(v, ev, norm, mean, rstd):
    """float32 error of norm(v) whose rows are off by ev already: (mean, rstd, y)"""
    w, b = np.abs(norm["weight"]), 0.0 if norm["bias"] is None else np.abs(norm["bias"])
    size = np.abs(v).mean(axis=1)
    c = np.abs(v - mean[:, None])
    em = A * size + ev.mean(axis=1)
    var = 1.0 / rstd ** 2
    # of the variance: twice the mean of c times its error (c's own rounding included)
    evar = 2 * (c * (ev + U * (np.abs(v) + np.abs(mean[:, None])))).mean(axis=1) + (em + ev.max(axis=1)) ** 2
    er = rstd * (A + evar / var)
    ey = rstd[:, None] * w * (ev + em[:, None] + A * (c + U * 0) + U * np.abs(v)) + c * er[:, None] * w + A * b
    return em, er, ey


@pytest.mark.parametrize("dtype,n,d", [(t, n, d) for t in SIZES for n, d in SIZES[t]])
def test_forward(dtype, n, d):
    for form in FORMS if n * d < 20000 else FORMS[:4]:
        say(f"[block norm] {dtype} {n} x {d} {form}")
        c = Case(dtype, n, d, form)
        h, u, st = c.forward()
        x, z, gate = _f64(c.x), _f64(c.z), None if c.gate is None else _f64(c.gate)
        post, pre = _norm64(c.post), _norm64(c.pre)
        r = S.block_norm(x, z, c.scale, gate, post, pre)
        ev, v = np.zeros((n, d)), z
        if post:
            v, m, rs = S.row_norm(z, post)
            em, er, ev = _norm_tol(z, ev, post, m, rs)
            _check("post mean", _f64(st[0]), r["stats"][0], em)
            _check("post rstd", _f64(st[1]), r["stats"][1], er)
        g = 1.0 if gate is None else np.abs(gate)
        eh = g * ev + 4 * U * (np.abs(c.scale * x) + g * np.abs(v) + (g * np.abs(post["bias"]) if post and post["bias"] is not None else 0))
        _check("h", _f64(h), r["h"], eh + HALF[dtype] * np.abs(r["h"]))
        if pre:
            em, er, eu = _norm_tol(r["h"], eh, pre, r["stats"][2], r["stats"][3])
            _check("pre mean", _f64(st[2]), r["stats"][2], em)
            _check("pre rstd", _f64(st[3]), r["stats"][3], er)
            _check("u", _f64(u), r["u"], eu + HALF[dtype] * np.abs(r["u"]))
        for present, rows in ((post, st[:2]), (pre, st[2:])):
            assert present or (rows == 7).all()


def _norm_grad_tol(t, xh, rstd, et, layer):
    """float32 error of a norm's dv for t = w dy off by et."""
    avg = lambda a: a.mean(axis=1, keepdims=True)
    at, ax = np.abs(t), np.abs(xh)
    e = et + A * at + ax * (avg(et * ax) + A * avg(at * ax)) + 4 * U * ax * avg(at * ax)
    if layer:
        e = e + avg(et) + A * avg(at)
    return rstd[:, None] * e


@pytest.mark.parametrize("dtype,n,d", [(t, n, d) for t in SIZES for n, d in SIZES[t]])
def test_backward(dtype, n, d):
    for form in FORMS if n * d < 20000 else FORMS[:4]:
        say(f"[block norm grad] {dtype} {n} x {d} {form}")
        c = Case(dtype, n, d, form)
        h, _, st = c.forward()
        for dh in ([c.dh, None] if c.pre else [c.dh]):
            got = c.backward(h, st, dh=dh)
            z, h64, s64 = _f64(c.z), _f64(h), _f64(st)
            gate, post, pre = None if c.gate is None else _f64(c.gate), _norm64(c.post), _norm64(c.pre)
            dh64 = None if dh is None else _f64(dh)
            du = _f64(c.du)
            r = S.block_norm_grad(dh64, du, z, h64, c.scale, gate, post, pre, s64)
            deep = (n / 256 + 96) * U
            eD = np.zeros((n, d))
            if pre:
                hh = (h64 - s64[2][:, None]) * s64[3][:, None]
                # xh itself: a subtraction, a product
                exh = 2 * U * np.abs(hh)
                t = du * pre["weight"]
                eD = _norm_grad_tol(t, hh, s64[3], 2 * U * np.abs(t), pre["kind"] == "layer")
                eD += U * np.abs(r["D"])
                _check("dpre_weight", _f64(got["dpre_weight"]), r["dpre_weight"],
                       (np.abs(du) * exh).sum(0) + deep * np.abs(du * hh).sum(0))
                _check("dpre_bias", _f64(got["dpre_bias"]), r["dpre_bias"], deep * np.abs(du).sum(0))
            _check("dx", _f64(got["dx"]), r["dx"], np.abs(c.scale) * eD + (HALF[dtype] + 2 * U) * np.abs(r["dx"]))
            g = np.ones(d) if gate is None else gate
            aD = np.abs(r["D"])
            if post:
                zh = (z - s64[0][:, None]) * s64[1][:, None]
                t = r["D"] * g * post["weight"]
                et = eD * np.abs(g * post["weight"]) + 4 * U * np.abs(t)
                edz = _norm_grad_tol(t, zh, s64[1], et, post["kind"] == "layer")
                e3 = (eD * np.abs(zh)).sum(0) + (deep + 4 * U) * (aD * np.abs(zh)).sum(0)
                e4 = eD.sum(0) + deep * aD.sum(0)
                _check("dpost_weight", _f64(got["dpost_weight"]), r["dpost_weight"], np.abs(g) * e3 * (1 + 4 * U) + 4 * U * np.abs(r["dpost_weight"]))
                _check("dpost_bias", _f64(got["dpost_bias"]), r["dpost_bias"], np.abs(g) * e4 + 4 * U * np.abs(r["dpost_bias"]))
                b = 0.0 if post["bias"] is None else np.abs(post["bias"])
                eg = np.abs(post["weight"]) * (e3 + 4 * U * (aD * np.abs(zh)).sum(0)) + b * (e4 + 4 * U * aD.sum(0))
            else:
                edz = eD * np.abs(g)
                eg = (eD * np.abs(z)).sum(0) + (deep + 4 * U) * (aD * np.abs(z)).sum(0)
            _check("dz", _f64(got["dz"]), r["dz"], edz + (HALF[dtype] + 4 * U) * np.abs(r["dz"]))
            if gate is not None:
                _check("dgate", _f64(got["dgate"]), r["dgate"], eg)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_and_optional(dtype):
    import torch

    c = Case(dtype, 700, 264, ("layer", "rms", True))
    h, u, st = (t.clone() for t in c.forward())
    g = c.backward(h, st)
    # without statistics, and without the parameters' gradients
    h2, u2, _ = c.forward(stats=False)
    assert torch.equal(h, h2) and torch.equal(u, u2)
    g2 = c.backward(h, st, want=False)
    assert torch.equal(g["dx"], g2["dx"]) and torch.equal(g["dz"], g2["dz"])
    # gradients over the gradients they come from
    dh, du = c.dh.clone(), c.du.clone()
    c.backward(h, st, dx=c.dh, dz=c.du)
    assert torch.equal(c.dh, g["dx"]) and torch.equal(c.du, g["dz"])
    c.dh, c.du = dh, du
    # h over x, u over z
    c.forward(h=c.x, u=c.z)
    assert torch.equal(c.x, h) and torch.equal(c.z, u)


def test_nothing_to_do():
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    w = torch.ones(64, device="cuda")
    norm = dict(kind="layer", weight=w, bias=None)
    par = [torch.full((64,), 7.0, device="cuda") for _ in range(5)]
    B.moe_block_norm(0, 64, None, None, "bf16", 1.0, None, norm, norm, None)
    B.moe_block_norm_backward(0, 64, None, None, None, None, "bf16", 1.0, w, norm, norm, None, None, None, *par,
                              None, 0)
    torch.cuda.synchronize()
    assert all((v == 0).all() for v in par)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_rows_stay_alone(dtype):
    """A row of NaN or infinities touches no other row; a row of one value has
    norms of bias, not of noise."""
    import torch

    c = Case(dtype, 40, 136, ("layer", "layer", True))
    h, u, st = (t.clone() for t in c.forward())
    g = c.backward(h, st)
    c.z[3], c.x[17, 5] = float("nan"), float("inf")
    h2, u2, st2 = c.forward()
    keep = [t for t in range(40) if t not in (3, 17)]
    assert torch.equal(h2[keep], h[keep]) and torch.equal(u2[keep], u[keep])
    assert h2[3].isnan().all() and u2[17].isnan().all()
    g2 = c.backward(h2, st2)
    assert torch.equal(g2["dx"][keep], g["dx"][keep]) and torch.equal(g2["dz"][keep], g["dz"][keep])
    c = Case(dtype, 5, 520, ("layer", None, False))
    c.z[:] = torch.tensor([0.0, 3.0, -1e5, 0.1, 7e3], device="cuda")[:, None].to(c.z.dtype)
    c.x.zero_()
    h, _, st = c.forward()
    assert torch.equal(h, c.post["bias"].to(h.dtype).expand_as(h))


def test_rows_past_32_bit_offsets():
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    n, d = (1 << 31) // 16384 + 5, 16384
    say(f"[block norm far] {n} x {d}")
    small = Case("bf16", 4, d, ("rms", "layer", True))
    hs, us, sts = small.forward()
    gs = small.backward(hs, sts)
    big = {key: torch.zeros((n, d), dtype=torch.bfloat16, device="cuda") for key in ("x", "z", "dh", "du")}
    for key, v in big.items():
        v[-4:] = getattr(small, key)
    h, u = torch.zeros_like(big["x"]), torch.zeros_like(big["x"])
    st = torch.zeros((4, n), device="cuda")
    B.moe_block_norm(n, d, big["x"], big["z"], "bf16", small.scale, small.gate, small.post, small.pre, h, u, st)
    assert torch.equal(h[-4:], hs) and torch.equal(u[-4:], us) and torch.equal(st[:, -4:], sts)
    nb = B.moe_block_norm_backward_workspace_bytes(n, d)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    dx, dz = big["x"], u
    B.moe_block_norm_backward(n, d, big["dh"], big["du"], big["z"], h, "bf16", small.scale, small.gate, small.post,
                              small.pre, st, dx, dz, None, None, None, None, None, ws, nb)
    assert torch.equal(dx[-4:], gs["dx"]) and torch.equal(dz[-4:], gs["dz"])


def test_differences():
    """The gradient against differences of the library's own forward pass."""
    import torch

    c = Case("f32", 6, 41, ("layer", "rms", True))
    h, u, st = c.forward()
    got = c.backward(h, st)
    loss = lambda: (lambda o: float((o[0].double() * c.dh.double()).sum() + (o[1].double() * c.du.double()).sum()))(
        c.forward())
    rng = np.random.default_rng(0)
    leaves = dict(dx=c.x, dz=c.z, dgate=c.gate, dpost_weight=c.post["weight"], dpost_bias=c.post["bias"],
                  dpre_weight=c.pre["weight"])
    for key, leaf in leaves.items():
        v = torch.from_numpy(rng.standard_normal(tuple(leaf.shape)).astype(np.float32)).cuda()
        keep, eps = leaf.clone(), 2.0 ** -7
        leaf.copy_(keep + eps * v)
        hi = loss()
        leaf.copy_(keep - eps * v)
        lo = loss()
        leaf.copy_(keep)
        want = float((got[key].double() * v.double()).sum())
        # differences of float32 outputs: rounding 2^-24 of about 500 terms over eps, and eps^2
        assert abs((hi - lo) / (2 * eps) - want) < 2e-3 * max(1.0, abs(want)) + 2e-2, key


def test_graph_and_streams():
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    c = Case("bf16", 600, 1024, ("layer", "layer", True))
    n, d = c.n, c.d
    h, u, dx, dz = (torch.zeros_like(c.x) for _ in range(4))
    st = torch.zeros((4, n), device="cuda")
    par = [torch.zeros(d, device="cuda") for _ in range(5)]
    nb = B.moe_block_norm_backward_workspace_bytes(n, d)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")

    def step():
        B.moe_block_norm(n, d, c.x, c.z, "bf16", c.scale, c.gate, c.post, c.pre, h, u, st)
        B.moe_block_norm_backward(n, d, c.dh, c.du, c.z, h, "bf16", c.scale, c.gate, c.post, c.pre, st, dx, dz,
                                  *par, ws, nb)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    side = torch.cuda.Stream()
    for rep in range(3):
        c.z.copy_(torch.randn((n, d), generator=torch.Generator().manual_seed(rep)).to(c.z.dtype))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (h, u, st, dx, dz, *par)]
        for t in (h, u, st, dx, dz, *par):
            t.fill_(3.0)
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((h, u, st, dx, dz, *par), want))
