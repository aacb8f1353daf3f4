"""What training an MoE layer adds to its forward pass, measured operator by
operator: layer norm with its gradient, the gated feed-forward block over
expert piles that keeps its pre-activations, that block's gradient, and the
router's gradient.

`listed()` gives the fixed cases and `draw()` further ones of the same
ranges; `prepare()` makes a case's inputs, and `run()` makes one pass: the
library's entry points where `own` is true, else the plain form, which is
elementary torch operations in float32, rounded once.  `exact()` is the
operators' definition in float64.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ---- cases --------------------------------------------------------------------


def listed():
    return [
        # one token's norm in front of a decode step: latency
        dict(name="norm-token", op="norm", n=1, d=4096, dtype="bf16"),
        # the norm in front of the Mixtral-shaped layer
        dict(name="norm-batch", op="norm", n=8192, d=4096, dtype="bf16"),
        # its gradient: rows, and the weight's and bias's sums over the batch
        dict(name="norm-grad-batch", op="norm_grad", n=8192, d=4096, dtype="bf16"),
        # an odd width and an odd number of rows in float32
        dict(name="norm-grad-odd-f32", op="norm_grad", n=4099, d=1021, dtype="f32"),
        # a few tokens of the Switch layer: bound by reading the weights
        dict(name="up-few", op="up", n=16, d=1024, E=8, k=1, d_ff=4096, dtype="bf16", zipf=0.0),
        # the Switch layer's training batch
        dict(name="up-switch", op="up", n=4096, d=1024, E=8, k=1, d_ff=4096, dtype="bf16", zipf=0.0),
        # gradients of the Switch layer and of the Mixtral-shaped layer
        dict(name="ffn-grad-switch", op="ffn_grad", n=4096, d=1024, E=8, k=1, d_ff=4096, dtype="bf16",
             zipf=0.0),
        dict(name="ffn-grad-mixtral", op="ffn_grad", n=8192, d=4096, E=8, k=2, d_ff=14336, dtype="bf16",
             zipf=0.0),
        # 128 experts under a skewed load: piles from a few rows to thousands
        dict(name="ffn-grad-zipf", op="ffn_grad", n=4096, d=2880, E=128, k=4, d_ff=2880, dtype="bf16",
             zipf=1.1),
        # a small float32 layer with odd sizes
        dict(name="ffn-grad-odd-f32", op="ffn_grad", n=333, d=501, E=5, k=2, d_ff=709, dtype="f32",
             zipf=0.5),
        # the router's gradient at 8 and at 128 experts
        dict(name="router-grad-e8", op="router_grad", n=8192, d=4096, E=8, k=2, dtype="bf16", zipf=0.0),
        dict(name="router-grad-e128", op="router_grad", n=4096, d=2880, E=128, k=4, dtype="bf16",
             zipf=1.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "up", "ffn_grad", "router_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    step = 8 if dtype == "bf16" else 1  # bf16 rows are multiples of 8 wide
    if op in ("norm", "norm_grad"):
        d = max(step, _log_int(rng, 16, 16384) // step * step)
        return dict(op=op, n=_log_int(rng, 1, min(65536, (1 << 25) // d)), d=d, dtype=dtype)
    E = _log_int(rng, 1, 128)
    k = rng.randint(1, min(E, 8))
    zipf = rng.choice([0.0, 0.7, 1.1])
    if op == "router_grad":
        d = _log_int(rng, 64, 4096) // step * step
        return dict(op=op, n=_log_int(rng, 1, 8192), d=d, E=E, k=k, dtype=dtype, zipf=zipf)
    d = _log_int(rng, 64, 4096) // step * step
    d_ff = _log_int(rng, 64, 4096) // step * step
    # at most 2^30 weights, 2^37 products of a row and a weight (2^33 in float32)
    while E * d * d_ff * 3 > 1 << 30:
        E = max(1, E // 2)
    k = min(k, E)
    most = (1 << (37 if dtype == "bf16" else 33)) // (d * d_ff * k)
    n = _log_int(rng, 1, max(1, min(8192, most)))
    return dict(op=op, n=n, d=d, E=E, k=k, d_ff=d_ff, dtype=dtype, zipf=zipf)


# ---- inputs -------------------------------------------------------------------


def _skew(case):
    """log-popularity of the experts: rank r is chosen like r^-zipf."""
    return [-case["zipf"] * math.log(r + 1.0) for r in range(case["E"])]


def _routing(case, normal, dev):
    """Router logits of a skewed batch, the chosen experts and their weights."""
    E, k = case["E"], case["k"]
    z = normal(case["n"], E) + torch.tensor(_skew(case), device=dev)
    p = torch.softmax(z, 1)
    w, idx = torch.topk(p, k, dim=1)
    if k > 1:
        w = w / w.sum(1, keepdim=True)
    return z, idx.to(torch.int32), w.contiguous()


def _piles(case, idx):
    """The piles of a dispatch: token of each pile row, pile row of each
    (token, slot), and the pile boundaries."""
    E, k = case["E"], case["k"]
    flat = idx.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=order.device)
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    return (order // k).to(torch.int32), inv.view(-1, k).to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(scale)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device=dev)

    n, d = case["n"], case["d"]
    f32 = torch.float32
    st = dict(case=dict(case))
    if case["op"] in ("norm", "norm_grad"):
        # a residual stream: a few channels stand out, and rows have a mean
        x = normal(n, d) + 2.0 * normal(n, 1)
        x = (x * (1.0 + 9.0 * (torch.rand(d, generator=gen, device=dev) < 0.02))).to(dt)
        st.update(x=x, weight=1.0 + normal(d, scale=0.2), bias=normal(d, scale=0.2))
        if case["op"] == "norm":
            st.update(y=empty(n, d), mean=empty(n, dtype=f32), rstd=empty(n, dtype=f32))
        else:  # the statistics that the forward pass kept
            xf = x.double()
            mean = xf.mean(1)
            rstd = (xf.var(1, unbiased=False) + EPS).rsqrt()
            st.update(dy=normal(n, d).to(dt), mean=mean.float(), rstd=rstd.float(),
                      dx=empty(n, d), dweight=empty(d, dtype=f32), dbias=empty(d, dtype=f32))
        return st

    E, k = case["E"], case["k"]
    R = n * k
    z, idx, w = _routing(case, normal, dev)
    perm, inv, offsets = _piles(case, idx)
    x = normal(n, d).to(dt)
    st.update(x=x, idx=idx, topk_w=w, perm=perm, inv=inv, offsets=offsets)
    if case["op"] == "router_grad":
        st.update(logits=z, wg=normal(E, d, scale=d ** -0.5).to(dt), dtopk_w=normal(n, k),
                  f=torch.bincount(idx[:, 0].long(), minlength=E).float() / n, alpha=0.01,
                  dx_perm=normal(R, d).to(dt), dlogits=empty(n, E, dtype=f32), dx=empty(n, d),
                  dwg=empty(E, d), dbias=empty(E, dtype=f32))
        return st

    f = case["d_ff"]
    w1, w3, w2 = empty(E, f, d), empty(E, f, d), empty(E, d, f)
    for m, fan in ((w1, d), (w3, d), (w2, f)):
        for e in range(E):
            m[e] = normal(*m.shape[1:], scale=fan ** -0.5)
    st.update(w1=w1, w3=w3, w2=w2, bounds=offsets.tolist())
    if case["op"] == "up":
        st.update(h=empty(R, f), g=empty(R, f), u=empty(R, f))
        return st
    # the pre-activations that the forward pass kept
    g, u = empty(R, f), empty(R, f)
    for e, lo, hi in _spans(st["bounds"]):
        xe = x[perm[lo:hi].long()]
        g[lo:hi], u[lo:hi] = xe @ w1[e].t(), xe @ w3[e].t()
    st.update(dy=normal(n, d).to(dt), g=g, u=u, dx_perm=empty(R, d), dw1=empty(E, f, d),
              dw3=empty(E, f, d), dw2=empty(E, d, f), dtopk_w=empty(n, k, dtype=f32))
    return st


def _spans(bounds):
    """(expert, first row, last row + 1) of the piles that hold rows."""
    return [(e, lo, hi) for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])) if hi > lo]


# ---- one pass -------------------------------------------------------------------


def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _shape(case):
    return (case["n"], case["d"], case["E"], case["k"], case.get("d_ff", case["d"]), -1)


def _workspace(st, nbytes):
    """The workspace that a program keeps beside its buffers."""
    if "ws" not in st:
        st["ws"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    return st["ws"]


def _weights(st):
    return dict(dtype=st["case"]["dtype"], w1=st["w1"], w3=st["w3"], w2=st["w2"])


def _own_norm(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    B.moe_layer_norm(c["n"], c["d"], st["x"], c["dtype"], st["weight"], st["bias"], EPS, st["y"],
                     st["mean"], st["rstd"])
    return {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}


def _own_norm_grad(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    nb = B.moe_layer_norm_backward_workspace_bytes(c["n"], c["d"])
    B.moe_layer_norm_backward(c["n"], c["d"], st["dy"], st["x"], c["dtype"], st["weight"], st["mean"],
                              st["rstd"], st["dx"], st["dweight"], st["dbias"], _workspace(st, nb), nb)
    return {"dx": st["dx"], "dweight": st["dweight"], "dbias": st["dbias"]}


def _own_up(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    B.moe_expert_up_save(_shape(c), st["x"], c["dtype"], st["perm"], st["offsets"], _weights(st), st["h"],
                         st["g"], st["u"])
    return {"h": st["h"], "g": st["g"], "u": st["u"]}


def _own_ffn_grad(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    nb = B.moe_grouped_ffn_backward_workspace_bytes(_shape(c), c["dtype"])
    B.moe_grouped_ffn_backward(_shape(c), st["dy"], st["x"], c["dtype"], st["perm"], st["inv"],
                               st["topk_w"], st["offsets"], _weights(st), st["g"], st["u"], st["dx_perm"],
                               st["dw1"], st["dw3"], st["dw2"], st["dtopk_w"], _workspace(st, nb), nb)
    return {key: st[key] for key in ("dx_perm", "dw1", "dw3", "dw2", "dtopk_w")}


def _own_router_grad(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    nb = B.moe_router_backward_workspace_bytes(_shape(c))
    B.moe_router_backward(_shape(c), st["logits"], st["idx"], st["topk_w"], st["dtopk_w"], st["f"],
                          st["alpha"], st["x"], c["dtype"], st["wg"], st["dx_perm"], st["inv"],
                          st["dlogits"], st["dx"], st["dwg"], st["dbias"], _workspace(st, nb), nb)
    return {key: st[key] for key in ("dlogits", "dx", "dwg", "dbias")}


_own = dict(norm=_own_norm, norm_grad=_own_norm_grad, up=_own_up, ffn_grad=_own_ffn_grad,
            router_grad=_own_router_grad)


# The plain form.  Piles have different lengths, so the experts' products are
# one product per expert.


def _plain_norm(st):
    x = st["x"].float()
    mean = x.sum(1, keepdim=True) / x.shape[1]
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).sum(1, keepdim=True) / x.shape[1] + EPS)
    y = c * rstd * st["weight"] + st["bias"]
    return {"y": y.to(st["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_grad(st):
    x, dy = st["x"].float(), st["dy"].float()
    rstd = st["rstd"][:, None]
    xh = (x - st["mean"][:, None]) * rstd
    t = dy * st["weight"]
    m1 = t.sum(1, keepdim=True) / x.shape[1]
    m2 = (t * xh).sum(1, keepdim=True) / x.shape[1]
    dx = rstd * (t - m1 - xh * m2)
    return {"dx": dx.to(st["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _plain_up(st):
    dt = st["x"].dtype
    out = {key: torch.empty_like(st[key]) for key in ("h", "g", "u")}
    for e, lo, hi in _spans(st["bounds"]):
        xe = st["x"][st["perm"][lo:hi].long()].float()
        g, u = xe @ st["w1"][e].float().t(), xe @ st["w3"][e].float().t()
        out["g"][lo:hi], out["u"][lo:hi] = g.to(dt), u.to(dt)
        out["h"][lo:hi] = (g / (1.0 + torch.exp(-g)) * u).to(dt)
    return out


def _plain_ffn_grad(st):
    dt = st["x"].dtype
    out = {key: torch.empty_like(st[key]) for key in ("dx_perm", "dw1", "dw3", "dw2")}
    inv = st["inv"].reshape(-1).long()
    roww = torch.empty_like(st["topk_w"].reshape(-1))
    roww[inv] = st["topk_w"].reshape(-1)
    drow = torch.empty_like(roww)
    for e, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        tok = st["perm"][lo:hi].long()
        x, dy, wr = st["x"][tok].float(), st["dy"][tok].float(), roww[lo:hi, None]
        g, u = st["g"][lo:hi].float(), st["u"][lo:hi].float()
        s = 1.0 / (1.0 + torch.exp(-g))
        h = g * s * u
        dh = dy @ st["w2"][e].float()
        drow[lo:hi] = (dh * h).sum(1)
        dh = dh * wr
        dg, du = dh * u * (s * (1.0 + g * (1.0 - s))), dh * (g * s)
        out["dx_perm"][lo:hi] = (dg @ st["w1"][e].float() + du @ st["w3"][e].float()).to(dt)
        out["dw1"][e], out["dw3"][e] = (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
        out["dw2"][e] = (dy.t() @ (h * wr)).to(dt)
    out["dtopk_w"] = drow[inv].view_as(st["topk_w"])
    return out


def _plain_router_grad(st):
    c, dt = st["case"], st["x"].dtype
    z, idx, w, dw, f = st["logits"], st["idx"].long(), st["topk_w"], st["dtopk_w"], st["f"]
    q = torch.exp(z - z.amax(1, keepdim=True))
    p = q / q.sum(1, keepdim=True)
    D = (w * dw).sum(1, keepdim=True)
    if c["k"] > 1:  # weights renormalised over the chosen experts
        dz = torch.zeros_like(z).scatter_add(1, idx, w * (dw - D))
    else:
        dz = p * (torch.zeros_like(z).scatter_add(1, idx, dw) - D)
    dz = dz + (st["alpha"] * c["E"] / c["n"]) * p * (f - (p * f).sum(1, keepdim=True))
    dx = dz @ st["wg"].float() + st["dx_perm"][st["inv"].long()].float().sum(1)
    return {"dlogits": dz, "dx": dx.to(dt), "dwg": (dz.t() @ st["x"].float()).to(dt), "dbias": dz.sum(0)}


_plain = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, up=_plain_up, ffn_grad=_plain_ffn_grad,
              router_grad=_plain_router_grad)


# ---- what a pass cannot do without ----------------------------------------------


def work(case):
    n, d, s = case["n"], case["d"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        return {"bytes": 2 * n * d * s + 8 * d + 8 * n, "flops": 8 * n * d}
    if case["op"] == "norm_grad":
        return {"bytes": 3 * n * d * s + 12 * d + 8 * n, "flops": 14 * n * d}
    E, R = case["E"], case["n"] * case["k"]
    if case["op"] == "router_grad":
        return {"bytes": 8 * n * E + (2 * n + R + 2 * E) * d * s + 16 * R, "flops": 4 * n * E * d}
    f = case["d_ff"]
    share = [math.exp(v) for v in _skew(case)]
    active = sum(1.0 - (1.0 - v / sum(share)) ** R for v in share)  # experts with rows, expected
    if case["op"] == "up":
        return {"bytes": (n * d + 2 * active * d * f + 3 * R * f) * s + 4 * R, "flops": 4 * R * d * f}
    moved = 2 * n * d + R * d + 2 * R * f + 3 * active * d * f + 3 * E * d * f
    return {"bytes": moved * s + 16 * R, "flops": 12 * R * d * f}


# ---- the definitions in float64 -------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    v = {key: t.double() if t.is_floating_point() and key not in ("w1", "w3", "w2", "g", "u") else t
         for key, t in st.items() if isinstance(t, torch.Tensor)}
    if case["op"] == "norm":
        mean = v["x"].mean(1)
        rstd = (v["x"].var(1, unbiased=False) + EPS).pow(-0.5)
        xh = (v["x"] - mean[:, None]) * rstd[:, None]
        return {"y": torch.addcmul(v["bias"], xh, v["weight"]), "mean": mean, "rstd": rstd}
    if case["op"] == "norm_grad":
        # the gradient of a row: W dy without its parts along 1 and xh
        xh = (v["x"] - v["mean"][:, None]) * v["rstd"][:, None]
        t = v["dy"] * v["weight"]
        dx = t - t.mean(1, keepdim=True) - xh * (xh * t).mean(1, keepdim=True)
        return {"dx": dx * v["rstd"][:, None], "dweight": torch.einsum("nd,nd->d", v["dy"], xh),
                "dbias": v["dy"].sum(0)}
    if case["op"] == "router_grad":
        p = torch.softmax(v["logits"], 1)
        idx, w, dw = v["idx"].long(), v["topk_w"], v["dtopk_w"]
        dp = torch.zeros_like(p)
        if case["k"] > 1:  # d w_j / d z = w_j (delta - w), over the chosen experts
            dz = torch.zeros_like(p).scatter_add(1, idx, w * dw)
            dz = dz - torch.zeros_like(p).scatter_add(1, idx, w) * (w * dw).sum(1, keepdim=True)
        else:
            dz = torch.zeros_like(p).scatter_add(1, idx, w * dw) - p * (w * dw)
        dp = dp + st["alpha"] * case["E"] / case["n"] * v["f"]
        dz = dz + p * dp - p * (p * dp).sum(1, keepdim=True)
        dx = torch.mm(dz, v["wg"])
        for j in range(case["k"]):
            dx = dx + v["dx_perm"][v["inv"][:, j].long()]
        return {"dlogits": dz, "dx": dx, "dwg": torch.mm(dz.t(), v["x"]), "dbias": dz.sum(0)}
    R, b = case["n"] * case["k"], st["bounds"]
    if case["op"] == "up":
        out = {key: torch.empty(R, case["d_ff"], dtype=torch.float64, device="cuda") for key in "hgu"}
        for e in range(case["E"]):
            r = slice(b[e], b[e + 1])
            xe = v["x"].index_select(0, v["perm"][r].long())
            out["g"][r] = torch.mm(xe, v["w1"][e].double().t())
            out["u"][r] = torch.mm(xe, v["w3"][e].double().t())
        out["h"] = out["g"] * torch.sigmoid(out["g"]) * out["u"]
        return out
    out = {"dx_perm": torch.empty(R, case["d"], dtype=torch.float64, device="cuda")}
    for key in ("dw1", "dw3", "dw2"):
        out[key] = torch.zeros(st[key].shape, dtype=torch.float64, device="cuda")
    wr = torch.zeros(R, dtype=torch.float64, device="cuda")
    wr.scatter_(0, v["inv"].reshape(-1).long(), v["topk_w"].reshape(-1))
    drow = torch.zeros_like(wr)
    for e in range(case["E"]):
        r = slice(b[e], b[e + 1])
        tok = v["perm"][r].long()
        x, dyw = v["x"].index_select(0, tok), v["dy"].index_select(0, tok)
        g, u = v["g"][r].double(), v["u"][r].double()
        sg = torch.sigmoid(g)
        a = g * sg
        dh = torch.mm(dyw, v["w2"][e].double())
        drow[r] = (dh * a * u).sum(1)
        dh = dh * wr[r, None]
        dg, du = dh * u * (sg + a * (1.0 - sg)), dh * a
        out["dx_perm"][r] = torch.mm(dg, v["w1"][e].double()) + torch.mm(du, v["w3"][e].double())
        out["dw1"][e], out["dw3"][e] = torch.mm(dg.t(), x), torch.mm(du.t(), x)
        out["dw2"][e] = torch.mm((dyw * wr[r, None]).t(), a * u)
    out["dtopk_w"] = drow.index_select(0, v["inv"].reshape(-1).long()).view(case["n"], case["k"])
    return out
