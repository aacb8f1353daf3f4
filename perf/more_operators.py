"""What serving an MXFP4 mixture-of-experts block adds to the layer, measured
operator by operator: the MXFP4 encoder and decoder, the product with an
MXFP4 matrix (bf16 or MXFP4 rows), the whole layer for a few tokens, and the
norms before and after a block with its gate and residual scale, with their
gradient.

`listed()` gives the fixed cases and `draw()` further ones of the same
ranges; `prepare()` makes a case's inputs, and `run()` makes one pass: the
library's entry points where `own` is true, else the plain form, which is
elementary torch operations in float32 (the router's logits in float64),
rounded once.  `exact()` is the operators' definition in float64.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5
MAX_FEW = 16  # tokens of the few-token layer


# ---- cases --------------------------------------------------------------------


def listed():
    return [
        # the rows of one decode step on their way into a 4-bit product: latency
        dict(name="mxfp4-rows-few", op="codec", rows=8, cols=2880, dtype="bf16"),
        # one up-projection of a Mixtral-shaped expert turned into MXFP4 and back
        dict(name="mxfp4-expert", op="codec", rows=14336, cols=4096, dtype="bf16"),
        # one token through a dense projection in MXFP4: bound by reading the weights
        dict(name="linear-token", op="linear", n=1, d=4096, m=14336, act="bf16", out="bf16", bias=False),
        # a ragged batch, an odd number of outputs, float32 results with a bias
        dict(name="linear-odd", op="linear", n=333, d=2880, m=5001, act="bf16", out="f32", bias=True),
        # a prompt's rows encoded as MXFP4 and multiplied in 4 bits on both sides
        dict(name="linear-batch-4x4", op="linear", n=8192, d=4096, m=14336, act="mxfp4", out="bf16",
             bias=False),
        # the 128-expert decode layer: one token, and eight
        dict(name="few-1-e128", op="few", n=1, d=2880, E=128, k=4, d_ff=2880, dtype="mxfp4", bias=False),
        dict(name="few-8-e128", op="few", n=8, d=2880, E=128, k=4, d_ff=2880, dtype="mxfp4", bias=False),
        # the Switch layer with as many tokens as the call takes, in bf16
        dict(name="few-16-switch", op="few", n=16, d=1024, E=8, k=1, d_ff=4096, dtype="bf16", bias=True),
        # one token's residual update and next norm between two decode layers: latency
        dict(name="norms-token", op="norms", n=1, d=2880, dtype="bf16", post="rms", pre="rms", gate=False),
        # the norms around the Mixtral-shaped layer's batch, and their gradient
        dict(name="norms-batch", op="norms", n=8192, d=4096, dtype="bf16", post="layer", pre="layer",
             gate=True),
        dict(name="norms-grad-batch", op="norms_grad", n=8192, d=4096, dtype="bf16", post="layer",
             pre="layer", gate=True),
        # an odd width and an odd number of rows in float32
        dict(name="norms-grad-odd-f32", op="norms_grad", n=4099, d=1021, dtype="f32", post="rms",
             pre="layer", gate=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["codec", "linear", "few", "norms", "norms_grad"])
    if op == "codec":
        cols = 32 * _log_int(rng, 1, 512)
        return dict(op=op, rows=_log_int(rng, 1, min(65536, (1 << 26) // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "linear":
        d, m = 32 * _log_int(rng, 2, 448), _log_int(rng, 16, 16384)
        n = _log_int(rng, 1, max(1, min(8192, (1 << 38) // (d * m))))
        return dict(op=op, n=n, d=d, m=m, act=rng.choice(["bf16", "mxfp4"]),
                    out=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    if op == "few":
        dtype = rng.choice(["mxfp4", "mxfp4", "bf16", "f32"])
        step = {"mxfp4": 32, "bf16": 8, "f32": 1}[dtype]
        d, f = (max(step, _log_int(rng, 64, 4096) // step * step) for _ in range(2))
        E = _log_int(rng, 1, 128)
        while E * d * f * 3 > 1 << 30:
            E = max(1, E // 2)
        return dict(op=op, n=rng.randint(1, MAX_FEW), d=d, E=E, k=rng.randint(1, min(E, 8)), d_ff=f,
                    dtype=dtype, bias=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    step = 8 if dtype == "bf16" else 1
    d = max(step, _log_int(rng, 16, 16384) // step * step)
    kinds = [None, "layer", "layer", "rms", "rms"]
    return dict(op=op, n=_log_int(rng, 1, min(65536, (1 << 25) // d)), d=d, dtype=dtype,
                post=rng.choice(kinds), pre=rng.choice(kinds), gate=rng.random() < 0.7)


# ---- inputs -------------------------------------------------------------------


def _scale_codes(x):
    """E8M0 codes of blocks of 32: floor(log2 of the largest magnitude) - 2,
    biased by 127, not below 0."""
    top = x.abs().amax(-1)
    e = torch.frexp(top).exponent
    return torch.where(top > 0, (e - 1 - 2 + 127).clamp(min=0), torch.zeros_like(e))


def _element_codes(a):
    """E2M1 codes of magnitudes, to nearest, ties to the even code."""
    c = (a > 0.25).to(torch.uint8)
    for border, closed in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= border) if closed else (a > border)
    return c


def _encode(x):
    """MXFP4 of the rows of x (float32): codes [rows][cols / 2], scales [rows][cols / 32]."""
    rows, cols = x.shape
    b = x.view(rows, cols // 32, 32)
    s = _scale_codes(b)
    v = b * torch.exp2(127.0 - s.to(torch.float32))[..., None]
    c = _element_codes(v.abs()) | (torch.signbit(v).to(torch.uint8) << 3)
    c = c.view(rows, cols // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), s.to(torch.uint8)


def _decode(q, s):
    """float32 values of an MXFP4 matrix."""
    rows, half = q.shape
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    pair = torch.stack((q & 15, q >> 4), -1).view(rows, half // 16, 32)
    scale = torch.exp2(s.double() - 127.0).float()
    return (lut[pair.int()] * scale[..., None]).view(rows, 2 * half)


def _norm(kind, normal, d):
    if kind is None:
        return None
    return dict(kind=kind, weight=1.0 + normal(d, scale=0.2),
                bias=normal(d, scale=0.2) if kind == "layer" else None, eps=EPS)


def _stats(v, kind):
    """What the forward pass keeps of a norm of the rows v (float64)."""
    mean = v.mean(1) if kind == "layer" else torch.zeros_like(v[:, 0])
    return mean, ((v - mean[:, None]).square().mean(1) + EPS).rsqrt()


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(scale)

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device=dev)

    u8, f32 = torch.uint8, torch.float32
    st = dict(case=dict(case))
    if case["op"] == "codec":
        rows, cols = case["rows"], case["cols"]
        # rows of different sizes, as a weight's output channels or tokens have
        x = normal(rows, cols) * torch.exp2(normal(rows, 1))
        st.update(x=x.to(DTYPES[case["dtype"]]), q=empty(rows, cols // 2, dtype=u8),
                  s=empty(rows, cols // 32, dtype=u8), y=empty(rows, cols, dtype=torch.bfloat16))
    elif case["op"] == "linear":
        n, d, m = case["n"], case["d"], case["m"]
        w, ws = _encode(normal(m, d, scale=d ** -0.5))
        st.update(x=normal(n, d).bfloat16(), w=w, w_s=ws, bias=normal(m) if case["bias"] else None,
                  y=empty(n, m, dtype=DTYPES[case["out"]]))
        if case["act"] == "mxfp4":
            st.update(q=empty(n, d // 2, dtype=u8), s=empty(n, d // 32, dtype=u8))
    elif case["op"] == "few":
        n, d, E, k, f = (case[key] for key in ("n", "d", "E", "k", "d_ff"))
        dt = DTYPES.get(case["dtype"], torch.bfloat16)
        st.update(x=normal(n, d).to(dt), wg=normal(E, d, scale=d ** -0.5).to(dt),
                  bias=normal(E, scale=0.5) if case["bias"] else None, y=empty(n, d, dtype=dt),
                  idx=empty(n, k, dtype=torch.int32), topk_w=empty(n, k, dtype=f32))
        for key, rows, cols in (("1", f, d), ("3", f, d), ("2", d, f)):
            if case["dtype"] == "mxfp4":
                w, s = empty(E, rows, cols // 2, dtype=u8), empty(E, rows, cols // 32, dtype=u8)
                for e in range(E):
                    w[e], s[e] = _encode(normal(rows, cols, scale=cols ** -0.5))
                st["s" + key] = s
            else:
                w = empty(E, rows, cols, dtype=dt)
                for e in range(E):
                    w[e] = normal(rows, cols, scale=cols ** -0.5)
            st["w" + key] = w
    else:
        n, d, dt = case["n"], case["d"], DTYPES[case["dtype"]]
        # the residual stream: a few channels stand out, and rows have a mean
        x = normal(n, d) + 2.0 * normal(n, 1)
        x = (x * (1.0 + 9.0 * (torch.rand(d, generator=gen, device=dev) < 0.02))).to(dt)
        z = normal(n, d, scale=0.7).to(dt)
        st.update(x=x, z=z, scale=1.25, gate=normal(d, scale=0.5) if case["gate"] else None,
                  post=_norm(case["post"], normal, d), pre=_norm(case["pre"], normal, d),
                  stats=empty(4, n, dtype=f32))
        if case["op"] == "norms":
            st.update(h=empty(n, d, dtype=dt), u=empty(n, d, dtype=dt) if case["pre"] else None)
        else:  # what the forward pass kept
            v, stats = z.double(), st["stats"]
            if case["post"]:
                stats[0], stats[1] = _stats(v, case["post"])
                v = (v - stats[0, :, None]) * stats[1, :, None] * st["post"]["weight"]
                if st["post"]["bias"] is not None:
                    v = v + st["post"]["bias"]
            h = st["scale"] * x.double() + (v if st["gate"] is None else v * st["gate"])
            if case["pre"]:
                stats[2], stats[3] = _stats(h, case["pre"])
            st.update(h=h.to(dt), dh=normal(n, d).to(dt), du=normal(n, d).to(dt) if case["pre"] else None,
                      dx=empty(n, d, dtype=dt), dz=empty(n, d, dtype=dt))
            for key in _param_grads(case):
                st[key] = empty(d, dtype=f32)
    return st


def _param_grads(case):
    """The parameters' gradients that a case of the norms has."""
    out = ["dgate"] if case["gate"] else []
    for name in ("post", "pre"):
        if case[name]:
            out.append("d%s_weight" % name)
        if case[name] == "layer":
            out.append("d%s_bias" % name)
    return out


# ---- one pass -------------------------------------------------------------------


def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _workspace(st, nbytes):
    """The workspace that a program keeps beside its buffers."""
    if "ws" not in st:
        st["ws"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    return st["ws"]


def _own_codec(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    B.moe_quantize_mxfp4(c["rows"], c["cols"], st["x"], c["dtype"], st["q"], st["s"])
    B.moe_dequantize_mxfp4(c["rows"], c["cols"], st["q"], st["s"], st["y"], "bf16")
    return {"y": st["y"]}


def _own_linear(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    n, d, m = c["n"], c["d"], c["m"]
    x, x_s = st["x"], None
    if c["act"] == "mxfp4":
        B.moe_quantize_mxfp4(n, d, x, "bf16", st["q"], st["s"])
        x, x_s = st["q"], st["s"]
    nb = B.moe_mxfp4_linear_workspace_bytes(n, d, m, c["act"])
    B.moe_mxfp4_linear(n, d, m, x, x_s, c["act"], st["w"], st["w_s"], st["bias"], st["y"], c["out"],
                       _workspace(st, nb), nb)
    return {"y": st["y"]}


def _own_few(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    shape = (c["n"], c["d"], c["E"], c["k"], c["d_ff"], -1)
    act = "f32" if c["dtype"] == "f32" else "bf16"
    w = dict(dtype=c["dtype"], **{key: st[key] for key in ("w1", "w3", "w2", "s1", "s3", "s2") if key in st})
    nb = B.moe_forward_few_workspace_bytes(shape, c["dtype"])
    B.moe_forward_few(shape, st["x"], act, st["wg"], st["bias"], w, st["y"], act, st["idx"], st["topk_w"],
                      _workspace(st, nb), nb)
    return {"y": st["y"], "idx": st["idx"], "topk_w": st["topk_w"]}


def _kept(st):
    """The rows of the statistics that the case's norms have."""
    rows = ([0, 1] if st["case"]["post"] else []) + ([2, 3] if st["case"]["pre"] else [])
    return {"stats%d" % r: st["stats"][r] for r in rows}


def _own_norms(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    B.moe_block_norm(c["n"], c["d"], st["x"], st["z"], c["dtype"], st["scale"], st["gate"], st["post"],
                     st["pre"], st["h"], st["u"], st["stats"])
    out = {"h": st["h"], **_kept(st)}
    if c["pre"]:
        out["u"] = st["u"]
    return out


def _own_norms_grad(st):
    from mixture_experts_layer_wave_amd import binding as B

    c = st["case"]
    nb = B.moe_block_norm_backward_workspace_bytes(c["n"], c["d"])
    B.moe_block_norm_backward(c["n"], c["d"], st["dh"], st["du"], st["z"], st["h"], c["dtype"], st["scale"],
                              st["gate"], st["post"], st["pre"], st["stats"], st["dx"], st["dz"],
                              st.get("dgate"), st.get("dpost_weight"), st.get("dpost_bias"),
                              st.get("dpre_weight"), st.get("dpre_bias"), _workspace(st, nb), nb)
    return {key: st[key] for key in ["dx", "dz"] + _param_grads(c)}


_own = dict(codec=_own_codec, linear=_own_linear, few=_own_few, norms=_own_norms, norms_grad=_own_norms_grad)


def _plain_codec(st):
    q, s = _encode(st["x"].float())
    return {"y": _decode(q, s).bfloat16()}


def _plain_linear(st):
    c = st["case"]
    x = st["x"].float()
    if c["act"] == "mxfp4":
        x = _decode(*_encode(x))
    y = x @ _decode(st["w"], st["w_s"]).t()
    if c["bias"]:
        y = y + st["bias"]
    return {"y": y.to(st["y"].dtype)}


def _plain_few(st):
    c = st["case"]
    z = st["x"].double() @ st["wg"].double().t()
    if c["bias"]:
        z = z + st["bias"]
    order = torch.sort(-z, dim=1, stable=True).indices[:, : c["k"]]
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = (p / p.sum(1, keepdim=True)).gather(1, order)
    if c["k"] > 1:
        p = p / p.sum(1, keepdim=True)
    x = st["x"].float()
    y = torch.zeros(c["n"], c["d"], device=x.device)
    for e in torch.unique(order).tolist():
        if c["dtype"] == "mxfp4":
            w1, w3, w2 = (_decode(st["w" + key][e], st["s" + key][e]) for key in "132")
        else:
            w1, w3, w2 = (st["w" + key][e].float() for key in "132")
        tok, slot = (order == e).nonzero(as_tuple=True)
        g, u = x[tok] @ w1.t(), x[tok] @ w3.t()
        o = (g / (1.0 + torch.exp(-g)) * u) @ w2.t()
        y[tok] += p[tok, slot][:, None].float() * o
    return {"y": y.to(st["x"].dtype), "idx": order.to(torch.int32), "topk_w": p.float()}


def _plain_norm(v, norm):
    """A norm of float32 rows: its values, and its mean and factor."""
    mean = v.sum(1, keepdim=True) / v.shape[1] if norm["kind"] == "layer" else torch.zeros_like(v[:, :1])
    c = v - mean
    rstd = 1.0 / torch.sqrt((c * c).sum(1, keepdim=True) / v.shape[1] + norm["eps"])
    y = c * rstd * norm["weight"]
    if norm["bias"] is not None:
        y = y + norm["bias"]
    return y, mean[:, 0], rstd[:, 0]


def _plain_norms(st):
    c, dt = st["case"], st["x"].dtype
    v, out = st["z"].float(), {}
    if c["post"]:
        v, out["stats0"], out["stats1"] = _plain_norm(v, st["post"])
    if c["gate"]:
        v = v * st["gate"]
    h = st["scale"] * st["x"].float() + v
    out["h"] = h.to(dt)
    if c["pre"]:
        u, out["stats2"], out["stats3"] = _plain_norm(h, st["pre"])
        out["u"] = u.to(dt)
    return out


def _plain_norm_grad(dy, v, mean, rstd, norm):
    """A norm's gradient: of its rows, its weight and its bias."""
    xh = (v - mean[:, None]) * rstd[:, None]
    t = dy * norm["weight"]
    dv = t - xh * ((t * xh).sum(1, keepdim=True) / v.shape[1])
    if norm["kind"] == "layer":
        dv = dv - t.sum(1, keepdim=True) / v.shape[1]
    return dv * rstd[:, None], (dy * xh).sum(0), dy.sum(0)


def _plain_norms_grad(st):
    c, dt, s = st["case"], st["z"].dtype, st["stats"]
    out, dh, z = {}, st["dh"].float(), st["z"].float()
    if c["pre"]:
        dv, out["dpre_weight"], db = _plain_norm_grad(st["du"].float(), st["h"].float(), s[2], s[3], st["pre"])
        dh = dh + dv
        if c["pre"] == "layer":
            out["dpre_bias"] = db
    out["dx"] = (st["scale"] * dh).to(dt)
    dn = dh
    if c["gate"]:
        v = z
        if c["post"]:
            v = (z - s[0][:, None]) * s[1][:, None] * st["post"]["weight"]
            if c["post"] == "layer":
                v = v + st["post"]["bias"]
        out["dgate"] = (dh * v).sum(0)
        dn = dh * st["gate"]
    if c["post"]:
        dn, out["dpost_weight"], db = _plain_norm_grad(dn, z, s[0], s[1], st["post"])
        if c["post"] == "layer":
            out["dpost_bias"] = db
    out["dz"] = dn.to(dt)
    return {key: out[key] for key in ["dx", "dz"] + _param_grads(c)}


_plain = dict(codec=_plain_codec, linear=_plain_linear, few=_plain_few, norms=_plain_norms,
              norms_grad=_plain_norms_grad)


# ---- what a pass cannot do without ----------------------------------------------


def work(case):
    if case["op"] == "codec":
        el = case["rows"] * case["cols"]
        return {"bytes": el * ((2 if case["dtype"] == "bf16" else 4) + 2) + el // 2 + el // 32, "flops": 4 * el}
    if case["op"] == "linear":
        n, d, m = case["n"], case["d"], case["m"]
        moved = 2 * n * d + m * (d // 2 + d // 32) + n * m * (2 if case["out"] == "bf16" else 4)
        return {"bytes": moved + (4 * m if case["bias"] else 0), "flops": 2 * n * d * m}
    n, d = case["n"], case["d"]
    if case["op"] == "few":
        E, k, f = case["E"], case["k"], case["d_ff"]
        s = 4 if case["dtype"] == "f32" else 2
        per = {"mxfp4": 0.5 + 1 / 32, "bf16": 2, "f32": 4}[case["dtype"]]
        active = E * (1.0 - (1.0 - k / E) ** n)  # experts with tokens, expected
        return {"bytes": int(3 * active * d * f * per) + (2 * n + E) * d * s + 8 * n * k,
                "flops": 6 * n * k * d * f + 2 * n * d * E}
    s, pre, post = 2 if case["dtype"] == "bf16" else 4, bool(case["pre"]), bool(case["post"])
    params = 4 * d * len(_param_grads(case))
    if case["op"] == "norms":
        return {"bytes": (3 + pre) * n * d * s + params + 8 * n * (pre + post),
                "flops": (3 + 8 * pre + 8 * post) * n * d}
    reads = 1 + 2 * pre + (post or case["gate"])
    return {"bytes": (reads + 2) * n * d * s + 2 * params + 8 * n * (pre + post),
            "flops": (3 + 14 * pre + 14 * post) * n * d}


# ---- the definitions in float64 -------------------------------------------------


def _exact_values(q, s):
    """Values of MXFP4 codes: sign, two exponent bits, one mantissa bit."""
    out = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
    for half in (0, 1):
        c = (q >> (4 * half)) & 15
        e, f = ((c >> 1) & 3).double(), (c & 1).double()
        mag = torch.where(e > 0, (1.0 + f / 2.0) * torch.exp2(e - 1.0), f / 2.0)
        out[:, half::2] = torch.where(c >= 8, -mag, mag)
    return out * torch.exp2(s.double() - 127.0).repeat_interleave(32, 1)


def _exact_rounded(x):
    """Rows of x rounded to MXFP4: a block's step structure from its largest
    magnitude, each value to the nearest multiple of its binade's step."""
    b = x.double().unflatten(1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    X = (torch.floor(torch.log2(top.clamp(min=2.0 ** -160))) - 2.0).clamp(min=-127.0)
    # log2 next to a power of two: settle the exponent by comparison
    X = torch.where(torch.exp2(X + 3.0) <= top, X + 1.0, X)
    X = torch.where((torch.exp2(X + 2.0) > top) & (X > -127.0), X - 1.0, X)
    v = b * torch.exp2(-X)
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return (torch.sign(v) * torch.clamp(torch.round(a / step) * step, max=6.0) * torch.exp2(X)).flatten(1)


def _exact_rows(v, norm):
    mean = v.mean(1) if norm["kind"] == "layer" else torch.zeros_like(v[:, 0])
    rstd = (v - mean[:, None]).pow(2).mean(1).add(norm["eps"]).pow(-0.5)
    y = torch.einsum("nd,n,d->nd", v - mean[:, None], rstd, norm["weight"].double())
    return (y if norm["bias"] is None else y + norm["bias"].double()), mean, rstd


def _exact_rows_grad(dy, v, mean, rstd, norm):
    """The part of W dy orthogonal to the rows' kept directions."""
    xh = (v - mean[:, None]) * rstd[:, None]
    t = dy * norm["weight"].double()
    dv = t - xh * torch.einsum("nd,nd->n", t, xh)[:, None] / v.shape[1]
    if norm["kind"] == "layer":
        dv = dv - t.mean(1, keepdim=True)
    return dv * rstd[:, None], torch.einsum("nd,nd->d", dy, xh), dy.sum(0)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "codec":
        return {"y": _exact_rounded(st["x"])}
    if case["op"] == "linear":
        x = _exact_rounded(st["x"]) if case["act"] == "mxfp4" else st["x"].double()
        y = torch.mm(x, _exact_values(st["w"], st["w_s"]).t())
        return {"y": y + st["bias"].double() if case["bias"] else y}
    if case["op"] == "few":
        z = torch.mm(st["x"].double(), st["wg"].double().t())
        if case["bias"]:
            z = z + st["bias"].double()
        prob = torch.softmax(z, 1)
        idx = torch.empty(case["n"], case["k"], dtype=torch.int32, device=z.device)
        left = z.clone()
        for j in range(case["k"]):  # the first of the largest, then without it
            best = left == left.amax(1, keepdim=True)
            idx[:, j] = best.int().argmax(1)
            left.scatter_(1, idx[:, j : j + 1].long(), -math.inf)
        w = prob.gather(1, idx.long())
        if case["k"] > 1:
            w = w / w.sum(1, keepdim=True)
        y = torch.zeros(case["n"], case["d"], dtype=torch.float64, device=z.device)
        for e in sorted(set(idx.flatten().tolist())):
            if case["dtype"] == "mxfp4":
                m = {key: _exact_values(st["w" + key][e], st["s" + key][e]) for key in "123"}
            else:
                m = {key: st["w" + key][e].double() for key in "123"}
            share = (w * (idx == e)).sum(1)  # 0 for tokens that do not take e
            rows = share.nonzero()[:, 0]
            xe = st["x"].double().index_select(0, rows)
            g = torch.mm(xe, m["1"].t())
            o = torch.mm(g * torch.sigmoid(g) * torch.mm(xe, m["3"].t()), m["2"].t())
            y.index_add_(0, rows, o * share[rows, None])
        return {"y": y, "idx": idx, "topk_w": w}
    z, gate = st["z"].double(), None if st["gate"] is None else st["gate"].double()
    if case["op"] == "norms":
        out, v = {}, z
        if case["post"]:
            v, out["stats0"], out["stats1"] = _exact_rows(z, st["post"])
        h = st["scale"] * st["x"].double() + (v if gate is None else v * gate)
        out["h"] = h
        if case["pre"]:
            out["u"], out["stats2"], out["stats3"] = _exact_rows(h, st["pre"])
        return out
    s, d_all, out = st["stats"].double(), st["dh"].double(), {}
    if case["pre"]:
        dv, out["dpre_weight"], out["dpre_bias"] = _exact_rows_grad(st["du"].double(), st["h"].double(), s[2],
                                                                    s[3], st["pre"])
        d_all = d_all + dv
    out["dx"] = st["scale"] * d_all
    into = d_all if gate is None else d_all * gate
    if case["post"]:
        out["dz"], out["dpost_weight"], out["dpost_bias"] = _exact_rows_grad(into, z, s[0], s[1], st["post"])
        v = (z - s[0, :, None]) * s[1, :, None] * st["post"]["weight"].double()
        v = v if st["post"]["bias"] is None else v + st["post"]["bias"].double()
    else:
        out["dz"], v = into, z
    out["dgate"] = torch.einsum("nd,nd->d", d_all, v)
    return {key: out[key] for key in ["dx", "dz"] + _param_grads(case)}
