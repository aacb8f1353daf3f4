"""GPU parity of the MXFP4 codec and product with the float64 oracle.

The codec is exact: its codes, scales and values are compared bit for bit.
The product's tolerance (derived, not measured): products of the stored values
are exact in float32, or below half a unit of the sum; a sum over d terms is
split over at least two accumulators fed 32 terms at a time, so it is at most
d / 32 + 64 additions deep, each off by at most 2^-24 of the running sum's
magnitudes; the result is rounded once (half a step: 2^-8 bf16, 2^-24 float32)."""

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


def _dev(a, dtype):
    torch, _ = _torch()
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def _f64(t):
    return t.double().cpu().numpy()


def _encode(x, dtype, cols=None):
    torch, B = _torch()
    rows, cols = x.shape
    q = torch.full((rows * cols // 2 + 64,), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((rows * cols // 32 + 64,), 7, dtype=torch.uint8, device="cuda")
    B.moe_quantize_mxfp4(rows, cols, x, dtype, q, s)
    torch.cuda.synchronize()
    assert (q[rows * cols // 2:] == 7).all() and (s[rows * cols // 32:] == 7).all()
    return q[: rows * cols // 2].view(rows, -1), s[: rows * cols // 32].view(rows, -1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (1, 2880), (8, 2880), (257, 96), (700, 4096), (5, 16384)])
def test_encode_and_decode(dtype, rows, cols):
    torch, B = _torch()
    say(f"[mxfp4] {dtype} {rows} x {cols}")
    rng = np.random.default_rng(rows + cols)
    x = _dev(rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1))), dtype)
    q, s = _encode(x, dtype)
    rq, rs = S.encode_mxfp4(_f64(x))
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)
    ref = oracle.decode_mxfp4(rq, rs)
    for out in ("bf16", "f32"):
        y = torch.full((rows + 1, cols), 7.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
        B.moe_dequantize_mxfp4(rows, cols, q.contiguous(), s.contiguous(), y, out)
        torch.cuda.synchronize()
        assert np.array_equal(_f64(y[:rows]), ref) and (y[rows] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_encode_edges(dtype):
    """Every border of the rounding at every sign, small and large exponents,
    zeros, float32 subnormals, infinities and NaN; neighbours of a bad block
    are not affected."""
    say(f"[mxfp4 edges] {dtype}")
    borders = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7.96875])
    block = np.concatenate([borders, -borders])
    rows = [block * 2.0 ** e for e in (-126, -125, -120, -3, 0, 1, 60, 120, 124)]
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    rows += [block * (1 + step), block * (1 - step / 2) if dtype == "f32" else block]
    rows += [np.zeros(32), -np.zeros(32), np.full(32, 2.0 ** -130), np.full(32, -2.0 ** -133)]
    for bad in (np.inf, -np.inf, np.nan):
        v = block.copy()
        v[17] = bad
        rows += [v, block]
    x = np.array(rows, np.float32).reshape(1, -1)
    x = np.concatenate([x, x[:, ::-1]])
    t = _dev(x, dtype)
    q, s = _encode(t, dtype)
    rq, rs = S.encode_mxfp4(_f64(t))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


def test_decode_every_code():
    torch, B = _torch()
    say("[mxfp4 decode] all codes at all scales")
    q = np.tile((np.arange(16, dtype=np.uint8) % 16) | ((np.arange(16, dtype=np.uint8) ^ 5) << 4), (256, 1)).astype(np.uint8)
    s = np.arange(256, dtype=np.uint8)[:, None]
    # E2M1's 4 and 6 at scale 2^126, and 2, 3, 4, 6 at 2^127, are 2^128 or more: past
    # the largest finite value of both output types (below 2^128), so they round to infinity
    ref = oracle.decode_mxfp4(q, s)
    ref = np.where(np.abs(ref) >= 2.0 ** 128, np.copysign(np.inf, ref), ref)
    for out, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        y = torch.zeros((256, 32), dtype=dt, device="cuda")
        B.moe_dequantize_mxfp4(256, 32, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), y, out)
        assert np.array_equal(_f64(y), ref, equal_nan=True), out


def test_codec_past_32_bit_offsets():
    """2^31 + elements: the last rows' values and codes."""
    torch, B = _torch()
    rows, cols = (1 << 31) // 16384 + 3, 16384
    say(f"[mxfp4 far] {rows} x {cols}")
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = _dev(np.random.default_rng(1).standard_normal((5, cols)), "bf16")
    x[-5:] = tail
    x[:5] = tail * 2
    q = torch.zeros((rows, cols // 2), dtype=torch.uint8, device="cuda")
    s = torch.zeros((rows, cols // 32), dtype=torch.uint8, device="cuda")
    B.moe_quantize_mxfp4(rows, cols, x, "bf16", q, s)
    rq, rs = S.encode_mxfp4(_f64(tail))
    assert np.array_equal(q[-5:].cpu().numpy(), rq) and np.array_equal(s[-5:].cpu().numpy(), rs)
    assert np.array_equal(q[:5].cpu().numpy(), rq) and np.array_equal(s[:5].cpu().numpy(), rs + 1)
    assert not q[5:-5].any() and not s[5:-5].any()
    x.fill_(3.0)
    B.moe_dequantize_mxfp4(rows, cols, q, s, x, "bf16")
    ref = oracle.decode_mxfp4(rq, rs)
    assert np.array_equal(_f64(x[-5:]), ref) and np.array_equal(_f64(x[:5]), 2 * ref)
    assert not x[5:-5].any()


# rows, width, outputs: one row to many, a single block of width, one output, odd
# numbers of both, widths that end inside a K step, every group of 16 rows
SIZES = [(1, 32, 1), (1, 4096, 300), (2, 96, 17), (4, 2880, 33), (5, 64, 1000), (8, 1024, 257), (9, 160, 16),
         (15, 544, 15), (16, 2880, 700), (17, 128, 40), (33, 320, 65), (64, 512, 129), (65, 2880, 513),
         (130, 96, 384), (257, 1056, 301), (300, 4096, 1025), (1000, 256, 72), (513, 7200, 130), (2050, 224, 530)]


def _product(n, d, m, act, out, bias, seed=0, x=None, stream=None, w=None):
    """(y, x64, w64, b64)"""
    torch, B = _torch()
    rng = np.random.default_rng(seed + n + 7 * d + 13 * m)
    xb = _dev(rng.standard_normal((n, d)), "bf16") if x is None else x
    w = _dev(rng.standard_normal((m, d)) * d ** -0.5, "f32") if w is None else w
    wq, ws = _encode(w, "f32")
    b = _dev(rng.standard_normal(m), "f32") if bias else None
    xin, xs, x64 = xb, None, _f64(xb)
    if act == "mxfp4":
        xin, xs = _encode(xb, "bf16")
        x64 = oracle.decode_mxfp4(xin.cpu().numpy(), xs.cpu().numpy())
        xin, xs = xin.contiguous(), xs.contiguous()
    y = torch.full((n * m + 64,), 7.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    nb = B.moe_mxfp4_linear_workspace_bytes(n, d, m, act)
    work = torch.full((nb + 256,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns, and a guard
    B.moe_mxfp4_linear(n, d, m, xin, xs, act, wq.contiguous(), ws.contiguous(), b, y, out, work, nb, stream)
    torch.cuda.synchronize()
    assert (y[n * m:] == 7).all() and (work[nb:] == 255).all()
    w64 = oracle.decode_mxfp4(wq.cpu().numpy(), ws.cpu().numpy())
    return y[: n * m].view(n, m), x64, w64, np.zeros(m) if b is None else _f64(b)


def _tolerance(ref, x64, w64, b64, out):
    depth = x64.shape[1] / 32 + 64
    return HALF[out] * np.abs(ref) + depth * U * (np.abs(x64) @ np.abs(w64).T + np.abs(b64))


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n,d,m", SIZES)
def test_linear(act, n, d, m):
    for out, bias in (("bf16", False), ("f32", True)):
        say(f"[mxfp4 linear] {act} {n} x {d} -> {m}, {out}, bias {bias}")
        y, x64, w64, b64 = _product(n, d, m, act, out, bias)
        ref = x64 @ w64.T + b64
        err = np.abs(_f64(y) - ref) / _tolerance(ref, x64, w64, b64, out)
        say(f"    largest error / tolerance {err.max():.3f}")
        assert err.max() <= 1.0


@pytest.mark.parametrize("act,n,d,m", [("bf16", 16, 3584, 50), ("bf16", 16, 4096, 300), ("bf16", 13, 5024, 33),
                                       ("bf16", 15, 4096, 17), ("mxfp4", 16, 14848, 40), ("mxfp4", 16, 16384, 20)])
def test_linear_rows_about_as_large_as_lds(act, n, d, m):
    say(f"[mxfp4 linear] long rows, {act} {n} x {d} -> {m}")
    y, x64, w64, b64 = _product(n, d, m, act, "f32", True)
    ref = x64 @ w64.T + b64
    assert (np.abs(_f64(y) - ref) <= _tolerance(ref, x64, w64, b64, "f32")).all()


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n,d,m", [(60, (1 << 24) - 32, 60), (16, (1 << 26) - 32, 15)])
def test_linear_of_the_longest_rows(act, n, d, m):
    """Matrices of close to 2^30 elements: x is 0 but in its first and last columns."""
    torch, B = _torch()
    say(f"[mxfp4 linear] far, {act} {n} x {d} -> {m}")
    torch.manual_seed(n)
    wq = torch.randint(0, 256, (m, d // 2), dtype=torch.uint8, device="cuda")
    ws = torch.randint(120, 130, (m, d // 32), dtype=torch.uint8, device="cuda")

    def both(t, per):
        return torch.cat([t[:, :512 // per], t[:, -512 // per:]], 1).cpu().numpy()

    w64 = oracle.decode_mxfp4(both(wq, 2), both(ws, 32))
    xs = None
    if act == "bf16":
        x = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
        x[:, :512] = torch.randn((n, 512), device="cuda")
        x[:, -512:] = torch.randn((n, 512), device="cuda")
        x64 = _f64(torch.cat([x[:, :512], x[:, -512:]], 1))
    else:
        x = torch.zeros((n, d // 2), dtype=torch.uint8, device="cuda")
        x[:, :256] = torch.randint(0, 256, (n, 256), dtype=torch.uint8, device="cuda")
        x[:, -256:] = torch.randint(0, 256, (n, 256), dtype=torch.uint8, device="cuda")
        xs = torch.full((n, d // 32), 125, dtype=torch.uint8, device="cuda")
        x64 = oracle.decode_mxfp4(both(x, 2), both(xs, 32))
    assert x64.shape[1] == w64.shape[1] == 1024
    y = torch.full((n, m), 7.0, device="cuda")
    nb = B.moe_mxfp4_linear_workspace_bytes(n, d, m, act)
    work = torch.empty(nb + 16, dtype=torch.uint8, device="cuda")
    B.moe_mxfp4_linear(n, d, m, x, xs, act, wq, ws, None, y, "f32", work, nb)
    torch.cuda.synchronize()
    ref = x64 @ w64.T
    assert (np.abs(_f64(y) - ref) <= _tolerance(ref, x64, w64, np.zeros(m), "f32")).all()


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_linear_of_the_largest_output(act):
    """Close to 2^30 outputs, thousands of tiles: rows from all over against 64 bits."""
    torch, B = _torch()
    n, d, m = 32700, 64, 32701
    say(f"[mxfp4 linear] large output, {act} {n} x {d} -> {m}")
    torch.manual_seed(2)
    wq = torch.randint(0, 256, (m, d // 2), dtype=torch.uint8, device="cuda")
    ws = torch.randint(120, 130, (m, d // 32), dtype=torch.uint8, device="cuda")
    w64 = oracle.decode_mxfp4(wq.cpu().numpy(), ws.cpu().numpy())
    x, xs = torch.randn((n, d), device="cuda").bfloat16(), None
    if act == "mxfp4":
        x, xs = (t.contiguous() for t in _encode(x, "bf16"))
    y = torch.full((n * m + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    nb = B.moe_mxfp4_linear_workspace_bytes(n, d, m, act)
    work = torch.empty(nb + 16, dtype=torch.uint8, device="cuda")
    B.moe_mxfp4_linear(n, d, m, x, xs, act, wq, ws, None, y, "bf16", work, nb)
    torch.cuda.synchronize()
    assert (y[n * m:] == 7).all()
    rows = [0, 1, 255, 256, 8191, 16385, 25000, n - 257, n - 2, n - 1]
    x64 = oracle.decode_mxfp4(x[rows].cpu().numpy(), xs[rows].cpu().numpy()) if xs is not None else _f64(x[rows])
    ref = x64 @ w64.T
    got = _f64(y[: n * m].view(n, m)[rows])
    assert (np.abs(got - ref) <= _tolerance(ref, x64, w64, np.zeros(m), "bf16")).all()


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n,d,m", [(450, 672, 2600), (200, 32, 6500), (450, 3200, 2600), (1025, 416, 2100),
                                   (1025, 64, 2100), (2100, 160, 2200), (2100, 32, 2200)])
def test_linear_of_about_as_many_tiles_as_compute_units(act, n, d, m):
    """Blocks whose groups of waves share K: steps that do not divide among them, fewer
    steps than groups, and the next larger tiles."""
    for out, bias in (("bf16", False), ("f32", True)):
        say(f"[mxfp4 linear] shared K, {act} {n} x {d} -> {m}, {out}")
        y, x64, w64, b64 = _product(n, d, m, act, out, bias)
        ref = x64 @ w64.T + b64
        assert (np.abs(_f64(y) - ref) <= _tolerance(ref, x64, w64, b64, out)).all()


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n,d,m", [(4600, 288, 4500), (7000, 64, 4200), (300, 544, 70001), (4352, 512, 4096)])
def test_linear_of_more_tiles_than_compute_units(act, n, d, m):
    """Blocks that take several tiles: ragged and whole ones behind each other, of one K
    step, of an odd and of an even number."""
    for out, bias in (("bf16", True), ("f32", False)):
        say(f"[mxfp4 linear] tiles in turn, {act} {n} x {d} -> {m}, {out}")
        y, x64, w64, b64 = _product(n, d, m, act, out, bias)
        for r in range(0, n, 1024):
            x = x64[r:r + 1024]
            ref = x @ w64.T + b64
            assert (np.abs(_f64(y[r:r + 1024]) - ref) <= _tolerance(ref, x, w64, b64, out)).all()


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n", [3, 70, 300])
def test_linear_keeps_nan_and_infinities_where_they_are(act, n):
    """A NaN block of W spoils its output column, one of x its row, no other."""
    torch, B = _torch()
    d, m = 160, 90
    say(f"[mxfp4 linear] NaN, {act}, {n} rows")
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((n, d)), rng.standard_normal((m, d))
    clean, _, _, _ = _product(n, d, m, act, "f32", False, x=_dev(x, "bf16"), w=_dev(w, "f32"))
    w[40, 150], w[77, 3] = np.inf, np.nan  # 255 in the encoding
    x[n - 1, 33] = np.inf if act == "bf16" else np.nan
    x[0, 159] = np.nan
    y, _, _, _ = _product(n, d, m, act, "f32", False, x=_dev(x, "bf16"), w=_dev(w, "f32"))
    bad = np.zeros((n, m), bool)
    bad[:, [40, 77]] = True
    bad[[0, n - 1]] = True
    got = _f64(y)
    assert not np.isfinite(got[bad]).any()
    assert np.array_equal(got[~bad], _f64(clean)[~bad])


def test_linear_rows_do_not_depend_on_the_stream_or_a_graph():
    torch, B = _torch()
    for act, n, d, m in (("bf16", 5, 1024, 200), ("mxfp4", 40, 512, 300), ("bf16", 600, 512, 300),
                         ("mxfp4", 600, 512, 300)):
        say(f"[mxfp4 linear] stream and graph, {act}, {n} rows")
        xb = _dev(np.random.default_rng(3).standard_normal((n, d)), "bf16")
        w = _dev(np.random.default_rng(4).standard_normal((m, d)), "f32")
        wq, ws = (t.contiguous() for t in _encode(w, "f32"))
        q, s = (t.contiguous() for t in _encode(xb, "bf16"))
        y = torch.zeros((n, m), device="cuda")
        nb = B.moe_mxfp4_linear_workspace_bytes(n, d, m, act)
        work = torch.zeros(nb + 16, dtype=torch.uint8, device="cuda")

        def step():
            if act == "mxfp4":
                B.moe_quantize_mxfp4(n, d, xb, "bf16", q, s)
            B.moe_mxfp4_linear(n, d, m, q if act == "mxfp4" else xb, s, act, wq, ws, None, y, "f32", work, nb)

        step()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            step()
        for rep in range(3):
            xb.copy_(_dev(np.random.default_rng(30 + rep).standard_normal((n, d)), "bf16"))
            step()
            torch.cuda.synchronize()
            want = y.clone()
            y.zero_()
            work.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)


def test_linear_of_nothing_leaves_the_output():
    torch, B = _torch()
    y = torch.full((4,), 7.0, device="cuda")
    B.moe_mxfp4_linear(0, 64, 4, None, None, "bf16", None, None, None, y, "f32")
    B.moe_quantize_mxfp4(0, 64, None, "bf16", None, None)
    torch.cuda.synchronize()
    assert (y == 7).all()
