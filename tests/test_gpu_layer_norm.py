"""GPU parity of moe_layer_norm and its gradient with the float64 oracle.

Tolerances (derived, not measured).  An output is rounded once, by at most
half a step: 2^-8 of the value for bf16, 2^-24 for float32.  Before that all
arithmetic is float32.  A row's sum adds at most 16 elements per thread, then
6 lane steps and 16 wave sums: under 40 additions deep, so a sum is off by at
most 40 * 2^-24 of the sum of magnitudes; products, the square root and the
division add a few 2^-24.  64 * 2^-24 of the magnitudes involved covers both.
A column sum over n rows is at most n / 256 + 64 + 32 additions deep."""

import numpy as np
import pytest

import oracle
from tests.gpu_support import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SIZES = {
    "bf16": [(2, 1024), (1, 8), (3, 16), (7, 136), (65, 512), (33, 520), (2, 2048), (1, 4096), (300, 4096), (5, 4104),
             (9, 8192), (3, 8200), (2, 16384), (5000, 64), (2600, 1024)],
    "f32": [(4, 511), (1, 1), (2, 3), (5, 17), (6, 64), (7, 65), (9, 255), (4, 257), (33, 1021), (5, 1024), (3, 2047),
            (9, 2049), (3, 4097), (2, 8193), (2, 16383), (1, 16384), (5000, 33), (2600, 500)],
}
CASES = [(t, n, d) for t in SIZES for n, d in SIZES[t]]


def _tensor(a, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)


def _f64(t):
    return t.double().cpu().numpy()


def _inputs(dtype, n, d, seed=0):
    rng = np.random.default_rng(1000 * n + d + seed)
    x = _tensor(rng.standard_normal((n, d)) + 2.0 * rng.standard_normal((n, 1)), dtype)
    dy = _tensor(rng.standard_normal((n, d)), dtype)
    w, b = _tensor(1 + 0.3 * rng.standard_normal(d), "f32"), _tensor(rng.standard_normal(d), "f32")
    return x, dy, w, b


def _forward(x, dtype, w, b, eps=1e-5, stats=True, stream=None):
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    n, d = x.shape
    y = torch.full((n + 1, d), 7.0, dtype=x.dtype, device="cuda")  # one row more than the call's
    mean = torch.full((n + 1,), 7.0, device="cuda")
    rstd = torch.full((n + 1,), 7.0, device="cuda")
    B.moe_layer_norm(n, d, x, dtype, w, b, eps, y, mean if stats else None, rstd if stats else None, stream)
    torch.cuda.synchronize()
    assert (y[n] == 7).all() and mean[n] == 7 and rstd[n] == 7  # rows behind the last are left as they were
    return y[:n], mean[:n], rstd[:n]


def _backward(dy, x, dtype, w, mean, rstd, want=("dw", "db")):
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    n, d = x.shape
    dx = torch.full((n + 1, d), 7.0, dtype=x.dtype, device="cuda")
    dw = torch.full((d + 1,), 7.0, device="cuda")
    db = torch.full((d + 1,), 7.0, device="cuda")
    nb = B.moe_layer_norm_backward_workspace_bytes(n, d)
    ws = torch.full((nb + 256,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns, and a guard
    B.moe_layer_norm_backward(n, d, dy, x, dtype, w, mean, rstd, dx, dw if "dw" in want else None,
                              db if "db" in want else None, ws, nb)
    torch.cuda.synchronize()
    assert (dx[n] == 7).all() and dw[d] == 7 and db[d] == 7 and (ws[nb:] == 255).all()
    return dx[:n], dw[:d], db[:d]


def _check(name, got, ref, tol):
    assert np.isfinite(got).all(), name
    worst = float(np.max((np.abs(got - ref) / np.maximum(tol, 1e-300)), initial=0.0))
    say(f"    {name}: largest error / tolerance {worst:.3f}")
    assert worst <= 1.0, name


@pytest.mark.parametrize("dtype,n,d", CASES)
def test_forward(dtype, n, d):
    say(f"[layer norm] {dtype} {n} x {d}")
    x, _, w, b = _inputs(dtype, n, d)
    for bias in (b, None):
        y, mean, rstd = _forward(x, dtype, w, bias)
        x64, w64 = _f64(x), _f64(w)
        b64 = _f64(b) if bias is not None else np.zeros(d)
        ref, m, r = oracle.layer_norm(x64, w64, b64, 1e-5)
        size = np.abs(x64).mean(axis=1)
        _check("mean", _f64(mean), m, 64 * U * size)
        # rstd: the variance's relative error halves; the mean's error enters squared
        _check("rstd", _f64(rstd), r, 64 * U * r)
        spread = np.abs(x64 - m[:, None]) + size[:, None]
        tol = HALF[dtype] * np.abs(ref) + 64 * U * (spread * r[:, None] * np.abs(w64) + np.abs(b64))
        _check("y", _f64(y), ref, tol)


@pytest.mark.parametrize("dtype,n,d", CASES)
def test_backward(dtype, n, d):
    say(f"[layer norm grad] {dtype} {n} x {d}")
    x, dy, w, _ = _inputs(dtype, n, d)
    x64, dy64, w64 = _f64(x), _f64(dy), _f64(w)
    _, m, r = oracle.layer_norm(x64, w64)
    mean, rstd = _tensor(m, "f32"), _tensor(r, "f32")
    dx, dw, db = _backward(dy, x, dtype, w, mean, rstd)
    m, r = _f64(mean), _f64(rstd)  # the gradient is of the statistics it was given
    rx, rw, rb = oracle.layer_norm_grad(dy64, x64, w64, m, r)
    # xh is off by 2^-24 of its terms' sizes
    xs = (np.abs(x64) + np.abs(m)[:, None]) * r[:, None]
    t = np.abs(dy64 * w64)
    tol = HALF[dtype] * np.abs(rx) + 64 * U * r[:, None] * (
        t + t.mean(axis=1, keepdims=True) + xs * (t * xs).mean(axis=1, keepdims=True))
    _check("dx", _f64(dx), rx, tol)
    depth = n / 256 + 96
    _check("dweight", _f64(dw), rw, depth * U * (np.abs(dy64) * xs).sum(axis=0))
    _check("dbias", _f64(db), rb, depth * U * np.abs(dy64).sum(axis=0))
    # the same call again gives the same bits
    for a, c in zip((dx, dw, db), _backward(dy, x, dtype, w, mean, rstd)):
        assert (a == c).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 72), ("bf16", 4096), ("f32", 21), ("f32", 5001)])
def test_gradient_against_differences(dtype, d):
    """<dx, v> against a central difference of sum(y dy) along v, with the
    library's forward pass in float64's place only for the sums: the forward
    is run at x +- h v (rounded to the stored type first)."""
    n, h = 3, 2.0 ** -6
    say(f"[layer norm difference] {dtype} {d}")
    x, dy, w, b = _inputs(dtype, n, d, seed=1)
    rng = np.random.default_rng(d)
    v = np.sign(rng.standard_normal((n, d)))
    xp, xm = _tensor(_f64(x) + h * v, dtype), _tensor(_f64(x) - h * v, dtype)
    _, mean, rstd = _forward(x, dtype, w, b)
    dx, dw, db = _backward(dy, x, dtype, w, mean, rstd)
    dy64 = _f64(dy)
    yp = _f64(_forward(xp, dtype, w, b)[0]) - _f64(_forward(xm, dtype, w, b)[0])
    step = _f64(xp) - _f64(xm)
    # the true directional difference, which the oracle's forward gives exactly
    op = (oracle.layer_norm(_f64(xp), _f64(w), _f64(b))[0] - oracle.layer_norm(_f64(xm), _f64(w), _f64(b))[0])
    got, want = (_f64(dx) * step).sum(), (op * dy64).sum()
    # the third-order term: |step / 2|^3 / 3 of a smooth row function with
    # derivatives of order w rstd^3; and half a step of each dx
    r = _f64(rstd)[:, None]
    tol = HALF[dtype] * np.abs(_f64(dx) * step).sum() + \
        4 * np.abs(dy64 * _f64(w)).sum() * float(np.max((np.abs(step) / 2 * r) ** 3)) + 1e-4 * np.abs(want)
    assert abs(got - want) <= tol, (got, want, tol)
    # and the kernel's own forward moves by the same amount, up to its outputs' rounding
    size = np.abs(_f64(_forward(x, dtype, w, b)[0])) + np.abs(yp)
    assert abs((yp * dy64).sum() - want) <= (2 * HALF[dtype] + 256 * U) * (size * np.abs(dy64)).sum() * 2


def test_rows_past_32_bit_offsets():
    """131500 rows of 16384: the last ones lie more than 2^32 bytes and 2^31
    elements in.  dy is zero in all but a few rows."""
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    say("[layer norm, offsets past 32 bits]")
    n, d = 131500, 16384
    rows = [0, 65536, n - 2, n - 1]
    xs, dys, w, b = _inputs("bf16", len(rows), d, seed=3)
    x, dy = (torch.zeros(n, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[rows], dy[rows] = xs, dys
    y, dx = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    mean, rstd = (torch.empty(n, device="cuda") for _ in range(2))
    dw, db = (torch.empty(d, device="cuda") for _ in range(2))
    nb = B.moe_layer_norm_backward_workspace_bytes(n, d)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    B.moe_layer_norm(n, d, x, "bf16", w, b, 1e-5, y, mean, rstd)
    B.moe_layer_norm_backward(n, d, dy, x, "bf16", w, mean, rstd, dx, dw, db, ws, nb)
    torch.cuda.synchronize()
    # the same rows by themselves, which the tests above hold to the oracle
    ys, means, rstds = _forward(xs, "bf16", w, b)
    dxs, dws, dbs = _backward(dys, xs, "bf16", w, means, rstds)
    assert torch.equal(y[rows], ys) and torch.equal(mean[rows], means) and torch.equal(rstd[rows], rstds)
    assert torch.equal(dx[rows], dxs)
    # Sums over rows: the same four addends (and exact zeros) in two orders, each
    # sum four roundings of at most 2^-24 of the addends' sizes.
    xh = (xs.double() - means.double()[:, None]) * rstds.double()[:, None]
    for p, q, size in ((dw, dws, (dys.double() * xh).abs().sum(0)), (db, dbs, dys.double().abs().sum(0))):
        assert ((p.double() - q.double()).abs() <= 9 * 2.0 ** -24 * size).all()
    other = torch.ones(n, dtype=torch.bool, device="cuda")
    other[rows] = False
    assert not dx[other].any()


def test_no_rows_and_optional_outputs():
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    say("[layer norm] no rows, optional outputs")
    d = 64
    dw, db = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
    B.moe_layer_norm(0, d, None, "bf16", None, None, 1e-5, None)
    B.moe_layer_norm_backward(0, d, None, None, "bf16", None, None, None, None, dw, db, None, 0)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()
    x, dy, w, b = _inputs("bf16", 5, d)
    y, mean, rstd = _forward(x, "bf16", w, b)
    y2, m2, r2 = _forward(x, "bf16", w, b, stats=False)
    assert (y == y2).all() and (m2 == 7).all() and (r2 == 7).all()
    dx, dw, db = _backward(dy, x, "bf16", w, mean, rstd)
    for want in (("dw",), ("db",), ()):
        dx2, dw2, db2 = _backward(dy, x, "bf16", w, mean, rstd, want)
        assert (dx == dx2).all()
        assert (dw2 == (dw if "dw" in want else 7)).all() and (db2 == (db if "db" in want else 7)).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 4096), ("f32", 37), ("f32", 4096)])
def test_rows_stay_apart(dtype, d):
    """A row of equal values has rstd 1 / sqrt(eps) and y = bias; a row with a
    NaN or an infinity spoils itself alone, and a far offset keeps its
    differences."""
    import torch

    say(f"[layer norm rows] {dtype} {d}")
    x, dy, w, b = _inputs(dtype, 6, d)
    x[1] = 3.0
    x[3, d // 2] = float("nan")
    x[4, 0] = float("inf")
    x[5] = 1024.0 + 8.0 * (torch.arange(d, device="cuda") % 2)  # exact in bf16 and float32
    y, mean, rstd = _forward(x, dtype, w, b)
    assert mean[1] == 3.0 and abs(float(rstd[1]) * np.sqrt(1e-5) - 1) < 64 * U
    assert (y[1] == b.to(y.dtype)).all()
    assert torch.isnan(y[3]).all() and torch.isnan(y[4, 0])
    ref, _, _ = oracle.layer_norm(_f64(x[[0, 2, 5]]), _f64(w), _f64(b))
    got = _f64(y[[0, 2, 5]])
    assert np.abs(got - ref).max() <= (HALF[dtype] * 4 + 1e-3) * np.abs(ref).max()
    dx, dw, db = _backward(dy, x, dtype, w, mean, rstd)
    alone, _, _ = _backward(dy[[0, 1, 2, 5]].contiguous(), x[[0, 1, 2, 5]].contiguous(), dtype, w,
                            mean[[0, 1, 2, 5]].contiguous(), rstd[[0, 1, 2, 5]].contiguous())
    assert torch.equal(dx[[0, 1, 2, 5]], alone)


def test_capture_replays_on_another_stream():
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    say("[layer norm] graph on a side stream")
    n, d = 300, 1024
    x, dy, w, b = _inputs("bf16", n, d)
    y, mean, rstd = _forward(x, "bf16", w, b)
    dx, dw, db = _backward(dy, x, "bf16", w, mean, rstd)
    out = [torch.zeros_like(t) for t in (y, mean, rstd, dx, dw, db)]
    nb = B.moe_layer_norm_backward_workspace_bytes(n, d)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()

    def step():
        B.moe_layer_norm(n, d, x, "bf16", w, b, 1e-5, out[0], out[1], out[2], s)
        B.moe_layer_norm_backward(n, d, dy, x, "bf16", w, out[1], out[2], out[3], out[4], out[5], ws, nb, s)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            step()
    for _ in range(3):
        for t in out:
            t.fill_(-1)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, c in zip(out, (y, mean, rstd, dx, dw, db)):
            assert torch.equal(a, c)
