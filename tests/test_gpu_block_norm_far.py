"""moe_block_norm where the rows that the norm in front sees lie far from zero.

That norm takes h before its rounding, float32 values of any row, in calls of
either type.  Tolerances (derived, not measured); U = 2^-24.

Rows of one value: a float64 sum of 2^14 values of 24 bits is exact, so the mean
is the value, its rest 0, and so are the differences: rstd = 1 / sqrt(eps) and
u = bias, rounded once.

Rows far from zero: an element of h is off by 2 U of its size (two roundings),
which is the offset's.  The mean is off by the average of that and by U of the
rest that its own last bit leaves (U of the offset), the differences by both and
U of themselves; sums of under 64 additions and the roundings around them are
covered by 96 U of the spread."""

import numpy as np
import pytest

from oracle import serve_oracle as S
from tests.gpu_support import say
from tests.test_gpu_block_norm import A, HALF, U, _check, _f64, _norm64, _tensor

pytestmark = pytest.mark.gpu

WIDTHS = [8, 136, 520, 1024, 2880, 4096, 8192, 8200, 16384]
VALUES = [(9984.0, 17.25), (-1e5, 3.0), (1.0, 1000.0), (-7.5, 1 / 3), (3e-3, 0.0), (1e30, 1e28), (0.0, 0.0)]


def _run(x, z, dtype, scale, post, pre, gate=None):
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    n, d = x.shape
    h, u = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    st = torch.full((4, n), 7.0, device="cuda")
    B.moe_block_norm(n, d, x, z, dtype, scale, gate, post, pre, h, u, st)
    torch.cuda.synchronize()
    return h, u, st


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_rows_of_one_value(d, dtype):
    """h = scale x + z, the same along a row, in 24 bits: the norm of it is the bias."""
    import torch

    say(f"[block norm in front, equal values] {dtype} {d}")
    rng = np.random.default_rng(d)
    rows = np.array(VALUES + list(zip(rng.uniform(1, 1e4, 60), rng.uniform(-10, 10, 60))))
    x, z = (_tensor(np.repeat(rows[:, i : i + 1], d, axis=1), dtype) for i in (0, 1))
    pre = dict(kind="layer", weight=_tensor(1 + 0.3 * rng.standard_normal(d), "f32"),
               bias=_tensor(rng.standard_normal(d), "f32"), eps=1e-5)
    h, u, st = _run(x, z, dtype, 1.1, None, pre)
    assert torch.equal(u, pre["bias"].to(u.dtype).expand_as(u))
    # the mean is h before its rounding
    want = np.float32(1.1).astype(np.float64) * _f64(x[:, 0]) + _f64(z[:, 0])
    assert (np.abs(_f64(st[2]) - want) <= 2 * U * np.abs(want)).all()
    assert np.abs(_f64(st[3]) * np.sqrt(np.float64(np.float32(1e-5))) - 1).max() <= 4 * U


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [1e3, -1e5])
@pytest.mark.parametrize("d", WIDTHS)
def test_rows_far_from_zero(d, offset, dtype):
    say(f"[block norm in front, offset {offset:g}] {dtype} {d}")
    rng = np.random.default_rng(d)
    n = 9
    x = _tensor(np.full((n, d), offset), dtype)
    z = _tensor(rng.standard_normal((n, d)) * 8.0, dtype)
    pre = dict(kind="layer", weight=_tensor(1 + 0.3 * rng.standard_normal(d), "f32"),
               bias=_tensor(rng.standard_normal(d), "f32"), eps=1e-5)
    scale = 1.25
    h, u, st = _run(x, z, dtype, scale, None, pre)
    r = S.block_norm(_f64(x), _f64(z), scale, None, None, _norm64(pre))
    m, rs = r["stats"][2][:, None], r["stats"][3][:, None]
    far = np.abs(r["h"]).max(axis=1, keepdims=True)
    away = np.abs(r["h"] - m)
    ediff = 5 * U * far + A * (away + away.mean(axis=1, keepdims=True))
    # of the variance: twice the mean of the differences times their error
    ers = rs * (A + rs ** 2 * ((2 * away * ediff).mean(axis=1, keepdims=True) + (ediff ** 2).max(axis=1, keepdims=True)))
    _check("mean", _f64(st[2]), r["stats"][2], (4 * U * far + A * away.mean(axis=1, keepdims=True))[:, 0])
    _check("rstd", _f64(st[3]), r["stats"][3], ers[:, 0])
    w, b = np.abs(_norm64(pre)["weight"]), np.abs(_norm64(pre)["bias"])
    tol = w * (ediff * rs + away * ers) * (1 + A) + A * b
    _check("u", _f64(u), r["u"], HALF[dtype] * (np.abs(r["u"]) + tol) + tol)
