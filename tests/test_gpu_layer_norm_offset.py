"""moe_layer_norm of float32 rows far from zero.

Tolerances (derived, not measured); U = 2^-24.  The mean of a row is known to
float32's last bit and what that bit leaves: off by 2^-53 and 64 U of the rest.
The differences x - mean (the float32 mean first: exact, as the two lie within a
factor of two of each other, then the rest) are off by 2 U of themselves and of
the rest, which is U of the offset at most: y and rstd are good to 64 U (a sum
of under 40 additions, and a few roundings) of the *spread* of the row, with a
second-order term in the offset; the mean is rounded once to its own type (U of
it).

Rows of one value: a float64 sum of 2^14 values of 24 bits is exact, so mean =
the value, the rest is 0, and so are the differences: rstd = 1 / sqrt(eps) and
y = bias."""

import numpy as np
import pytest

import oracle
from tests.gpu_support import say
from tests.test_gpu_layer_norm import HALF, U, _check, _f64, _forward, _tensor

pytestmark = pytest.mark.gpu

WIDTHS = [1, 2, 3, 17, 37, 64, 255, 257, 1000, 1021, 2047, 2049, 4096, 5001, 8193, 16383, 16384]


@pytest.mark.parametrize("d", WIDTHS)
def test_rows_of_one_value(d):
    import torch

    say(f"[layer norm, equal values] f32 {d}")
    rng = np.random.default_rng(d)
    values = np.concatenate([[1000.1, 1e5 + 0.1, -7.3, 1 / 3, 3e-3, 1e30, -1e-20, 0.0], rng.uniform(1, 1000, 200)])
    x = _tensor(np.repeat(values[:, None], d, axis=1), "f32")
    w, b = _tensor(1 + 0.3 * rng.standard_normal(d), "f32"), _tensor(rng.standard_normal(d), "f32")
    y, mean, rstd = _forward(x, "f32", w, b)
    assert torch.equal(mean, x[:, 0])
    assert np.abs(_f64(rstd) * np.sqrt(np.float64(np.float32(1e-5))) - 1).max() <= 4 * U
    assert torch.equal(y, b.expand_as(y))


@pytest.mark.parametrize("offset", [1e3, -1e5])
@pytest.mark.parametrize("d", [d for d in WIDTHS if d >= 17])
def test_rows_far_from_zero(d, offset):
    say(f"[layer norm, offset {offset:g}] f32 {d}")
    rng = np.random.default_rng(d)
    x = _tensor(offset + rng.standard_normal((9, d)), "f32")
    w, b = _tensor(1 + 0.3 * rng.standard_normal(d), "f32"), _tensor(rng.standard_normal(d), "f32")
    y, mean, rstd = _forward(x, "f32", w, b)
    x64, w64, b64 = _f64(x), _f64(w), _f64(b)
    ref, m, r = oracle.layer_norm(x64, w64, b64, float(np.float32(1e-5)))
    away = np.abs(x64 - m[:, None])
    spread = away + away.mean(axis=1, keepdims=True) + 41 * U * abs(offset)
    _check("mean", _f64(mean), m, U * np.abs(m) + 64 * U * spread.mean(axis=1))
    _check("rstd", _f64(rstd), r, 64 * U * r)
    _check("y", _f64(y), ref, HALF["f32"] * np.abs(ref) + 64 * U * (spread * r[:, None] * np.abs(w64) + np.abs(b64)))
