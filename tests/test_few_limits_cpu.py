"""The widths that moe_forward_few takes, on the host alone.

A wave's loads reach the eight rows of a group of weights by 32-bit byte offsets
from the group's first row.  In bf16 and MXFP4 one matrix has less than 2^30
elements, so seven rows of it stay below 2^31 bytes.  float32 matrices have no
such limit, so rows are limited to 2^26 - 1 elements: 8 * 4 * (2^26 - 1) < 2^31.
Every call here is refused before anything is launched: past the limit for its
shape, below it for its workspace."""

import ctypes

import pytest

from mixture_experts_layer_wave_amd import binding as B

FAKE = 1 << 20  # never dereferenced
WIDE = 1 << 26


def _call(shape, dt):
    w = B.ExpertWeights(dtype=B.DTYPES[dt], w1=FAKE, w3=FAKE, w2=FAKE, s1=FAKE, s3=FAKE, s2=FAKE)
    act = B.MOE_F32 if dt == "f32" else B.MOE_BF16
    return B.lib.moe_forward_few(ctypes.byref(B._shape(shape)), FAKE, act, FAKE, None, ctypes.byref(w), FAKE, act, None,
                                 None, FAKE, 0, None)


@pytest.mark.parametrize("d,f", [(WIDE, 8), (WIDE + 4, 1), (160_000_000, 8), (1 << 29, 1), ((1 << 31) - 1, 1), (8, WIDE),
                                 (1, WIDE + 1), (8, 160_000_000), (WIDE, WIDE)])
def test_float32_rows_past_32_bit_offsets_are_refused(d, f):
    shape = (1, d, 1, 1, f)
    assert _call(shape, "f32") == -2
    assert B.moe_forward_few_workspace_bytes(shape, "f32") == 0


@pytest.mark.parametrize("d,f", [(WIDE - 1, 8), (WIDE - 4, 1), (8, WIDE - 1), (WIDE - 1, WIDE - 1)])
def test_float32_rows_below_are_taken(d, f):
    shape = (1, d, 1, 1, f)
    need = B.moe_forward_few_workspace_bytes(shape, "f32")
    assert need >= 4 * f and _call(shape, "f32") == -5  # (no workspace given)


@pytest.mark.parametrize("dt,least", [("bf16", 8), ("mxfp4", 32)])
def test_stored_forms_are_limited_by_the_matrix(dt, least):
    """The widest rows that a matrix below 2^30 elements has keep the offsets in 31 bits."""
    most = (1 << 30) // least
    assert _call((1, most, 1, 1, least), dt) == -2
    assert _call((1, most - least, 1, 1, least), dt) == -5
    assert 7 * (most - least) * 2 < 1 << 31
