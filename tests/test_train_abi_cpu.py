"""Host-side checks of the training entry points: sizes and refusals, all
before anything is launched (no GPU needed)."""

import ctypes

import pytest

from mixture_experts_layer_wave_amd import binding as B

FAKE = 1 << 20  # never dereferenced: every call below fails before a launch
F32, BF16, MXFP4, MXFP8 = 0, 1, 2, 3


def _norm(n=4, d=64, x=FAKE, act=BF16, w=FAKE, b=FAKE, eps=1e-5, y=FAKE):
    return B.lib.moe_layer_norm(n, d, x, act, w, b, eps, y, FAKE, FAKE, None)


def test_layer_norm_refusals():
    assert _norm(n=-1) == -2 and _norm(n=1 << 30) == -2
    assert _norm(d=0) == -2 and _norm(d=16392) == -2 and _norm(d=16392, act=F32) == -2
    assert _norm(d=60) == -2            # bf16 rows are multiples of 8 wide
    assert _norm(act=MXFP4) == -3 and _norm(act=MXFP8) == -3
    assert _norm(eps=-1e-5) == -2 and _norm(eps=float("nan")) == -2
    assert _norm(x=None) == -1 and _norm(w=None) == -1 and _norm(y=None) == -1
    assert _norm(x=FAKE + 8) == -4 and _norm(y=FAKE + 2) == -4
    assert _norm(n=0, x=None, y=None, w=None) == 0  # nothing to do


def _norm_grad(n=4, d=64, dy=FAKE, x=FAKE, act=BF16, w=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, ws=FAKE, nb=None):
    nb = B.moe_layer_norm_backward_workspace_bytes(n, d) if nb is None else nb
    return B.lib.moe_layer_norm_backward(n, d, dy, x, act, w, mean, rstd, dx, FAKE, FAKE, ws, nb, None)


def test_layer_norm_backward_refusals():
    assert _norm_grad(n=-1) == -2 and _norm_grad(d=0) == -2 and _norm_grad(d=60) == -2
    assert _norm_grad(act=MXFP4) == -3
    for name in ("dy", "x", "w", "mean", "rstd", "dx"):
        assert _norm_grad(**{name: None}) == -1, name
    for name in ("dy", "x", "dx"):
        assert _norm_grad(**{name: FAKE + 8}) == -4, name
    assert _norm_grad(ws=None) == -5 and _norm_grad(ws=FAKE + 4) == -4
    need = B.moe_layer_norm_backward_workspace_bytes(4, 64)
    assert need >= 4 * 2 * 64 * 4 and need % 256 == 0
    assert _norm_grad(nb=need - 1) == -5
    # at most one partial row per compute unit
    assert B.moe_layer_norm_backward_workspace_bytes(100000, 64) == 256 * 2 * 64 * 4
    assert B.moe_layer_norm_backward_workspace_bytes(-1, 64) == 0
    assert B.moe_layer_norm_backward_workspace_bytes(0, 64) == 0
    assert B.moe_layer_norm_backward_workspace_bytes(4, 16385) == 0
    with pytest.raises(B.MoeError) as ei:
        B.moe_layer_norm_backward(4, 0, FAKE, FAKE, "bf16", FAKE, FAKE, FAKE, FAKE, None, None, FAKE, 0,
                                  stream=0)
    assert ei.value.status == -2
