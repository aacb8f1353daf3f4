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


def _weights(dtype=BF16, **kw):
    fields = dict(dtype=dtype, w1=FAKE, w3=FAKE, w2=FAKE)
    fields.update(kw)
    return B.ExpertWeights(**fields)


def _up(shape=(4, 64, 4, 2, 64), a=FAKE, act=BF16, off=FAKE, w=None, h=FAKE, g=FAKE, u=FAKE):
    sp = None if shape is None else ctypes.byref(B._shape(shape))
    w = _weights(act) if w is None else w
    return B.lib.moe_expert_up_save(sp, a, act, FAKE, off, ctypes.byref(w), h, g, u, None)


def _back(shape=(4, 64, 4, 2, 64), act=BF16, w=None, nb=1 << 40, **kw):
    sp = None if shape is None else ctypes.byref(B._shape(shape))
    w = _weights(act) if w is None else w
    v = dict(dy=FAKE, a=FAKE, perm=FAKE, inv=FAKE, tw=FAKE, off=FAKE, g=FAKE, u=FAKE, da=FAKE, dw1=FAKE,
             dw3=FAKE, dw2=FAKE, dtw=FAKE, ws=FAKE)
    v.update(kw)
    return B.lib.moe_grouped_ffn_backward(
        sp, v["dy"], v["a"], act, v["perm"], v["inv"], v["tw"], v["off"], ctypes.byref(w), v["g"], v["u"],
        v["da"], v["dw1"], v["dw3"], v["dw2"], v["dtw"], v["ws"], nb, None)


@pytest.mark.parametrize("call", [_up, _back])
def test_ffn_training_refuses_shapes_and_types(call):
    assert call(shape=None) == -1
    assert call(shape=(0, 64, 4, 2, 64)) == -2
    assert call(shape=(4, 64, 4, 5, 64)) == -2
    assert call(shape=(4, 60, 4, 2, 64)) == -2 and call(shape=(4, 64, 4, 2, 60)) == -2
    assert call(shape=(4, 1 << 20, 4, 2, 64)) == -2 and call(shape=(4, 64, 4, 2, 1 << 20), act=F32) == -2
    # bf16 operands are addressed with 32-bit offsets, as in the forward pass
    assert call(shape=(65536, 4096, 8, 2, 14336)) == -2
    assert call(shape=(32768, 4096, 8, 2, 8192), act=F32) == -2 and call(shape=(4, 32768, 4, 2, 16384), act=F32) == -2
    assert call(act=MXFP8) == -3 and call(act=MXFP4) == -3
    assert call(act=F32, w=_weights(BF16)) == -3 and call(act=BF16, w=_weights(F32)) == -3
    # MXFP4 weights are not trained
    assert call(w=_weights(MXFP4, s1=FAKE, s3=FAKE, s2=FAKE)) == -3
    assert call(w=_weights(BF16, act_quant=MXFP8)) == -3
    assert call(w=_weights(BF16, w1=None)) == -1 and call(w=_weights(BF16, w2=FAKE + 8)) == -4
    assert call(w=_weights(BF16, slot=FAKE, n_slots=0)) == -2


def test_up_save_refuses_pointers():
    for name in ("a", "off", "h", "g", "u"):
        assert _up(**{name: None}) == -1, name
    for name in ("a", "h", "g", "u"):
        assert _up(**{name: FAKE + 8}) == -4, name


def test_ffn_backward_refuses_pointers_and_workspaces():
    names = ("dy", "a", "off", "g", "u", "da", "dw1", "dw3", "dw2")
    for name in names + ("perm", "inv", "tw", "dtw"):  # the last four are given together
        assert _back(**{name: None}) == -1, name
    for name in set(names) - {"off"}:
        assert _back(**{name: FAKE + 8}) == -4, name
    shape = (4, 64, 4, 2, 64)
    for dt in ("bf16", "f32"):
        need = B.moe_grouped_ffn_backward_workspace_bytes(shape, dt)
        assert need % 256 == 0 and need >= 3 * 8 * 64 * (2 if dt == "bf16" else 4)
        assert _back(act=B.DTYPES[dt], nb=need - 1) == -5
    assert _back(ws=None) == -5 and _back(ws=FAKE + 4) == -4
    assert B.moe_grouped_ffn_backward_workspace_bytes(shape, "mxfp4") == 0
    assert B.moe_grouped_ffn_backward_workspace_bytes((4, 60, 4, 2, 64), "bf16") == 0
    assert B.moe_grouped_ffn_backward_workspace_bytes((0, 64, 4, 2, 64), "f32") == 0


def _router(shape=(4, 64, 4, 2, 64), act=BF16, nb=1 << 40, **kw):
    sp = None if shape is None else ctypes.byref(B._shape(shape))
    v = dict(z=FAKE, idx=FAKE, w=FAKE, dw=FAKE, f=FAKE, x=FAKE, wg=FAKE, da=FAKE, inv=FAKE, dz=FAKE, dx=FAKE,
             dwg=FAKE, db=FAKE, ws=FAKE)
    v.update(kw)
    return B.lib.moe_router_backward(sp, v["z"], v["idx"], v["w"], v["dw"], v["f"], 0.01, v["x"], act, v["wg"],
                                     v["da"], v["inv"], v["dz"], v["dx"], v["dwg"], v["db"], v["ws"], nb, None)


def test_router_backward_refusals():
    assert _router(shape=None) == -1
    assert _router(shape=(4, 64, 4, 5, 64)) == -2 and _router(shape=(1 << 24, 64, 4, 1, 64)) == -2
    assert _router(shape=(4, 1 << 19, 1024, 2, 64)) == -2
    assert _router(shape=(4, 1 << 20, 4, 2, 64)) == -2 and _router(shape=(4, 60, 4, 2, 64)) == -2
    assert _router(act=MXFP4) == -3 and _router(act=MXFP8) == -3
    for name in ("z", "idx", "w", "dw", "x", "wg", "dz", "dx", "dwg", "da", "inv"):
        assert _router(**{name: None}) == -1, name  # da_perm and inv are given together
    for name in ("x", "wg", "da", "dx", "dwg"):
        assert _router(**{name: FAKE + 8}) == -4, name
    shape = (4, 64, 4, 2, 64)
    need = B.moe_router_backward_workspace_bytes(shape)
    assert need % 256 == 0 and need >= 4 * (64 + 1) * 4
    assert _router(nb=need - 1) == -5 and _router(ws=None) == -5 and _router(ws=FAKE + 4) == -4
    assert B.moe_router_backward_workspace_bytes((0, 64, 4, 2, 64)) == 0
    # the partial planes of W_g's gradient stay within the bytes of x; two
    # bf16 halves of dlogits, 32 experts wide at least, follow them
    for n, d, E in ((8192, 4096, 8), (4096, 2880, 128), (65536, 256, 64)):
        most = max(n * 2, 4 * E) * (d + 1) + 4 * n * -(-E // 32) * 32 + 512
        assert B.moe_router_backward_workspace_bytes((n, d, E, 1, 8)) <= most
