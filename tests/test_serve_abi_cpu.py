"""Host-side checks of the MXFP4, few-token and block-norm entry points: sizes
and refusals, all before anything is launched (no GPU needed)."""

import ctypes

import pytest

from mixture_experts_layer_wave_amd import binding as B

FAKE = 1 << 20  # never dereferenced: every call below fails before a launch
F32, BF16, MXFP4, MXFP8 = 0, 1, 2, 3


def _codec(fn, rows=4, cols=64, dtype=BF16, **kw):
    v = dict(x=FAKE, q=FAKE, s=FAKE)
    v.update(kw)
    if fn == "quantize":
        return B.lib.moe_quantize_mxfp4(rows, cols, v["x"], dtype, v["q"], v["s"], None)
    return B.lib.moe_dequantize_mxfp4(rows, cols, v["q"], v["s"], v["x"], dtype, None)


@pytest.mark.parametrize("fn", ["quantize", "dequantize"])
def test_codec_refusals(fn):
    assert _codec(fn, rows=-1) == -2 and _codec(fn, rows=1 << 31) == -2
    assert _codec(fn, cols=0) == -2 and _codec(fn, cols=-32) == -2 and _codec(fn, cols=48) == -2
    assert _codec(fn, dtype=MXFP4) == -3 and _codec(fn, dtype=MXFP8) == -3
    for name in ("x", "q", "s"):
        assert _codec(fn, **{name: None}) == -1, name
        assert _codec(fn, **{name: FAKE + 8}) == -4, name
    assert _codec(fn, rows=0, x=None, q=None, s=None) == 0  # nothing to do


def _linear(n=4, d=64, m=10, act=BF16, out=BF16, nb=1 << 40, **kw):
    v = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, bias=FAKE, y=FAKE, work=FAKE)
    v.update(kw)
    return B.lib.moe_mxfp4_linear(n, d, m, v["x"], v["xs"], act, v["w"], v["ws"], v["bias"], v["y"], out,
                                  v["work"], nb, None)


def test_linear_refusals():
    assert _linear(n=-1) == -2 and _linear(d=0) == -2 and _linear(d=48) == -2 and _linear(m=0) == -2
    assert _linear(n=1 << 20, d=1024) == -2 and _linear(n=1 << 20, m=1024) == -2
    assert _linear(d=1 << 15, m=1 << 15) == -2
    assert _linear(act=F32) == -3 and _linear(act=MXFP8) == -3
    assert _linear(out=MXFP4) == -3 and _linear(out=MXFP8) == -3
    for name in ("x", "w", "ws", "y"):
        assert _linear(**{name: None}) == -1, name
        assert _linear(**{name: FAKE + 8}) == -4, name
    assert _linear(act=MXFP4, xs=None) == -1 and _linear(act=MXFP4, xs=FAKE + 4) == -4
    assert _linear(n=0, x=None, w=None, ws=None, y=None) == 0
    for n, d, m, act in ((1, 64, 10, "bf16"), (333, 2880, 5001, "bf16"), (8192, 4096, 14336, "bf16"),
                         (8192, 4096, 14336, "mxfp4")):
        need = B.moe_mxfp4_linear_workspace_bytes(n, d, m, act)
        assert need % 256 == 0
        if need:
            assert _linear(n=n, d=d, m=m, act=B.DTYPES[act], nb=need - 1) == -5
            assert _linear(n=n, d=d, m=m, act=B.DTYPES[act], work=None) == -5
            assert _linear(n=n, d=d, m=m, act=B.DTYPES[act], work=FAKE + 4) == -4
    assert B.moe_mxfp4_linear_workspace_bytes(4, 48, 10, "bf16") == 0
    assert B.moe_mxfp4_linear_workspace_bytes(4, 64, 10, "f32") == 0
    assert B.moe_mxfp4_linear_workspace_bytes(0, 64, 10, "bf16") == 0


def _weights(dtype=BF16, **kw):
    fields = dict(dtype=dtype, w1=FAKE, w3=FAKE, w2=FAKE)
    if dtype == MXFP4:
        fields.update(s1=FAKE, s3=FAKE, s2=FAKE)
    fields.update(kw)
    return B.ExpertWeights(**fields)


def _few(shape=(4, 64, 4, 2, 64), act=BF16, out=BF16, w=None, nb=1 << 40, **kw):
    sp = None if shape is None else ctypes.byref(B._shape(shape))
    w = _weights(act) if w is None else w
    v = dict(x=FAKE, wg=FAKE, bias=FAKE, y=FAKE, idx=FAKE, tw=FAKE, ws=FAKE)
    v.update(kw)
    return B.lib.moe_forward_few(sp, v["x"], act, v["wg"], v["bias"], ctypes.byref(w), v["y"], out, v["idx"],
                                 v["tw"], v["ws"], nb, None)


def test_forward_few_refusals():
    assert _few(shape=None) == -1
    assert _few(shape=(0, 64, 4, 2, 64)) == -2 and _few(shape=(17, 64, 4, 2, 64)) == -2
    assert _few(shape=(4, 64, 4, 5, 64)) == -2 and _few(shape=(4, 64, 1025, 2, 64)) == -2
    assert _few(shape=(4, 60, 4, 2, 64)) == -2 and _few(shape=(4, 64, 4, 2, 60)) == -2
    assert _few(w=_weights(MXFP4), shape=(4, 80, 4, 2, 64)) == -2
    assert _few(w=_weights(F32), act=F32, shape=(16, 64, 64, 32, 1 << 21)) == -2
    assert _few(act=MXFP8) == -3 and _few(act=F32, w=_weights(BF16)) == -3 and _few(w=_weights(F32)) == -3
    assert _few(w=_weights(MXFP4, act_quant=MXFP8), shape=(4, 128, 4, 2, 128)) == -3
    assert _few(out=MXFP4) == -3
    for name in ("x", "wg", "y"):
        assert _few(**{name: None}) == -1, name
        assert _few(**{name: FAKE + 8}) == -4, name
    for name in ("w1", "w3", "w2"):
        assert _few(w=_weights(BF16, **{name: None})) == -1, name
        assert _few(w=_weights(BF16, **{name: FAKE + 8})) == -4, name
    for name in ("s1", "s3", "s2"):
        assert _few(w=_weights(MXFP4, **{name: None})) == -1, name
    assert _few(w=_weights(BF16, slot=FAKE, n_slots=0)) == -2
    shape = (4, 64, 4, 2, 64)
    for dt in ("f32", "bf16", "mxfp4"):
        need = B.moe_forward_few_workspace_bytes(shape, dt)
        assert need % 256 == 0 and need >= 4 * 4 * 4 + 8 * 64 * (4 if dt == "f32" else 2)
        act = F32 if dt == "f32" else BF16
        assert _few(act=act, w=_weights(B.DTYPES[dt]), nb=need - 1) == -5
    assert _few(ws=None) == -5 and _few(ws=FAKE + 4) == -4
    assert B.moe_forward_few_workspace_bytes((17, 64, 4, 2, 64), "bf16") == 0
    assert B.moe_forward_few_workspace_bytes(shape, "mxfp8") == 0


def _ref(kind=0, eps=1e-5, w=FAKE, b=FAKE):
    return B.Norm(kind, eps, w, b)


def _norms(n=4, d=64, act=BF16, post=_ref(), pre=_ref(1), **kw):
    v = dict(x=FAKE, z=FAKE, gate=FAKE, h=FAKE, u=FAKE, stats=FAKE)
    v.update(kw)
    return B.lib.moe_block_norm(n, d, v["x"], v["z"], act, 1.0, v["gate"], B._norm(post), B._norm(pre), v["h"],
                                v["u"], v["stats"], None)


def test_block_norm_refusals():
    assert _norms(n=-1) == -2 and _norms(n=1 << 30) == -2
    assert _norms(d=0) == -2 and _norms(d=16392) == -2 and _norms(d=60) == -2
    assert _norms(act=MXFP4) == -3
    for side in ("post", "pre"):
        assert _norms(**{side: _ref(kind=2)}) == -3 and _norms(**{side: _ref(kind=-1)}) == -3
        assert _norms(**{side: _ref(eps=-1.0)}) == -2 and _norms(**{side: _ref(eps=float("nan"))}) == -2
        assert _norms(**{side: _ref(w=None)}) == -1
    for name in ("x", "z", "h", "u"):
        assert _norms(**{name: None}) == -1, name
        assert _norms(**{name: FAKE + 8}) == -4, name
    assert _norms(n=0, x=None, z=None, h=None, u=None) == 0


def _back(n=4, d=64, act=BF16, post=_ref(), pre=_ref(1), nb=1 << 40, **kw):
    v = dict(dh=FAKE, du=FAKE, z=FAKE, h=FAKE, gate=FAKE, stats=FAKE, dx=FAKE, dz=FAKE, dgate=FAKE, dpw=FAKE,
             dpb=FAKE, dqw=FAKE, dqb=FAKE, ws=FAKE)
    v.update(kw)
    return B.lib.moe_block_norm_backward(n, d, v["dh"], v["du"], v["z"], v["h"], act, 1.0, v["gate"],
                                         B._norm(post), B._norm(pre), v["stats"], v["dx"], v["dz"], v["dgate"],
                                         v["dpw"], v["dpb"], v["dqw"], v["dqb"], v["ws"], nb, None)


def test_block_norm_backward_refusals():
    assert _back(n=-1) == -2 and _back(d=0) == -2 and _back(d=60) == -2 and _back(act=MXFP4) == -3
    for side in ("post", "pre"):
        assert _back(**{side: _ref(kind=5)}) == -3 and _back(**{side: _ref(w=None)}) == -1
    for name in ("du", "z", "h", "stats", "dx", "dz"):
        assert _back(**{name: None}) == -1, name
    for name in ("dh", "du", "z", "h", "dx", "dz"):
        assert _back(**{name: FAKE + 8}) == -4, name
    # gradients of what the call does not have
    assert _back(gate=None) == -1
    assert _back(post=None) == -1 and _back(post=None, dpw=None) == -1
    assert _back(pre=None) == -1 and _back(pre=None, dqw=None) == -1
    # without a norm in front, the gradient comes through dh
    assert _back(pre=None, dqw=None, dqb=None, dh=None) == -1
    need = B.moe_block_norm_backward_workspace_bytes(4, 64)
    assert need >= 4 * 4 * 64 * 4 and need % 256 == 0
    assert _back(nb=need - 1) == -5 and _back(ws=None) == -5 and _back(ws=FAKE + 4) == -4
    assert B.moe_block_norm_backward_workspace_bytes(0, 64) == 0
    assert B.moe_block_norm_backward_workspace_bytes(4, 16385) == 0
    with pytest.raises(B.MoeError) as ei:
        B.moe_block_norm(4, 0, FAKE, FAKE, "bf16", 1.0, None, None, dict(kind="rms", weight=FAKE), FAKE, FAKE,
                         stream=0)
    assert ei.value.status == -2
