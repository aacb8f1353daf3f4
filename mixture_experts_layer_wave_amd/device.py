"""Device-side holders of one MoE layer for the C ABI (marshalling only).

:class:`DeviceLayer` uploads the stored arrays of a layer (as produced by
:func:`mixture_experts_layer_wave_amd.workloads.make_layer`) to device
memory, sizes the workspace with ``moe_workspace_bytes`` and calls the
library's entry points.  :class:`TrainingLayer` adds the norm in front of the
layer, the buffers that a training step keeps, and the gradients.
:class:`DecodeBlock` serves a layer a few tokens at a time: experts encoded as
MXFP4, the norms around the layer, and an output projection.  torch provides
device memory and streams only.
"""

from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import binding as B


def to_device(a, device="cuda"):
    """numpy array -> device tensor with the same bytes (bf16 bits as int16)."""
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


def bf16_tensor_to_f64(t: torch.Tensor) -> np.ndarray:
    """int16 tensor of bf16 bit patterns -> float64 numpy (via torch's bf16)."""
    return t.view(torch.bfloat16).to(torch.float64).cpu().numpy()


class DeviceLayer:
    """One layer's inputs in HBM plus the output and workspace buffers."""

    def __init__(self, layer: dict, device: str = "cuda", renorm: int | None = None,
                 act_quant: str | None = None):
        self.layer = layer
        self.device = device
        self.n, self.d, self.E, self.k, self.d_ff = (layer[key] for key in ("n", "d", "E", "k", "d_ff"))
        self.act = layer["x_dtype"]
        self.wdt = layer["w_dtype"]
        rn = (1 if layer["renorm"] else 0) if renorm is None else renorm
        self.shape = B.Shape(self.n, self.d, self.E, self.k, self.d_ff, rn)
        self.x = to_device(layer["x"], device)
        self.wg = to_device(layer["wg"], device)
        self.bias = to_device(layer.get("bias"), device)
        self.w = {key: to_device(layer.get(key), device) for key in ("w1", "w3", "w2", "s1", "s3", "s2")}
        self.act_quant = act_quant
        self.weights = B.ExpertWeights(B.DTYPES[self.wdt], *(B._ptr(self.w[key]) for key in ("w1", "w3", "w2", "s1", "s3", "s2")),
                                       None, 0, B.DTYPES[act_quant] if act_quant else 0)
        self.ws_bytes = B.moe_workspace_bytes(self.shape, self.wdt)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        ydt = torch.int16 if self.act == "bf16" else torch.float32
        self.y = torch.empty((self.n, self.d), dtype=ydt, device=device)
        self.idx = torch.empty((self.n, self.k), dtype=torch.int32, device=device)
        self.topw = torch.empty((self.n, self.k), dtype=torch.float32, device=device)

    def forward(self, stream=None, out: str | None = None, y=None):
        B.moe_forward(self.shape, self.x, self.act, self.wg, self.bias, self.weights,
                      self.y if y is None else y, out or self.act, self.idx, self.topw,
                      self.ws, self.ws_bytes, stream)
        return self.y if y is None else y

    def y_f64(self, y=None) -> np.ndarray:
        y = self.y if y is None else y
        if y.dtype == torch.int16:
            return bf16_tensor_to_f64(y)
        return y.to(torch.float64).cpu().numpy()


class TrainingLayer(DeviceLayer):
    """A layer with a layer norm in front of it, for training:

        xn = norm(x),  y = layer(xn),  aux = alpha E sum_i f_i P_i

    :meth:`forward_train` keeps what the gradient needs; :meth:`backward`
    takes dy, the loss's gradient with respect to y, and fills ``grads``
    (x, norm_weight, norm_bias, wg, bias, w1, w3, w2; the gradient of aux
    included).  Neither allocates nor synchronises, so a step can be captured
    in a HIP graph.  bf16 or f32 weights.
    """

    def __init__(self, layer: dict, device: str = "cuda", renorm: int | None = None, alpha: float = 0.01,
                 eps: float = 1e-5):
        super().__init__(layer, device, renorm)
        n, d, E, k, f = self.n, self.d, self.E, self.k, self.d_ff
        R, adt = n * k, self.x.dtype
        self.alpha, self.eps = alpha, eps

        def empty(*shape, dtype=adt):
            return torch.empty(shape, dtype=dtype, device=device)

        f32, i32 = torch.float32, torch.int32
        self.norm_weight = torch.ones(d, dtype=f32, device=device)
        self.norm_bias = torch.zeros(d, dtype=f32, device=device)
        self.xn, self.mean, self.rstd = empty(n, d), empty(n, dtype=f32), empty(n, dtype=f32)
        self.logits = empty(n, E, dtype=f32)
        self.P, self.f, self.aux = empty(E, dtype=f32), empty(E, dtype=f32), empty(1, dtype=f32)
        self.counts, self.offsets = empty(E, dtype=i32), empty(E + 1, dtype=i32)
        self.perm, self.inv = empty(R, dtype=i32), empty(n, k, dtype=i32)
        self.h, self.g, self.u = empty(R, f), empty(R, f), empty(R, f)
        self.yp = empty(R, d, dtype=f32)
        self.da_perm, self.dtopk_w = empty(R, d), empty(n, k, dtype=f32)
        self.dlogits, self.dxn = empty(n, E, dtype=f32), empty(n, d)
        self.grads = dict(x=empty(n, d), norm_weight=empty(d, dtype=f32), norm_bias=empty(d, dtype=f32),
                          wg=empty(E, d), bias=empty(E, dtype=f32), w1=empty(E, f, d), w3=empty(E, f, d),
                          w2=empty(E, d, f))
        need = max(B.moe_layer_norm_backward_workspace_bytes(n, d), B.moe_router_backward_workspace_bytes(self.shape),
                   B.moe_grouped_ffn_backward_workspace_bytes(self.shape, self.wdt),
                   B.moe_router_stats_workspace_bytes(self.shape), B.moe_dispatch_workspace_bytes(self.shape))
        self.train_ws = torch.empty(need, dtype=torch.uint8, device=device)

    def forward_train(self, stream=None):
        s, ws, nb = self.shape, self.train_ws, self.train_ws.numel()
        B.moe_layer_norm(self.n, self.d, self.x, self.act, self.norm_weight, self.norm_bias, self.eps, self.xn,
                         self.mean, self.rstd, stream)
        B.moe_router_topk(s, self.xn, self.act, self.wg, self.bias, self.logits, self.idx, self.topw, stream)
        B.moe_router_stats(s, self.logits, self.idx, self.alpha, self.P, self.f, self.aux, ws, nb, stream)
        B.moe_dispatch(s, self.idx, self.counts, self.offsets, self.perm, self.inv, ws=ws, ws_bytes=nb,
                       stream=stream)
        B.moe_expert_up_save(s, self.xn, self.act, self.perm, self.offsets, self.weights, self.h, self.g, self.u,
                             stream)
        B.moe_expert_down(s, self.h, self.offsets, self.weights, self.yp, stream)
        B.moe_combine(s, self.yp, "f32", self.inv, self.topw, self.y, self.act, stream)
        return self.y

    def backward(self, dy, stream=None):
        s, ws, nb, gr = self.shape, self.train_ws, self.train_ws.numel(), self.grads
        B.moe_grouped_ffn_backward(s, dy, self.xn, self.act, self.perm, self.inv, self.topw, self.offsets,
                                   self.weights, self.g, self.u, self.da_perm, gr["w1"], gr["w3"], gr["w2"],
                                   self.dtopk_w, ws, nb, stream)
        B.moe_router_backward(s, self.logits, self.idx, self.topw, self.dtopk_w, self.f, self.alpha, self.xn,
                              self.act, self.wg, self.da_perm, self.inv, self.dlogits, self.dxn, gr["wg"],
                              gr["bias"], ws, nb, stream)
        B.moe_layer_norm_backward(self.n, self.d, self.dxn, self.x, self.act, self.norm_weight, self.mean,
                                  self.rstd, gr["x"], gr["norm_weight"], gr["norm_bias"], ws, nb, stream)
        return gr


def encode_mxfp4(w, stream=None):
    """(codes, scales) of a device tensor [..., cols] of bf16 or float32, of any
    strides, in MXFP4, by moe_quantize_mxfp4.  Everything runs on ``stream``
    (the current one by default), the copy of a tensor that is not contiguous
    included."""
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"encode_mxfp4 takes bfloat16 or float32 tensors, not {w.dtype}")
    if not w.is_cuda or w.dim() == 0 or w.shape[-1] == 0:
        raise ValueError(f"encode_mxfp4 takes device tensors [..., cols], not {w.device} {list(w.shape)}")
    if stream is None:
        on = contextlib.nullcontext()
    else:
        on = torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream))
    with on:
        if w.device.index != torch.cuda.current_device():
            raise ValueError(f"encode_mxfp4: a tensor on {w.device}, a stream on cuda:{torch.cuda.current_device()}")
        # (memory of this stream, so that it is free for others only behind the encoder)
        w = w.contiguous()
        cols = w.shape[-1]
        q = torch.empty((*w.shape[:-1], cols // 2), dtype=torch.uint8, device=w.device)
        s = torch.empty((*w.shape[:-1], cols // 32), dtype=torch.uint8, device=w.device)
        B.moe_quantize_mxfp4(w.numel() // cols, cols, w, "f32" if w.dtype == torch.float32 else "bf16", q, s)
    return q, s


def _expect(name, t, shape, dtypes, device, contiguous=True):
    """Raises unless t is a tensor of this shape, of one of these types, there."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} is {list(t.shape)}, not {list(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, not {' or '.join(map(str, dtypes))}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")


class DecodeBlock:
    """A layer with the norms around it, for at most 16 tokens a step:

        z = layer(u),  h <- scale h + gate * post(z),  u <- pre(h),  logits = u head^T

    with the experts and the head in MXFP4.  ``w1``, ``w3`` [E][d_ff][d], ``w2``
    [E][d][d_ff] and ``head`` [m][d] (or None) are bf16 or float32 device
    tensors, encoded once; ``wg`` [E][d] is bf16, ``bias`` [E] and ``gate`` [d]
    float32 or None.  ``post`` and ``pre`` are dicts (kind "layer" or "rms",
    weight, bias, eps; [d] float32) or None.  ValueError for any other shape,
    type or device, and for parameters used as they are (not encoded) that are
    not contiguous.  Without ``pre`` u is h itself.  :meth:`step` works on the
    block's own h and u [n][d] in place, returns the logits or, without a head,
    u, and neither allocates nor synchronises, so it can be captured in a HIP
    graph.
    """

    def __init__(self, n, wg, w1, w3, w2, k, bias=None, scale=1.0, gate=None, post=None, pre=None, head=None,
                 renorm=-1):
        if w1.dim() != 3:
            raise ValueError(f"w1 is {list(w1.shape)}, not [E, d_ff, d]")
        E, d_ff, d = w1.shape
        dev = w1.device
        f32, stored = (torch.float32,), (torch.bfloat16, torch.float32)
        _expect("w1", w1, (E, d_ff, d), stored, dev, False)
        _expect("w3", w3, (E, d_ff, d), stored, dev, False)
        _expect("w2", w2, (E, d, d_ff), stored, dev, False)
        if head is not None:
            _expect("head", head, (head.shape[0] if head.dim() else 0, d), stored, dev, False)
        _expect("wg", wg, (E, d), (torch.bfloat16,), dev)
        vectors = [("bias", bias, E), ("gate", gate, d)]
        for side, norm in (("post", post), ("pre", pre)):
            if isinstance(norm, dict):
                if norm["kind"] not in (*B.NORMS, *B.NORMS.values()):
                    raise ValueError(f"{side}: no norm {norm['kind']!r}")
                _expect(side + " weight", norm["weight"], (d,), f32, dev)
                vectors.append((side + " bias", norm.get("bias"), d))
        for name, v, size in vectors:
            if v is not None:
                _expect(name, v, (size,), f32, dev)
        self.n, self.d, self.wg, self.bias = n, d, wg, bias
        self.shape = B.Shape(n, d, E, k, d_ff, renorm)
        self.scale, self.gate, self.post, self.pre = scale, gate, post, pre
        self.experts = dict(dtype="mxfp4")
        for key, w in (("1", w1), ("3", w3), ("2", w2)):
            self.experts["w" + key], self.experts["s" + key] = encode_mxfp4(w)
        self.weights = B._weights(self.experts)

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=dev)

        self.h, self.z = empty(n, d), empty(n, d)
        self.u = empty(n, d) if pre else self.h
        self.idx, self.topw = empty(n, k, dtype=torch.int32), empty(n, k, dtype=torch.float32)
        # moe_forward_few or moe_forward, us: 128 experts 2880 x 2880, top-4, 1 token 29 and 32,
        # 4 tokens 61 and 65, 8 tokens 98 and 95, 16 tokens 170 and 145; 8 experts 1024 x 4096,
        # top-2, 4 tokens 29 and 32, 8 tokens 35 and 35, 16 tokens 44 and 37.  Rows past 7168
        # elements do not fit moe_forward's kernels with the codes in LDS: 8 experts 4096 wide,
        # top-2, d_ff = 7168, 16 tokens 170 and 141, 7200 175 and 195, 14336 306 and 337 (8
        # tokens: 77 and 141, 87 and 194, 143 and 334).
        few = n <= 4 or (n <= B.MOE_FEW_MAX_TOKENS and max(d, d_ff) > 7168)
        self.layer, size = ((B.moe_forward_few, B.moe_forward_few_workspace_bytes) if few else
                            (B.moe_forward, B.moe_workspace_bytes))
        need = size(self.shape, "mxfp4")
        self.head = None
        if head is not None:
            self.head, self.m = encode_mxfp4(head), head.shape[0]
            self.logits = empty(n, self.m, dtype=torch.float32)
            need = max(need, B.moe_mxfp4_linear_workspace_bytes(n, d, self.m, "bf16"))
        self.ws = empty(max(need, 16), dtype=torch.uint8)

    def step(self, stream=None):
        nb = self.ws.numel()
        u = self.u if self.pre else self.h
        self.layer(self.shape, u, "bf16", self.wg, self.bias, self.weights, self.z, "bf16", self.idx,
                   self.topw, self.ws, nb, stream)
        B.moe_block_norm(self.n, self.d, self.h, self.z, "bf16", self.scale, self.gate, self.post, self.pre,
                         self.h, u if self.pre else None, None, stream)
        if self.head:
            B.moe_mxfp4_linear(self.n, self.d, self.m, u, None, "bf16", *self.head, None, self.logits, "f32", self.ws,
                               nb, stream)
        return self.logits if self.head else u
