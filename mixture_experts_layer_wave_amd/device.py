"""Device-side holders of one MoE layer for the C ABI (marshalling only).

:class:`DeviceLayer` uploads the stored arrays of a layer (as produced by
:func:`mixture_experts_layer_wave_amd.workloads.make_layer`) to device
memory, sizes the workspace with ``moe_workspace_bytes`` and calls the
library's entry points.  :class:`TrainingLayer` adds the norm in front of the
layer, the buffers that a training step keeps, and the gradients.  torch
provides device memory and streams only.
"""

from __future__ import annotations

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
