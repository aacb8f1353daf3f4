"""The gradient through both norms and a trained layer, for every parameter.

h, u = norms(x0, z0); y = layer(u); h2 = h + norm(y), float32, and a weighted sum
of h2 for a loss.  A difference quotient needs the same experts on both sides:
the router's bias is a ladder of steps of 6, wider than what the tokens add (their
logits spread by about 1), so that no step of 2^-9 changes a choice, and every
comparison is asserted to be made.

Tolerance: eps^2 of the curvature, and float32 rounding of about 1000 terms over
eps: 1e-2 of the value and 5e-2."""

import numpy as np
import pytest

from tests.gpu_support import say
from tests.test_gpu_decode_block import _norm

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -9


def test_gradient_of_every_parameter():
    import torch
    from mixture_experts_layer_wave_amd import binding as B
    from mixture_experts_layer_wave_amd import workloads as W
    from mixture_experts_layer_wave_amd.device import TrainingLayer

    wl = W.Workload("around", 24, 40, 4, 2, 56, "f32", "f32", 91, 92)
    layer = W.make_layer(wl, use_fixture=False, cache=False)
    layer["bias"] = np.array([0.0, 12.0, 6.0, 18.0], np.float32)
    L = TrainingLayer(layer, alpha=0.0)
    n, d = L.n, L.d
    rng = np.random.default_rng(8)
    vec = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()
    x0, z0, r = vec(n, d), vec(n, d), vec(n, d)
    gate = 1 + 0.1 * vec(d)
    n1, n2, n3 = _norm(rng, d, "rms"), _norm(rng, d, "rms"), _norm(rng, d, "layer")
    h, h2 = torch.empty_like(x0), torch.empty_like(x0)
    s1, s2 = torch.empty((4, n), device="cuda"), torch.empty((4, n), device="cuda")

    def forward():
        B.moe_block_norm(n, d, x0, z0, "f32", 1.0, gate, n1, n2, h, L.x, s1)
        y = L.forward_train()
        B.moe_block_norm(n, d, h, y, "f32", 0.5, None, n3, None, h2, None, s2)
        return float((h2.double() * r.double()).sum())

    forward()
    e = lambda: torch.empty_like(x0)
    dh, dy, dx, dz = e(), e(), e(), e()
    p = [torch.empty(d, device="cuda") for _ in range(5)]
    nb = B.moe_block_norm_backward_workspace_bytes(n, d)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    B.moe_block_norm_backward(n, d, r, None, L.y, h2, "f32", 0.5, None, n3, None, s2, dh, dy, None, p[0], p[1], None,
                              None, ws, nb)
    g = {key: v.clone() for key, v in L.backward(dy).items()}
    B.moe_block_norm_backward(n, d, dh, g["x"], z0, h, "f32", 1.0, gate, n1, n2, s1, dx, dz, p[2], p[3], None, p[4],
                              None, ws, nb)
    torch.cuda.synchronize()
    idx = L.idx.clone()
    assert torch.equal(idx, torch.tensor([3, 1], dtype=torch.int32, device="cuda").expand(n, 2))
    leaves = dict(x=(x0, dx), z=(z0, dz), gate=(gate, p[2]), post=(n1["weight"], p[3]), pre=(n2["weight"], p[4]),
                  last_weight=(n3["weight"], p[0]), last_bias=(n3["bias"], p[1]), norm_weight=(L.norm_weight, g["norm_weight"]),
                  norm_bias=(L.norm_bias, g["norm_bias"]), wg=(L.wg, g["wg"]), bias=(L.bias, g["bias"]),
                  w1=(L.w["w1"], g["w1"]), w3=(L.w["w3"], g["w3"]), w2=(L.w["w2"], g["w2"]))
    for name, (leaf, grad) in leaves.items():
        v = torch.randn(leaf.shape, generator=torch.Generator().manual_seed(3)).cuda()
        keep = leaf.clone()
        ends = []
        for sign in (1, -1):
            leaf.copy_(keep + sign * EPS * v)
            ends.append(forward())
            assert torch.equal(L.idx, idx), name
        leaf.copy_(keep)
        want = float((grad.double() * v.double()).sum())
        got = (ends[0] - ends[1]) / (2 * EPS)
        say(f"    {name}: gradient {want:.4f}, differences {got:.4f}")
        assert abs(got - want) <= 1e-2 * abs(want) + 5e-2, name
