"""A training step of norm + layer: the forward pass that keeps, and the
gradients chained as a training step chains them, against the float64 oracle,
captured and replayed, on two streams at once, and against moe_forward.

Tolerance.  Every stage's own test holds it to derived element bounds; here
the chain is held by relative 2-norms.  With float32 each stage adds a few
hundred 2^-24.  With bf16 weights each stored intermediate (xn, h, g, u, dg,
du, w h, da, dxn, the outputs) is one rounding of at most 2^-8 of its value,
2^-8 / sqrt(3) in the root mean square; the longest chain to an output holds
eight of them (xn, g or u, dg, da, dxn, dx and the two of dtopk_w's path
through the router): sqrt(8) 2^-8 / sqrt(3) = 6.4e-3.  The norm's and router's
projections take away parts of a gradient but not of its errors; a factor of
3 covers that."""

import numpy as np
import pytest

import oracle
from mixture_experts_layer_wave_amd import workloads as W
from tests.gpu_support import SMALL, say, small
from tests.golden.make_routing_fixtures import find_redraws

pytestmark = pytest.mark.gpu

NORM = {"bf16": 3 * (8 / 3) ** 0.5 * 2.0 ** -8, "f32": 2.0 ** -24 * 4096}

LAYERS = {
    "bf16": small("train-bf16", 300, 136, 5, 2, 200, "bf16", 31),
    "bf16-top1": small("train-bf16-top1", 200, 64, 8, 1, 96, "bf16", 33),
    "f32": small("train-f32", 90, 20, 6, 2, 36, "f32", 35, act="f32"),
    "f32-every-expert": small("train-f32-soft", 60, 20, 3, 3, 36, "f32", 37, act="f32"),
}


def _layer(name):
    wl = LAYERS[name]
    L = W.make_layer(wl, redraws=find_redraws(wl), use_fixture=False, cache=False)
    L["bias"] = np.linspace(-0.3, 0.3, wl.E).astype(np.float32)
    return L


def _f64(t):
    import torch

    return (t.view(torch.bfloat16) if t.dtype == torch.int16 else t).double().cpu().numpy()


def _dy(D, seed):
    import torch

    t = torch.from_numpy(np.random.default_rng(seed).standard_normal((D.n, D.d)).astype(np.float32)).cuda()
    return t.to(torch.bfloat16).view(torch.int16) if D.act == "bf16" else t


@pytest.mark.parametrize("name", sorted(LAYERS))
def test_step_matches_the_oracle(name):
    import torch
    from mixture_experts_layer_wave_amd.device import TrainingLayer

    say(f"[training] {name}")
    T = TrainingLayer(_layer(name), alpha=0.1)
    rng = np.random.default_rng(5)
    T.norm_weight.copy_(torch.from_numpy((1 + 0.2 * rng.standard_normal(T.d)).astype(np.float32)))
    T.norm_bias.copy_(torch.from_numpy((0.2 * rng.standard_normal(T.d)).astype(np.float32)))
    dy = _dy(T, 6)
    y = T.forward_train()
    grads = T.backward(dy)
    torch.cuda.synchronize()

    x, w, b = _f64(T.x), _f64(T.norm_weight), _f64(T.norm_bias)
    w1, w3, w2, wg = (
        _f64(T.w["w1"]), _f64(T.w["w3"]), _f64(T.w["w2"]), _f64(T.wg))
    idx = T.idx.cpu().numpy()  # the library's choice: near ties may fall differently after the norm
    renorm = T.k > 1
    xn, mean, rstd = oracle.layer_norm(x, w, b, T.eps)
    z = xn @ wg.T + _f64(T.bias)
    tw, p = oracle.router_weights(z, idx, renorm)
    f = np.bincount(idx[:, 0], minlength=T.E) / T.n
    dp = oracle.dispatch(idx, T.E)
    perm, inv, offsets = dp["perm"], dp["inv"].reshape(T.n, T.k), dp["offsets"]
    assert np.array_equal(inv, T.inv.cpu().numpy()) and np.array_equal(offsets, T.offsets.cpu().numpy())
    h, g, u = oracle.expert_up(xn, perm, offsets, w1, w3)
    want_y = np.zeros((T.n, T.d))
    for t in range(T.n):
        for j in range(T.k):
            want_y[t] += tw[t, j] * (h[inv[t, j]] @ w2[idx[t, j]].T)
    aux = 0.1 * T.E * (f * p.mean(axis=0)).sum()
    da, dw1, dw3, dw2, dtw = oracle.grouped_ffn_grad(_f64(dy), xn, perm, inv, tw, offsets, w1, w3, w2, g, u)
    dz, dxn, dwg, db = oracle.router_grad(z, idx, tw, dtw, f, 0.1, renorm, xn, wg, da, inv)
    dx, dnw, dnb = oracle.layer_norm_grad(dxn, x, w, mean, rstd)
    ref = dict(x=dx, norm_weight=dnw, norm_bias=dnb, wg=dwg, bias=db, w1=dw1, w3=dw3, w2=dw2)
    lim = NORM[T.act]
    err = np.linalg.norm(_f64(y) - want_y) / np.linalg.norm(want_y)
    say(f"    y {err:.2e}, aux {float(T.aux)} against {aux}")
    assert err <= lim and abs(float(T.aux) - aux) <= 1e-3 * aux
    for key, want in ref.items():
        got = _f64(grads[key])
        err = np.linalg.norm(got - want) / np.linalg.norm(want)
        say(f"    d{key}: {err:.2e} of {lim:.2e}")
        assert np.isfinite(got).all() and err <= lim, key


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_forward_train_matches_moe_forward(name):
    """With the norm's output as its input, moe_forward gives the same layer."""
    import torch
    from mixture_experts_layer_wave_amd.device import TrainingLayer

    T = TrainingLayer(_layer(name))
    y = T.forward_train().clone()
    idx = T.idx.clone()
    T.x.copy_(T.xn)
    T.forward()
    torch.cuda.synchronize()
    assert torch.equal(idx, T.idx)
    a, c = _f64(y), _f64(T.y)
    assert np.linalg.norm(a - c) <= NORM[T.act] * np.linalg.norm(c)


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_captured_step_replays(name):
    """Forward and backward in one HIP graph; every replay, with eager steps
    of the same buffers in between, gives the eager step's bits, and follows
    new inputs."""
    import torch
    from mixture_experts_layer_wave_amd.device import TrainingLayer

    say(f"[training graph] {name}")
    T = TrainingLayer(_layer(name))
    dy = _dy(T, 8)
    x2, dy2 = T.x.flip(0).contiguous(), _dy(T, 9)
    x1, dy1 = T.x.clone(), dy.clone()

    def step(stream=None):
        T.forward_train(stream)
        T.backward(dy, stream)

    def result():
        torch.cuda.synchronize()
        return [T.y.clone(), T.aux.clone()] + [T.grads[key].clone() for key in sorted(T.grads)]

    step()
    eager1 = result()
    T.x.copy_(x2), dy.copy_(dy2)
    step()
    eager2 = result()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step(s)
    for rep in range(4):
        first = rep % 2 == 0
        T.x.copy_(x1 if first else x2), dy.copy_(dy1 if first else dy2)
        for t in T.grads.values():
            t.fill_(3)
        T.train_ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        for p, q in zip(result(), eager1 if first else eager2):
            assert torch.equal(p, q), rep
        step()  # eager work between the replays
        torch.cuda.synchronize()


def test_calls_take_the_current_stream():
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    side = torch.cuda.Stream()
    assert B._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert B._stream(None) == side.cuda_stream == B._stream(side)
    assert B._stream(None) == torch.cuda.current_stream().cuda_stream != side.cuda_stream


def test_two_steps_at_once_on_two_streams():
    import torch
    from mixture_experts_layer_wave_amd.device import TrainingLayer

    say("[training] two streams")
    Ts = [TrainingLayer(_layer("bf16")), TrainingLayer(_layer("bf16-top1"))]
    dys = [_dy(T, 20 + i) for i, T in enumerate(Ts)]
    want = []
    for T, dy in zip(Ts, dys):
        T.forward_train(), T.backward(dy)
        torch.cuda.synchronize()
        want.append([T.grads[key].clone() for key in sorted(T.grads)])
    streams = [torch.cuda.Stream() for _ in Ts]
    torch.cuda.synchronize()
    for _ in range(5):
        for T in Ts:
            for t in T.grads.values():
                t.fill_(3)
        torch.cuda.synchronize()
        for T, dy, s in zip(Ts, dys, streams):
            T.forward_train(s), T.backward(dy, s)
        torch.cuda.synchronize()
        for T, w in zip(Ts, want):
            for p, key in zip(w, sorted(T.grads)):
                assert torch.equal(p, T.grads[key]), key


def test_gradient_against_differences():
    """The gradient of every input of the step along its own sign, against the
    change of the linear loss sum(y dy) of the library's forward pass.  Every
    token takes every expert, so the choice of experts stays what it is and
    the loss is smooth."""
    import torch
    from mixture_experts_layer_wave_amd.device import TrainingLayer

    say("[training] differences")
    T = TrainingLayer(_layer("f32-every-expert"), alpha=0.0)
    dy = _dy(T, 30)

    def loss():
        T.forward_train()
        torch.cuda.synchronize()
        return float((T.y.double() * dy.double()).sum())

    loss()
    T.backward(dy)
    torch.cuda.synchronize()
    var = dict(x=T.x, norm_weight=T.norm_weight, norm_bias=T.norm_bias, wg=T.wg, bias=T.bias, w1=T.w["w1"],
               w3=T.w["w3"], w2=T.w["w2"])
    grads = {key: T.grads[key].clone() for key in var}
    size = float((T.y.double().abs() * dy.double().abs()).sum())
    for key, v in var.items():
        step = torch.sign(grads[key]) * 2.0 ** -9
        keep = v.clone()
        v.copy_(keep + step)
        hi, plus = loss(), v.double()
        v.copy_(keep - step)
        lo, minus = loss(), v.double()
        want = float((grads[key].double() * (plus - minus)).sum())
        v.copy_(keep)
        # float32 noise: (d + d_ff + 64) 2^-24 of the terms, sqrt(d_ff) times y's
        # size; third order: relative to the difference the square of what a step
        # moves an activation by, 2^-9 d (all signs along the gradient) = 0.04
        tol = 8 * (T.d + T.d_ff + 64) * 2.0 ** -24 * size * T.d_ff ** 0.5 + 0.04 ** 2 * 4 * abs(want)
        say(f"    {key}: {hi - lo:.6e} against {want:.6e}, tolerance {tol:.1e}")
        assert abs(hi - lo - want) <= tol, key
