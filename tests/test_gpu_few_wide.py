"""moe_forward_few with a hidden of 2^25 columns: its row chunks as bytes, were
they all in LDS, pass 2^31 (16 rows of 2^19 chunks of 272 bytes).

W2 is zero but for 3000 columns spread over the row, so that the reference needs
only those of the hidden, and a sum has 3000 terms that are not zero.  Tolerance
(derived, not measured), U = 2^-24: a hidden value's two products are 8 terms
deep; 1.1 bounds silu's slope, 16 + 2 |g| units cover silu itself and 4 the
products around it; the output's sum is at most 3000 additions and 64 more deep,
and is rounded once."""

import numpy as np
import pytest

from tests.gpu_support import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def test_hidden_of_two_gigabytes():
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    n, d, f = 16, 8, (1 << 25) + 12
    say(f"[few wide] float32 n {n} d {d} f {f}")
    shape = (n, d, 1, 1, f, 0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    w1 = torch.randn((1, f, d), generator=gen, device="cuda") * d ** -0.5
    w3 = torch.randn((1, f, d), generator=gen, device="cuda") * d ** -0.5
    x = torch.randn((n, d), generator=gen, device="cuda")
    cols = torch.randperm(f, generator=gen, device="cuda")[:2990]
    cols = torch.cat([cols, torch.tensor([0, 1, 63, 64, 1023, f - 65, f - 64, f - 13, f - 2, f - 1], device="cuda")]).unique()
    w2 = torch.zeros((1, d, f), device="cuda")
    w2[0][:, cols] = torch.randn((d, len(cols)), generator=gen, device="cuda")
    wg = torch.ones((1, d), device="cuda")
    nb = B.moe_forward_few_workspace_bytes(shape, "f32")
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    y = torch.full((n + 1, d), 7.0, device="cuda")
    B.moe_forward_few(shape, x, "f32", wg, None, dict(dtype="f32", w1=w1, w3=w3, w2=w2), y, "f32", None, None, ws, nb)
    torch.cuda.synchronize()
    assert (y[n] == 7).all()
    f64 = lambda t: t.double().cpu().numpy()
    X, W1, W3, W2 = f64(x), f64(w1[0][cols]), f64(w3[0][cols]), f64(w2[0][:, cols])
    g, u = X @ W1.T, X @ W3.T
    s = g / (1 + np.exp(-g))
    eg, eu = (72 * U * (np.abs(X) @ np.abs(m).T) for m in (W1, W3))
    eh = (1.1 * eg + (16 + 2 * np.abs(g)) * U * np.abs(s)) * np.abs(u) + np.abs(s) * eu + 1.1 * eg * eu
    h = np.abs(s * u)
    ref = (s * u) @ W2.T
    tol = U * np.abs(ref) + (eh + 4 * U * h) @ np.abs(W2).T + (3000 + 64) * U * (h @ np.abs(W2).T)
    worst = (np.abs(f64(y[:n]) - ref) / tol).max()
    say(f"    largest error / tolerance {worst:.3f}")
    assert worst <= 1
