"""moe_router_backward where rows lie past 32-bit offsets: of x, dx and da_perm
(more than 2^32 bytes and 2^31 elements in), and of the logits and dlogits
(and, with bf16 rows, what the products read of them).

Only a few tokens have a weight gradient, so all other tokens' dlogits are
zero and their dx is the row of da_perm that they gather, bit for bit.  The
few are held to the same tokens run by themselves, which
test_gpu_router_grad.py holds to the oracle.  dW_g and dbias: sums with as many
addends that are not zero as there are such tokens, twice that with dlogits in
two halves: at most 16 roundings of 2^-24 of the addends' sizes, dlogits' 2^-16
with bf16 rows, and the output's own half step."""

import pytest

from tests.gpu_support import say
from tests.test_gpu_router_grad import HALF, SPLIT, U

pytestmark = pytest.mark.gpu


def _call(dtype, n, d, E, z, idx, w, dw, x, wg, da, inv):
    import torch
    from mixture_experts_layer_wave_amd import binding as B

    shape = (n, d, E, 1, 8, 0)
    dz, db = torch.full_like(z, 7.0), torch.empty(E, device="cuda")
    dx, dwg = torch.full_like(x, 7.0), torch.empty_like(wg)
    nb = B.moe_router_backward_workspace_bytes(shape)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    B.moe_router_backward(shape, z, idx, w, dw, None, 0.0, x, dtype, wg, da, inv, dz, dx, dwg, db, ws, nb)
    torch.cuda.synchronize()
    return dz, dx, dwg, db


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,E", [(40000, 65536, 2), ((1 << 21) + 100, 8, 1024)])
def test_rows_past_32_bit_offsets(dtype, n, d, E):
    import torch

    say(f"[router grad, offsets past 32 bits] {dtype} n={n} d={d} E={E}")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(n + E)

    def normal(*size, dtype=torch.float32):
        return torch.empty(size, dtype=dtype, device="cuda").normal_(generator=gen)

    rows = [0, n // 2 + 1, n - 2, n - 1]
    z, x, da = normal(n, E), normal(n, d, dtype=dt), normal(n, d, dtype=dt)
    wg = normal(E, d, dtype=dt)
    idx = (torch.arange(n, device="cuda", dtype=torch.int32) % E)[:, None].contiguous()
    inv = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.int32)[:, None].contiguous()
    p = torch.softmax(z[rows].double(), dim=1)
    w = torch.zeros(n, 1, device="cuda")
    w[rows] = p.gather(1, idx[rows].long()).float()
    dw = torch.zeros(n, 1, device="cuda")
    dw[rows] = torch.tensor([[1.0], [-2.0], [0.5], [3.0]], device="cuda")
    dz, dx, dwg, db = _call(dtype, n, d, E, z, idx, w, dw, x, wg, da, inv)

    few = [t[rows].contiguous() for t in (z, idx, w, dw, x)]
    order = torch.arange(len(rows), device="cuda", dtype=torch.int32)[:, None].contiguous()
    gathered = da[inv[rows, 0].long()].contiguous()
    dz1, dx1, dwg1, db1 = _call(dtype, len(rows), d, E, *few, wg, gathered, order)
    assert dz1.any() and torch.equal(dz[rows], dz1) and torch.equal(dx[rows], dx1)
    dz[rows] = 0
    assert not dz.any()
    for t0 in range(0, n, 1 << 17):  # dx = da[inv], inv from the last row back
        t1 = min(n, t0 + (1 << 17))
        same = (dx[t0:t1] == da[n - t1:n - t0].flip(0)).all(dim=1)
        same[[t - t0 for t in rows if t0 <= t < t1]] = True
        assert same.all(), t0
    dz64, x64 = dz1.double(), few[4].double()
    ref, size = dz64.T @ x64, dz64.abs().T @ x64.abs()
    for got in (dwg, dwg1):
        assert ((got.double() - ref).abs() <= HALF[dtype] * ref.abs() + (SPLIT[dtype] + 16 * U) * 1.01 * size).all()
    for got in (db, db1):
        assert ((got.double() - dz64.sum(0)).abs() <= 16 * U * dz64.abs().sum(0)).all()
