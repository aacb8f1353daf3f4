"""moe_router_backward on logits that are NaN or -inf throughout.

A NaN logit makes its token's probabilities NaN, and with them whatever is
taken from them: dlogits (raw weights, or the auxiliary loss), the token's dx
and the sums over tokens.  Only a token whose logits are -inf, every one of
them, has no gradient.  The numbers of experts leave lanes without an expert
(5, 48, 100, 300), or none (8, 64, 128)."""

import pytest

from tests.gpu_support import say
from tests.test_gpu_router_grad import _batch, _run

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("E", [1, 5, 8, 48, 64, 100, 128, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_and_masked_tokens(dtype, E, renorm):
    import torch

    say(f"[router grad, NaN] {dtype} E={E} renorm={renorm}")
    n, d, k = 45, 72, min(E, 2)
    shape = (n, d, E, k, 8, renorm)
    b = _batch(dtype, n, d, E, k, renorm)
    spoilt, dead = [2, 17], [9]
    if E > 1:
        spoilt += [5, 31, 44]
    base = {aux: _run(b, dtype, shape, aux=aux) for aux in (True, False)}
    b["z"][[2, 17]] = NAN            # every logit
    if E > 1:
        b["z"][[5, 31]] = -INF       # one NaN, the rest masked
        b["z"][5, 0] = NAN
        b["z"][31, E - 1] = NAN
        b["z"][44, E // 2] = NAN     # one NaN among numbers
    b["z"][9] = -INF
    keep = [t for t in range(n) if t not in spoilt + dead]
    for aux in (True, False):
        dz, dx, dwg, db = _run(b, dtype, shape, aux=aux)
        assert not dz[dead].any() and torch.isfinite(dx[dead]).all()
        assert torch.equal(dz[keep], base[aux][0][keep]) and torch.equal(dx[keep], base[aux][1][keep])
        if aux or not renorm:        # something takes the probabilities
            for got in (dz[spoilt], dx[spoilt], dwg, db):
                assert torch.isnan(got).all()
        else:                        # the weights' own gradient: no logit enters
            assert torch.equal(dz[spoilt], base[aux][0][spoilt]) and torch.equal(dx[spoilt], base[aux][1][spoilt])
            assert torch.isfinite(dwg).all() and torch.isfinite(db).all()
