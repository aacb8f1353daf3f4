"""moe_forward_few's choice of experts where the float64 logits decide it: tokens
are redrawn until every gap among their k + 1 largest logits is more than the
logits' rounding can close, so the choices have to be the oracle's exactly.

A logit of d terms is off by a float32 sum at most d / 32 + 64 (bf16) or d / 8 +
64 (float32) additions deep, with its bias by one more rounding: `ez`.  Two
logits 2 ez apart keep their order."""

import numpy as np
import pytest

from tests.gpu_support import say
from tests.test_gpu_few import CASES, Few, U

pytestmark = pytest.mark.gpu


def _gaps(L):
    """(smallest gap among each token's k + 1 largest logits, twice what rounding moves them)"""
    import oracle

    n, d, E, k, f, wdt = L.args
    x, wg = L.x.double().cpu().numpy(), L.wg.double().cpu().numpy()
    z = oracle.router_logits(x, wg, None if L.bias is None else L.bias.double().cpu().numpy())
    top = -np.sort(-z, axis=1)[:, : min(k + 1, E)]
    gap = (top[:, :-1] - top[:, 1:]).min(axis=1, initial=np.inf)
    ez = ((d / 8 if wdt == "f32" else d / 32) + 64) * U * (np.abs(x) @ np.abs(wg).T).max(axis=1)
    return gap, 2 * (ez + 2 * U * np.abs(z).max(axis=1))


@pytest.mark.parametrize("n,d,E,k,f,wdt", CASES)
def test_choices_that_the_logits_decide(n, d, E, k, f, wdt):
    import torch

    say(f"[few choices] {wdt} n {n} d {d} E {E} k {k} f {f}")
    L = Few(n, d, E, k, f, wdt, seed=7)
    rng = np.random.default_rng(d + E)
    for _ in range(200):
        gap, need = _gaps(L)
        poor = np.nonzero(gap <= need)[0]
        if len(poor) == 0:
            break
        new = rng.standard_normal((len(poor), d)).astype(np.float32)
        L.x[torch.from_numpy(poor).cuda()] = torch.from_numpy(new).cuda().to(L.dt)
    gap, need = _gaps(L)
    assert (gap > need).all()  # (of the inputs)
    r, m = L.ref()
    y, idx, tw = L.run()
    assert np.array_equal(idx.cpu().numpy(), r["idx"])
    ew, ty = L.tolerances(r, m, L.act)
    assert (np.abs(tw.double().cpu().numpy() - r["w"]) <= ew).all()
    assert (np.abs(y.double().cpu().numpy() - r["y"]) <= ty).all()
