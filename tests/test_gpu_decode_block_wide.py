"""Which of the two calls of the layer a DecodeBlock takes, and steps of blocks
on both sides of each border, against the float64 oracle (tolerances as in
test_gpu_decode_block_forms.py, each stage from the one before it as stored)."""

import numpy as np
import pytest

from oracle import serve_oracle as S
from tests.gpu_support import say
from tests.test_gpu_decode_block import _dec, _f64, _norm, _norm64
from tests.test_gpu_decode_block_forms import _check_choices, _layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,d,f,few", [(4, 64, 96, True), (5, 64, 96, False), (16, 64, 96, False), (5, 64, 7168, False),
                                       (1, 64, 7200, True), (5, 64, 7200, True), (16, 64, 7200, True),
                                       (16, 7200, 64, True), (17, 64, 7200, False)])
def test_steps_on_both_sides_of_the_rule(n, d, f, few):
    import torch
    from mixture_experts_layer_wave_amd import binding as B
    from mixture_experts_layer_wave_amd.device import DecodeBlock

    E, k = 4, 2
    say(f"[decode block] n {n} d {d} f {f}")
    rng = np.random.default_rng(n + d + f)
    bf = lambda *s, scale=1.0: torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).cuda().bfloat16()
    blk = DecodeBlock(n, bf(E, d, scale=d ** -0.5), bf(E, f, d, scale=d ** -0.5), bf(E, f, d, scale=d ** -0.5),
                      bf(E, d, f, scale=f ** -0.5), k, post=_norm(rng, d, "rms"), pre=_norm(rng, d, "rms"))
    assert blk.layer is (B.moe_forward_few if few else B.moe_forward)
    blk.h.copy_(bf(n, d))
    blk.u.copy_(bf(n, d))
    w = {key: _dec(blk.experts["w" + key], blk.experts["s" + key]) for key in "132"}
    for step in range(2):
        h0, u0 = _f64(blk.h), _f64(blk.u)
        out = blk.step()
        torch.cuda.synchronize()
        idx = blk.idx.cpu().numpy()
        _check_choices(u0, _f64(blk.wg), idx)
        y, size = _layer(u0, _f64(blk.wg), w, idx, True)
        z = _f64(blk.z)
        # float32 sums of d and of f terms, f / 32 + 64 additions deep at most, beside the roundings
        deep = (max(d, f) / 32 + 64) * 2.0 ** -24
        assert (np.abs(z - y) <= 2.0 ** -8 * np.abs(y) + (2.0 ** -8 + 2.0 ** -13 + 4 * deep) * size).all(), step
        b = S.block_norm(h0, z, 1.0, None, _norm64(blk.post), _norm64(blk.pre))
        slack = 2.0 ** -14 * (1 + np.abs(b["h"]).max(axis=1, keepdims=True))
        assert (np.abs(_f64(blk.h) - b["h"]) <= 2.0 ** -8 * np.abs(b["h"]) + slack).all()
        assert (np.abs(_f64(out) - b["u"]) <= 2.0 ** -8 * np.abs(b["u"]) + 4 * slack).all()
