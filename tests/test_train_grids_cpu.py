"""Shapes whose launches would have 2^32 threads or more are refused before any
launch (no GPU needed)."""

import pytest

from mixture_experts_layer_wave_amd import binding as B
from tests.test_train_abi_cpu import BF16, F32, _back, _up

SHAPE, NULL = -2, -1


# (the missing pointer keeps a call that is not refused from being launched)
@pytest.mark.parametrize("act,shape", [
    (BF16, (8, 8, 1024, 1, (1 << 20) - 8)),       # the weight gradients' tiles, 24 million of them
    (BF16, (8, (1 << 20) - 8, 1024, 1, 8)),
    (F32, (8, 1, 1024, 1, (1 << 19) - 1)),
    (F32, ((1 << 29) - 1, 1, 1, 1, 1)),           # pile rows
    (F32, (1 << 28, 1, 4, 1, 1)),
])
def test_refused(act, shape):
    assert _up(shape=shape, act=act, a=None) == SHAPE and _back(shape=shape, act=act, dy=None) == SHAPE
    assert B.moe_grouped_ffn_backward_workspace_bytes(shape, act) == 0


# Long lists of experts, wide layers and long batches that fit the card.
@pytest.mark.parametrize("act,shape", [
    (BF16, (8192, 4096, 8, 2, 14336)),
    (BF16, (16384, 7168, 256, 8, 2048)),
    (BF16, (4096, 4096, 1024, 8, 4096)),
    (F32, (4096, 4096, 256, 2, 4096)),
    (BF16, (8, 8, 8, 1, (1 << 20) - 8)),
    (F32, (1 << 27, 2, 4, 1, 2)),
    (BF16, (1 << 26, 8, 1024, 1, 8)),
])
def test_not_refused(act, shape):
    assert B.moe_grouped_ffn_backward_workspace_bytes(shape, act) > 0
    assert _up(shape=shape, act=act, a=None) == NULL and _back(shape=shape, act=act, dy=None) == NULL
