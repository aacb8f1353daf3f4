"""What DecodeBlock refuses before anything is encoded (no GPU needed): the
library gets addresses alone, so a tensor of another shape or type would be
misread, or read past its end."""

import pytest
import torch

from mixture_experts_layer_wave_amd.device import DecodeBlock

E, D, F, M, BF = 4, 64, 96, 50, torch.bfloat16


def _args(**kw):
    norm = lambda: dict(kind="rms", weight=torch.ones(D), bias=None, eps=1e-5)
    v = dict(n=2, wg=torch.zeros(E, D, dtype=BF), w1=torch.zeros(E, F, D, dtype=BF), w3=torch.zeros(E, F, D, dtype=BF),
             w2=torch.zeros(E, D, F, dtype=BF), k=2, bias=torch.zeros(E), gate=torch.zeros(D), post=norm(), pre=norm(),
             head=torch.zeros(M, D, dtype=BF))
    v.update(kw)
    return v


def _norm(**kw):
    v = dict(kind="layer", weight=torch.ones(D), bias=torch.zeros(D), eps=1e-5)
    v.update(kw)
    return v


BAD = [
    ("w1", dict(w1=torch.zeros(F, D, dtype=BF))),
    ("w1", dict(w1=torch.zeros(E, F, D, dtype=torch.float16))),
    ("w3", dict(w3=torch.zeros(E, F, D // 2, dtype=BF))),
    ("w3", dict(w3=torch.zeros(E, F, D, dtype=torch.int16))),
    ("w2", dict(w2=torch.zeros(E, F, D, dtype=BF))),  # not transposed
    ("w2", dict(w2=torch.zeros(E - 1, D, F, dtype=BF))),
    ("head", dict(head=torch.zeros(M, D // 2, dtype=BF))),
    ("head", dict(head=torch.zeros(D, dtype=BF))),
    ("head", dict(head=torch.zeros(M, D, dtype=torch.float16))),
    ("wg", dict(wg=torch.zeros(E, D))),
    ("wg", dict(wg=torch.zeros(E - 1, D, dtype=BF))),
    ("wg", dict(wg=torch.zeros(D, E, dtype=BF).t())),
    ("bias", dict(bias=torch.zeros(E, dtype=BF))),
    ("bias", dict(bias=torch.zeros(E - 1))),
    ("bias", dict(bias=torch.zeros(2 * E)[::2])),
    ("gate", dict(gate=torch.zeros(D, dtype=BF))),
    ("gate", dict(gate=torch.zeros(1))),
    ("post: no norm", dict(post=_norm(kind="batch"))),
    ("post weight", dict(post=_norm(weight=torch.ones(D, dtype=BF)))),
    ("post bias", dict(post=_norm(bias=torch.zeros(D // 2)))),
    ("pre weight", dict(pre=_norm(weight=torch.ones(D + 1)))),
    ("pre bias", dict(pre=_norm(bias=torch.zeros(2 * D)[::2]))),
    ("wg is on", dict(wg=torch.zeros(E, D, dtype=BF, device="meta"))),
    ("gate is on", dict(gate=torch.zeros(D, device="meta"))),
]


@pytest.mark.parametrize("name,kw", BAD, ids=[f"{i}-{name}" for i, (name, _) in enumerate(BAD)])
def test_refused(name, kw):
    with pytest.raises(ValueError, match="^" + name):
        DecodeBlock(**_args(**kw))


@pytest.mark.parametrize("kw", [dict(), dict(bias=None, gate=None, post=None, pre=None, head=None),
                                dict(post=_norm(), pre=_norm(bias=None)), dict(post=_norm(kind=0), pre=_norm(kind=1)), dict(w1=torch.zeros(E, F, D)),
                                dict(w2=torch.zeros(E, F, D, dtype=BF).transpose(1, 2))])
def test_right_ones_get_as_far_as_the_encoder(kw):
    with pytest.raises(ValueError, match="encode_mxfp4 takes device tensors"):
        DecodeBlock(**_args(**kw))
