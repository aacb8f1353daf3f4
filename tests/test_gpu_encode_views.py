"""encode_mxfp4 of tensors that are views: the codes are those of a contiguous
copy, bit for bit, on any stream."""

import pytest

from tests.gpu_support import say

pytestmark = pytest.mark.gpu

VIEWS = {
    "transposed": lambda t: t(96, 64).transpose(0, 1),
    "experts transposed": lambda t: t(3, 64, 96).transpose(1, 2),
    "columns of a wider matrix": lambda t: t(40, 256)[:, 64:160],
    "rows of a fused matrix": lambda t: t(5, 48, 64)[:, 16:],
    "every other row": lambda t: t(40, 64)[::2],
    "every other column": lambda t: t(40, 128)[:, ::2],
    "one row again and again": lambda t: t(1, 64).expand(33, 64),
    "one value": lambda t: t(1, 1).expand(7, 32),
    "contiguous": lambda t: t(40, 64),
    "one row": lambda t: t(64),
    "no rows": lambda t: t(0, 64),
}


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("view", VIEWS)
def test_views(view, dtype):
    import torch
    from mixture_experts_layer_wave_amd import binding as B
    from mixture_experts_layer_wave_amd.device import encode_mxfp4

    say(f"[encode] {view} {dtype}")
    gen = torch.Generator().manual_seed(3)
    w = VIEWS[view](lambda *s: torch.randn(s, generator=gen).to(getattr(torch, dtype)).cuda())
    plain = torch.empty(w.shape, dtype=w.dtype, device="cuda")
    plain.copy_(w)
    cols = w.shape[-1]
    rows = w.numel() // cols
    want = (torch.zeros((*w.shape[:-1], cols // 2), dtype=torch.uint8, device="cuda"),
            torch.zeros((*w.shape[:-1], cols // 32), dtype=torch.uint8, device="cuda"))
    B.moe_quantize_mxfp4(rows, cols, plain, "f32" if dtype == "float32" else "bf16", *want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream, torch.cuda.current_stream(), 0):
        q, s = encode_mxfp4(w, stream)
        torch.cuda.synchronize()
        assert q.shape == want[0].shape and s.shape == want[1].shape
        assert torch.equal(q, want[0]) and torch.equal(s, want[1])


def test_a_copy_lives_as_long_as_its_stream_needs_it():
    """Many views encoded on a side stream in a row, with the current stream
    taking and filling memory meanwhile."""
    import torch
    from mixture_experts_layer_wave_amd.device import encode_mxfp4

    ws = [torch.randn((512, 1024), generator=torch.Generator().manual_seed(i)).cuda().t() for i in range(8)]
    want = [tuple(t.clone() for t in encode_mxfp4(w.contiguous())) for w in ws]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for rep in range(5):
        got = []
        for w in ws:
            got.append(encode_mxfp4(w, side))
            torch.empty((1024, 512), device="cuda").fill_(float("nan"))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, v in zip(got, want) for a, b in zip(g, v))


def test_other_types_are_refused():
    import torch
    from mixture_experts_layer_wave_amd.device import encode_mxfp4

    for dtype in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError):
            encode_mxfp4(torch.zeros((4, 64), dtype=dtype, device="cuda"))
    with pytest.raises(ValueError):
        encode_mxfp4(torch.zeros((), device="cuda"))
