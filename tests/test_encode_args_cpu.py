"""What encode_mxfp4 refuses before any launch (no GPU needed)."""

import pytest
import torch

from mixture_experts_layer_wave_amd.device import encode_mxfp4


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int16, torch.uint8])
def test_other_types_are_refused(dtype):
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        encode_mxfp4(torch.zeros((4, 64), dtype=dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_host_tensors_are_refused(dtype):
    with pytest.raises(ValueError, match="device tensors"):
        encode_mxfp4(torch.zeros((4, 64), dtype=dtype))
