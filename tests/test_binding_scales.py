"""The scaled product's token scales are taken by address and stride: the binding refuses what does not lie as they say
(CPU only: each call is refused before the library's)."""

import pytest
import torch

import combine_moe_layout_03_amd as M


def call(token_scale, stride=4):
    a, w = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(1, 4, 16, dtype=torch.int8)
    M.moe_grouped_gemm_deq_i8(a, 16, 4, 16, torch.zeros(1, dtype=torch.int32), w, torch.zeros(1, 4), token_scale,
                              torch.zeros(4, 4), token_scale_stride=stride)


@pytest.mark.parametrize("scale", [
    torch.zeros(8)[::2],                                              # every other float, read as neighbours
    torch.zeros(4, 2)[:, :1],
    torch.zeros(4, 8, dtype=torch.uint8)[:, :4].view(torch.float32),  # the scales of packed rows, without their stride
    torch.zeros(4, dtype=torch.float64), torch.zeros(8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32),
    torch.zeros(8, dtype=torch.float16),
], ids=["sliced", "column", "packed", "fp64", "bf16", "int32", "fp16"])
def test_refused(scale):
    with pytest.raises(ValueError, match="token_scale must be contiguous float32 or bytes"):
        call(scale)


@pytest.mark.parametrize("scale,stride", [(torch.zeros(4), 4), (torch.zeros(4, 1), 4), (torch.zeros(64, dtype=torch.uint8), 16),
                                          (torch.zeros(64, dtype=torch.int8)[8:], 16), (torch.zeros(4, 3), 12)])
def test_taken(scale, stride):
    """These pass that check (and are refused as host tensors)."""
    with pytest.raises(ValueError, match="must be a device tensor"):
        call(scale, stride)
