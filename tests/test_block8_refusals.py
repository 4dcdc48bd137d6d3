"""Calls of the block-scaled FP8 helpers that the binding refuses with its own error, on the CPU."""
import pytest
import torch

import bit_gemm_group_b200 as wq


@pytest.mark.parametrize("rows", [0, -1, -128, 64])
def test_block_rows_that_are_none(rows):
    with pytest.raises(wq.WQError):
        wq.quantize_fp8_block(torch.zeros(8, 256, dtype=torch.bfloat16), rows)


@pytest.mark.parametrize("Wq,scales", [
    (torch.zeros(64, 512, dtype=torch.uint8), torch.zeros(1, 4)),         # another K
    (torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(1, 2)),      # no codes
    (torch.zeros(256, 256, dtype=torch.uint8), torch.zeros(2, 4)),        # scales of another K
])
def test_a_weight_of_another_shape(Wq, scales):
    """Large enough buffers whose rows lie elsewhere than the product would read them."""
    X = torch.zeros(4, 256, dtype=torch.bfloat16)
    Y = torch.zeros(4, Wq.shape[0], dtype=torch.bfloat16)
    with pytest.raises(wq.WQError, match="Wq must|w_scales must"):
        wq.wq_gemm_fp8_block(X, Wq, scales, Y, torch.zeros(256, dtype=torch.uint8))
