"""Calls of the block-scaled FP8 helpers that the binding refuses with its own error, on the CPU."""
import pytest
import torch

import bit_gemm_group_b200 as wq


@pytest.mark.parametrize("rows", [0, -1, -128, 64])
def test_block_rows_that_are_none(rows):
    with pytest.raises(wq.WQError):
        wq.quantize_fp8_block(torch.zeros(8, 256, dtype=torch.bfloat16), rows)
