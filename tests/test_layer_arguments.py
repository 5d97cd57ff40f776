"""Arguments of the operators around the gated delta rule that would not fit what the library takes: refused before any
tensor is looked at or made, so that no GPU is needed to see it."""
import pytest
import torch

import kimi_delta_attention_21_b200 as K
from kimi_delta_attention_21_b200 import _lib as L


@pytest.mark.parametrize("block_rows", [2 ** 32 + 1, 2 ** 32 + 128, -2 ** 32 + 1, -2 ** 32 + 128, 2 ** 31, 2 ** 63 - 1])
def test_block_rows_beyond_32_bits_are_refused(block_rows):
    """Cut to 32 bits they would read as 1 or 128, beside scales made for one block of rows."""
    n0 = L.load().kda_launch_count()
    with pytest.raises(ValueError, match="block_rows"):
        K.quant_fp8(torch.zeros(300, 256), block_rows)
    assert L.load().kda_launch_count() == n0


def test_block_rows_beyond_any_integer_are_refused():
    with pytest.raises(OverflowError):
        K.quant_fp8(torch.zeros(4, 4), 2 ** 64 + 1)
    with pytest.raises(TypeError):
        K.quant_fp8(torch.zeros(4, 4), 1.5)


@pytest.mark.gpu
@pytest.mark.parametrize("block_rows", [2 ** 32 + 1, 2 ** 32 + 128, -2 ** 32 + 1])
def test_block_rows_beyond_32_bits_are_refused_on_the_gpu(block_rows):
    n0 = L.load().kda_launch_count()
    with pytest.raises(ValueError, match="block_rows"):
        K.quant_fp8(torch.zeros(300, 256, device="cuda"), block_rows)
    assert L.load().kda_launch_count() == n0
