"""Element types of the few-token layer's binding, without a GPU: x and y are
bfloat16 or its bits; a float16 tensor has the same size and would be read as
other numbers."""
import pytest
import torch

from fp8_block_scaled_pow2_b200 import moe

T, H, I, E, K = 2, 256, 128, 8, 2


def call(x, y):
    p13 = torch.zeros(moe.moe_prepared_weights_size(E + 1, 2 * I, H), dtype=torch.uint8)
    p2 = torch.zeros(moe.moe_prepared_weights_size(E + 1, H, I), dtype=torch.uint8)
    moe.moe_layer_few_mxfp4(x, torch.zeros(T, E), p13, p2, I, torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K), y,
                            torch.zeros(1 << 16, dtype=torch.uint8))


@pytest.mark.parametrize("xt,yt", [(torch.float16, torch.bfloat16), (torch.bfloat16, torch.float16),
                                   (torch.float32, torch.bfloat16), (torch.bfloat16, torch.int32)])
def test_other_types_are_refused(xt, yt):
    with pytest.raises(ValueError, match="bfloat16"):
        call(torch.zeros(T, H, dtype=xt), torch.zeros(T, H, dtype=yt))


@pytest.mark.parametrize("xt,yt", [(torch.bfloat16, torch.bfloat16), (torch.int16, torch.uint16), (torch.uint16, torch.int16)])
def test_bfloat16_and_its_bits_pass_the_type_check(xt, yt):
    with pytest.raises(ValueError, match="CUDA"):                # the next refusal: tensors that are not on a GPU
        call(torch.zeros(T, H, dtype=xt), torch.zeros(T, H, dtype=yt))
