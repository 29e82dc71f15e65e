"""The expert layers with a one-call path take rows of their own type, whatever the number of tokens. Refused before any
launch, so this runs on the host."""
import os

import pytest
import torch

from int4_weight_quantized_amd import ops
from int4_weight_quantized_amd.fp8_experts import Fp8Experts
from int4_weight_quantized_amd.mxfp4_experts import Mxfp4Experts

E, H, I, TOPK = 4, 128, 64, 2
U8 = torch.uint8


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(ops.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()


def mxfp4(dtype):
    return Mxfp4Experts(torch.zeros((E, 2 * I, H // 2), dtype=U8), torch.zeros((E, 2 * I, 4), dtype=U8),
                        torch.zeros((E, H, I // 2), dtype=U8), torch.zeros((E, H, 4), dtype=U8), TOPK, 16, dtype=dtype,
                        decode_tokens=4)


def fp8(dtype):
    return Fp8Experts(torch.zeros((E, 2 * I, H), dtype=U8), torch.zeros((E, 1, 1)), torch.zeros((E, H, I), dtype=U8),
                      torch.zeros((E, 1, 1)), TOPK, 16, dtype=dtype, decode_tokens=4)


@pytest.mark.parametrize("layer", [mxfp4, fp8])
@pytest.mark.parametrize("own", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 4, 5, 16])
def test_rows_of_another_type_are_refused(layer, own, T):
    run = layer(own)
    for other in (torch.bfloat16, torch.float16, torch.float32):
        if other != own:
            with pytest.raises(TypeError, match="the layer's type"):
                run(torch.zeros((T, H), dtype=other), torch.zeros((T, E)))
