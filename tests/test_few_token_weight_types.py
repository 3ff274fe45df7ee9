"""moe.Weight takes the e4m3 tensors that the staged calls take: as bytes or as torch's float8_e4m3fn."""
import pytest
import torch

import combine_expert_histogram_amd as moe


@pytest.mark.parametrize("fmt,scale", [("e4m3", torch.ones((2, 1, 2))), ("e4m3_mx", torch.zeros((2, 2, 128), dtype=torch.int32))])
def test_e4m3_weights_of_both_types(fmt, scale):
    data = torch.randn((2, 128, 256)).to(torch.float8_e4m3fn)
    for d in (data, data.view(torch.uint8)):
        w = moe.Weight(fmt, 128, 256, d, scale, experts=2)
        assert w.data.data_ptr() == data.data_ptr()
    for dtype in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int8):
        with pytest.raises(ValueError):
            moe.Weight(fmt, 128, 256, data.view(dtype), scale, experts=2)


@pytest.mark.parametrize("fmt,scale", [("e2m1_mx", torch.zeros((1, 128), dtype=torch.int32)),
                                       ("int4", torch.ones((1, 128, 1), dtype=torch.bfloat16))])
def test_four_bit_codes_are_bytes(fmt, scale):
    data = torch.zeros((128, 64), dtype=torch.uint8)
    moe.Weight(fmt, 128, 128, data, scale)
    with pytest.raises(ValueError):
        moe.Weight(fmt, 128, 128, data.view(torch.float8_e4m3fn), scale)
