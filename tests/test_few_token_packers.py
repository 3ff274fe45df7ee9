"""The packers (int4_weight, e2m1_weight) lay a weight out in memory of its own, for every view that they accept."""
import numpy as np
import pytest
import torch

import combine_expert_histogram_amd as moe
from oracle import bf16 as obf16
from oracle import few_token as oft


def off_by_one(t):
    """The same values in a view that starts one element into its storage."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


def int4_values(w):
    return oft.dequant("int4", w.data.numpy(), obf16.to_f32(w.scale.view(torch.int16).numpy().view(np.uint16)),
                       None if w.zero is None else w.zero.numpy(), w.group)


@pytest.mark.parametrize("k", [128, 256])
@pytest.mark.parametrize("group", [32, 128])
def test_int4_packer_takes_any_view_and_keeps_its_own_copy(k, group):
    rng = np.random.default_rng(k + group)
    q = torch.from_numpy(rng.integers(0, 16, (8, k)).astype(np.uint8))
    scale = torch.from_numpy(np.exp2(rng.integers(-8, 3, (8, k // group))).astype(np.float32)).to(torch.bfloat16)
    zero = torch.from_numpy(rng.integers(0, 16, (8, k // group)).astype(np.uint8))
    want = (q.double() - zero.double().repeat_interleave(group, 1)) * scale.double().repeat_interleave(group, 1)
    views = [off_by_one(t) for t in (q, scale, zero)]
    w = moe.int4_weight(*views)
    np.testing.assert_array_equal(int4_values(w), want.numpy())
    for t in views:                                              # the caller's tensors are free again
        t.zero_()
    np.testing.assert_array_equal(int4_values(w), want.numpy())


@pytest.mark.parametrize("k", [128, 256])
def test_e2m1_packer_takes_any_view_and_keeps_its_own_copy(k):
    rng = np.random.default_rng(k)
    codes = torch.from_numpy(rng.integers(0, 16, (8, k)).astype(np.uint8))
    e8m0 = torch.from_numpy(rng.integers(100, 140, (8, k // 32)).astype(np.uint8))
    want = oft.e2m1_decode(codes.numpy()) * np.exp2(e8m0.numpy().astype(np.float64) - 127).repeat(32, 1)
    views = [off_by_one(codes), off_by_one(e8m0)]
    w = moe.e2m1_weight(*views)
    values = lambda: oft.dequant("e2m1_mx", w.data.numpy(), w.scale.numpy().view(np.uint32))  # noqa: E731
    np.testing.assert_array_equal(values(), want)
    for t in views:
        t.zero_()
    np.testing.assert_array_equal(values(), want)


def test_int4_packer_refuses_zero_points_that_are_not_whole():
    q, s = torch.zeros((8, 128), dtype=torch.uint8), torch.ones((8, 4))
    whole = torch.full((8, 4), 7.0)
    assert (moe.int4_weight(q, s, whole).zero == 7).all()
    for value in (7.5, 0.25, float("nan"), float("inf")):
        bad = whole.clone()
        bad[3, 1] = value
        with pytest.raises(ValueError):
            moe.int4_weight(q, s, bad)
