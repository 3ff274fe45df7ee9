"""Inputs and bounds shared by the few-token tests: random weights in every format, their exact float64 values, and
error bounds that count roundings."""
from __future__ import annotations

import numpy as np

from oracle import bf16 as obf16
from oracle import few_token as oft
from oracle import fp8, mx

# (format, group, with zero points)
FORMATS = [("e4m3", 128, False), ("e4m3_mx", 32, False), ("e2m1_mx", 32, False), ("int4", 128, False),
           ("int4", 128, True), ("int4", 64, True), ("int4", 32, False), ("int4", 32, True)]
FORMAT_IDS = [f"{f}_g{g}{'_z' if z else ''}" for f, g, z in FORMATS]

BF16_HALF = 2.0 ** -8       # torch.finfo(bfloat16).eps / 2: one rounding to bf16, relative
F32_HALF = 2.0 ** -24       # one rounding to fp32, relative


def random_weight(rng, fmt, group, with_zero, n, k, experts=1):
    """Random codes over the whole code space and scales that differ by group.  Returns (arguments of moe.Weight as
    numpy arrays, exact float64 [experts, n, k])."""
    nb = k // 128
    if fmt == "e4m3":
        data = rng.integers(0, 256, (experts, n, k)).astype(np.uint8)
        data[(data & 0x7F) == 0x7F] = 0x3A                      # no NaN codes
        scale = np.exp2(rng.uniform(-9, -6, (experts, n // 128, nb))).astype(np.float32)
        zero = None
    elif fmt == "int4":
        data = rng.integers(0, 256, (experts, n, k // 2)).astype(np.uint8)
        scale = obf16.from_f32(np.exp2(rng.uniform(-8, -5, (experts, nb, n, 128 // group))).astype(np.float32))
        zero = rng.integers(0, 16, scale.shape).astype(np.uint8) if with_zero else None
    else:
        data = rng.integers(0, 256, (experts, n, k if fmt == "e4m3_mx" else k // 2)).astype(np.uint8)
        if fmt == "e4m3_mx":
            data[(data & 0x7F) == 0x7F] = 0x3A
        lo = 127 - (14 if fmt == "e4m3_mx" else 9)
        codes = rng.integers(lo, lo + 5, (experts, nb, n, 4)).astype(np.uint8)
        scale, zero = mx.pack_codes(codes)[..., 0], None
    exact = np.stack([oft.dequant(fmt, data[e], obf16.to_f32(scale[e]) if fmt == "int4" else scale[e],
                                  None if zero is None else zero[e], group) for e in range(experts)])
    return dict(fmt=fmt, n=n, k=k, data=data, scale=scale, zero=zero, group=group, experts=experts), exact


def activations(rng, rows, cols):
    return obf16.from_f32(rng.standard_normal((rows, cols)).astype(np.float32))


def scale_elements(w, e):
    """[n, k] scale of each element of expert e of an int4 weight"""
    s = obf16.to_f32(w["scale"][e]).astype(np.float64)
    return s.transpose(1, 0, 2).reshape(w["n"], -1).repeat(w["group"], 1)


def fp32_error(w, e, x, exact):
    """Bound on the fp32 error of x @ exact.T, [rows, n], for expert e of a random_weight.

    The products are exact (8-bit significands); each partial sum is rounded at most once relative to a running size
    of at most sum |x w|, and the scales add a few more roundings.  A matrix instruction may truncate where it aligns
    its products, which is at most twice a rounding.  int4 sums (128 + q) x and takes (128 + zero) sum x off again,
    so the sizes there are up to 143 scales in each of the two sums instead of |q - zero| of them."""
    k = x.shape[1]
    if w["fmt"] == "int4":
        return 2 * F32_HALF * (k + 8) * 2 * 143 * (np.abs(x) @ scale_elements(w, e).T)
    return 2 * F32_HALF * (k + 4) * (np.abs(x) @ np.abs(exact).T)
