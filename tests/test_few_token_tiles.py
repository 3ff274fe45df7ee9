"""The strict comparison rejects what it has to (CPU): mistakes are planted in the float64 reference, rounded to bf16 as a
kernel would, for every product and layer that the GPU tests compare with it."""
import numpy as np
import pytest

import few_token_tiles as ft
from few_token_helpers import FORMAT_IDS, FORMATS, activations
from oracle import bf16 as obf16


def values(bits):
    return obf16.to_f32(bits).astype(np.float64)


def rounded(y):
    return values(obf16.from_f32(y.astype(np.float32)))


def rejected(got, exact, var, what, share=1.0):
    """share: of the tiles, at least.  A short piece of K adds little to a tile now and then."""
    r = ft.ratios(rounded(got), exact, var)
    live = ft.ratios(np.zeros_like(exact), exact, var) > 0       # tiles of tokens with an expert
    assert live.any() and (r[live] > 1).mean() >= share, (what, float(r[live].min()))


@pytest.mark.parametrize("fmt,group,z", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("k", sorted({k for _, _, k in ft.DEEP}))
def test_products(fmt, group, z, k):
    rng = np.random.default_rng(k)
    m, n = 4, 256
    _, part, exact, _ = ft.product_case(rng, fmt, group, z, m, n, k)
    x = values(activations(rng, m, k))
    y, var = x @ exact.T, ft.variance(part, 0, x, exact)
    assert (ft.ratios(rounded(y), y, var) <= 1).all()
    assert (ft.SIGMAS * np.sqrt(var) < 0.01 * np.abs(y).std()).all()
    rejected(0 * y, y, var, "zeros")
    rejected(-y, y, var, "sign")
    rejected(np.roll(y, 1, 0), y, var, "another token's")
    rejected(np.roll(y, ft.TILE, 1), y, var, "another tile's")
    for at in (0, k // 2, k - 32):
        keep = np.ones(k)
        keep[at:at + 32] = 0
        rejected((x * keep) @ exact.T, y, var, f"32 of K left out at {at}", 0.95)


@pytest.mark.parametrize("fmt,group,z", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("shape", [s for s, _ in ft.DEEP_LAYERS], ids=lambda s: "H%d_I%d_L%d_d%d" % s)
def test_layers(fmt, group, z, shape):
    """One or two experts a token; left out are a K block, and a scale group, of either product."""
    rng = np.random.default_rng(sum(shape))
    H, I, L, distinct = shape
    c = ft.layer_weights(rng, fmt, group, z, H, I, L, 1)
    T, E, e0, k = 2, L, 0, 1 if fmt == "int4" else 2
    x, ids, tw = ft.layer_tokens(rng, c, T, E, k)
    x = values(x)
    y, var = ft.layer_reference(c, x, ids, tw, e0)
    assert (ft.ratios(rounded(y), y, var) <= 1).all()
    rejected(0 * y, y, var, "zeros")
    rejected(-y, y, var, "sign")
    for length, share in ((128, 1.0), (32, 0.95)):
        keep_x, keep_h = np.ones(H), np.ones(I)
        keep_x[H // 2:H // 2 + length], keep_h[I // 2:I // 2 + length] = 0, 0
        left_out = f"{length} left out"
        rejected(ft.layer_reference(c, x, ids, tw, e0, keep_x=keep_x)[0], y, var, "of H: " + left_out, share)
        rejected(ft.layer_reference(c, x, ids, tw, e0, keep_h=keep_h)[0], y, var, "of I: " + left_out, share)
