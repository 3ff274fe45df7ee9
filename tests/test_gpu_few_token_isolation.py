"""GPU: what a token's batch, another token's values and another expert's weights may change in its output, and groups of
zeros whose scale is out of range."""
import numpy as np
import pytest
import torch

import combine_expert_histogram_amd as moe
import few_token_tiles as ft
from few_token_helpers import FORMAT_IDS, FORMATS, activations, random_weight
from gpu_helpers import dev, require_gpu
from oracle import mx
from test_gpu_few_token_tiles import check, layer_weights, run_layer, to_gpu, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3_mx", "e2m1_mx"])
def test_a_group_of_zeros_may_carry_any_e8m0_code(fmt):
    """The staged quantiser gives a group of zeros the code 0 (2^-127), outside the range of the others."""
    require_gpu()
    rng = np.random.default_rng(6)
    m, n, k = 5, 64, 512
    w, _ = random_weight(rng, fmt, 32, False, n, k)
    x = dev(activations(rng, m, k).view(np.int16))
    zeros = rng.integers(0, 2, (n, k // 32)).astype(bool)
    sign, per_group = (0x80, 32) if fmt == "e4m3_mx" else (0x88, 16)
    w["data"][0][zeros.repeat(per_group, 1)] &= sign             # zeros of either sign
    codes = np.array(mx.unpack_codes(np.ascontiguousarray(w["scale"][0].T)))
    outs = []
    for code in (127, 0, 1, 254):
        codes[zeros] = code
        w["scale"] = np.ascontiguousarray(mx.pack_codes(codes).T)[None]
        outs.append(moe.matvec(x, to_gpu(w)))
    assert torch.isfinite(outs[0]).all() and outs[0].any()
    for out in outs[1:]:
        assert torch.equal(out, outs[0])


@pytest.mark.parametrize("f", [0, 2, 4], ids=lambda f: FORMAT_IDS[f])
def test_a_token_in_other_batches(f):
    """A token's sums may be ordered otherwise in another batch; each batch is held to the same bound, and the same batch
    gives the same bits."""
    require_gpu()
    c, g1, g2 = layer_weights(f, (512, 640, 6, 6))
    x, ids, tw = ft.layer_tokens(np.random.default_rng(70), c, 70, 12, 3)
    out, var = ft.layer_reference(c, values(x), ids, tw, 4)
    for size in (70, 1, 5, 16, 33):
        parts = [slice(t, t + size) for t in range(0, 70, size)]
        once = [np.concatenate([run_layer(c, g1, g2, x[p], ids[p], tw[p], 12, 4) for p in parts]) for _ in range(2)]
        np.testing.assert_array_equal(once[0], once[1])
        check(once[0], out, var, f"{FORMAT_IDS[f]} batches of {size}")


# ---------------------------------------------------------------- one token's NaN weights
def spoil(w, e):
    """Every weight of matrix e a NaN."""
    if w["fmt"] == "int4":
        w["scale"][e] = 0x7FC0
    else:
        w["data"][e] = 0x7F


@pytest.mark.parametrize("f", [0, 1, 4, 7], ids=lambda f: FORMAT_IDS[f])
@pytest.mark.parametrize("T,H", [(3, 256), (12, 256), (40, 256), (64, 256), (1, 6144), (12, 6144), (40, 6144)])
def test_nan_weights_reach_only_the_tokens_that_name_them(f, T, H):
    """Expert 3 holds NaNs and only the last token names it; the others' experts come before and after it, in the same
    wavefronts of the second launch, with several passes where the tokens are many."""
    require_gpu()
    rng = np.random.default_rng(T + H)
    c = ft.layer_weights(rng, *FORMATS[f], H, 640, 8, 8)
    x, ids, tw = ft.layer_tokens(rng, c, T, 8, 3)
    for t in range(T):
        ids[t] = rng.permutation([0, 1, 2, 4, 5, 6, 7])[:3]
    ids[T - 1, 1] = 3
    ref = run_layer(c, to_gpu(c["w1"]), to_gpu(c["w2"]), x, ids, tw, 8, 0)
    assert np.isfinite(ref).all()
    for which in ("w1", "w2"):
        bad = dict(c[which], data=c[which]["data"].copy(), scale=c[which]["scale"].copy())
        spoil(bad, 3)
        g = {"w1": c["w1"], "w2": c["w2"], which: bad}
        got = run_layer(c, to_gpu(g["w1"]), to_gpu(g["w2"]), x, ids, tw, 8, 0)
        np.testing.assert_array_equal(got[:-1], ref[:-1])
        assert np.isnan(got[-1]).all()


@pytest.mark.parametrize("f", [0, 1, 4, 7], ids=lambda f: FORMAT_IDS[f])
@pytest.mark.parametrize("m,n", [(1, 256), (7, 256), (20, 256), (40, 256), (3, 65664), (20, 65664), (64, 65664)])
def test_a_nan_weight_row_stays_in_its_output(f, m, n):
    require_gpu()
    fmt, group, z = FORMATS[f]
    rng = np.random.default_rng(m + n)
    w, _, _, _, _ = ft.tiled_weight(rng, fmt, group, z, n, 384, rows=128 if fmt == "e4m3" else 36)
    x = dev(activations(rng, m, 384).view(np.int16))
    ref = moe.matvec(x, to_gpu(w))
    bad = dict(w, data=w["data"].copy(), scale=w["scale"].copy())
    rows = [5, 17, n - 1]
    if fmt == "int4":
        bad["scale"][0][1, rows, 0] = 0x7FC0
    else:
        bad["data"][0][rows, 200] = 0x7F
    got = moe.matvec(x, to_gpu(bad))
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.isfinite(ref).all() and torch.equal(got[:, keep], ref[:, keep])
    assert torch.isnan(got[:, rows]).all()
