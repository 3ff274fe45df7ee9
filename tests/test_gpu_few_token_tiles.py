"""GPU: the few-token products and layers at real depth, tile by tile against float64 (few_token_tiles states the bound)."""
import functools

import numpy as np
import pytest

import combine_expert_histogram_amd as moe
import few_token_tiles as ft
from few_token_helpers import FORMAT_IDS, FORMATS, activations
from gpu_helpers import dev, host_u16, require_gpu, say
from oracle import bf16 as obf16

pytestmark = pytest.mark.gpu


def values(bits):
    return obf16.to_f32(bits).astype(np.float64)


def to_gpu(w):
    bits = {np.dtype(np.uint32): np.int32, np.dtype(np.uint16): np.int16}
    scale = w["scale"].view(bits.get(w["scale"].dtype, w["scale"].dtype))
    return moe.Weight(w["fmt"], w["n"], w["k"], dev(w["data"]), dev(scale),
                      zero=None if w["zero"] is None else dev(w["zero"]), group=w["group"], experts=w["experts"])


def check(got, exact, var, what):
    r = ft.ratios(got, exact, var)
    say(f"{what}: worst tile {r.max():.3f} of what it may be")
    assert (r <= 1).all(), (what, np.argwhere(r > 1)[:8].tolist())


# ---------------------------------------------------------------- products
@pytest.mark.parametrize("fmt,group,z", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("m,n,k", ft.DEEP)
def test_deep_products(fmt, group, z, m, n, k):
    require_gpu()
    rng = np.random.default_rng(m + n + k)
    w, part, exact, row_of = ft.product_case(rng, fmt, group, z, m, n, k)
    x = activations(rng, m, k)
    xv = values(x)
    got = values(host_u16(moe.matvec(dev(x.view(np.int16)), to_gpu(w))))
    check(got, (xv @ exact.T)[:, row_of], ft.variance(part, 0, xv, exact)[:, row_of], f"{fmt} g{group} {m}x{w['n']}x{k}")


# ---------------------------------------------------------------- layers
@functools.lru_cache(maxsize=1)
def layer_weights(f, shape):
    c = ft.layer_weights(np.random.default_rng(sum(shape)), *FORMATS[f], *shape)
    return c, to_gpu(c["w1"]), to_gpu(c["w2"])


def run_layer(c, g1, g2, x, ids, tw, E, e0):
    d = moe.Dims(S=1, Ts=x.shape[0], k=ids.shape[1], E=E, e0=e0, L=c["L"], H=c["H"])
    return values(host_u16(moe.few_token_layer(d, c["I"], dev(x.view(np.int16)), dev(ids), dev(tw), g1, g2)))


@pytest.mark.parametrize("f,shape,tokens", [(f, s, t) for f in range(len(FORMATS)) for s, ts in ft.DEEP_LAYERS for t in ts],
                         ids=lambda p: FORMAT_IDS[p] if isinstance(p, int) else "_".join(str(v) for v in p))
def test_deep_layers(f, shape, tokens):
    require_gpu()
    c, g1, g2 = layer_weights(f, shape)
    T, E, e0, k = tokens
    x, ids, tw = ft.layer_tokens(np.random.default_rng(sum(tokens)), c, T, E, k)
    out, var = ft.layer_reference(c, values(x), ids, tw, e0)
    check(run_layer(c, g1, g2, x, ids, tw, E, e0), out, var, f"layer {FORMAT_IDS[f]} {shape} {tokens}")


@pytest.mark.parametrize("f", [i for i, (fmt, _, _) in enumerate(FORMATS) if fmt == "int4"], ids=lambda f: FORMAT_IDS[f])
def test_int4_layer_of_ordinary_size(f):
    """Hidden 7168, intermediate 2048: one token and sixteen, over one matrix that eight experts repeat."""
    require_gpu()
    shape = (7168, 2048, 8, 1)
    c, g1, g2 = layer_weights(f, shape)
    for T in (1, 16):
        x, ids, tw = ft.layer_tokens(np.random.default_rng(T), c, T, 8, 8 // T or 1)
        out, var = ft.layer_reference(c, values(x), ids, tw, 0)
        check(run_layer(c, g1, g2, x, ids, tw, 8, 0), out, var, f"layer {FORMAT_IDS[f]} {shape} T={T}")
