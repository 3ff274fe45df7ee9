"""GPU: the router's top-k, the matrix-vector products and the few-token layer against float64, with error bounds that
count roundings."""
import math

import numpy as np
import pytest
import torch

import combine_expert_histogram_amd as moe
from few_token_helpers import (BF16_HALF, F32_HALF, FORMAT_IDS, FORMATS, activations, fp32_error, random_weight,
                               scale_elements)
from gpu_helpers import dev, host_u16, require_gpu, say
from oracle import bf16 as obf16
from oracle import few_token as oft

pytestmark = pytest.mark.gpu

POISON = 0x5A5A


def to_gpu(w):
    scale = w["scale"]
    scale = scale.view(np.int32) if scale.dtype == np.uint32 else scale.view(np.int16) if scale.dtype == np.uint16 else scale
    return moe.Weight(w["fmt"], w["n"], w["k"], dev(w["data"]), dev(scale),
                      zero=None if w["zero"] is None else dev(w["zero"]), group=w["group"], experts=w["experts"])


def values(bits):
    return obf16.to_f32(bits).astype(np.float64)


def check(got, exact, bound, what):
    """|got - exact| <= bound + one bf16 rounding of a value within bound of exact"""
    err = np.abs(got - exact)
    allowed = bound + BF16_HALF * (np.abs(exact) + bound) + 2.0 ** -133
    worst = float((err / allowed).max()) if err.size else 0.0
    say(f"{what}: worst error {worst:.3f} of the bound")
    assert bool(np.isfinite(got).all()) and worst <= 1.0, what


# ---------------------------------------------------------------- matvec
MATVEC_SHAPES = [(1, 128, 128), (1, 4096, 1024), (2, 4, 128), (3, 20, 1152), (15, 260, 256), (16, 128, 2048),
                 (17, 36, 640), (31, 128, 128), (33, 132, 384), (64, 68, 256), (65, 16, 128), (130, 44, 384)]


@pytest.mark.parametrize("fmt,group,z", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("m,n,k", MATVEC_SHAPES)
def test_matvec(fmt, group, z, m, n, k):
    require_gpu()
    n = -(-n // 128) * 128 if fmt == "e4m3" else n
    rng = np.random.default_rng(m * 1000 + n + k)
    w, exact = random_weight(rng, fmt, group, z, n, k)
    x = activations(rng, m, k)
    got = values(host_u16(moe.matvec(dev(x.view(np.int16)).view(torch.bfloat16), to_gpu(w))))
    xv = values(x)
    check(got, xv @ exact[0].T, fp32_error(w, 0, xv, exact[0]), f"matvec {fmt} g{group} {m}x{n}x{k}")


# wide matrices: more row tiles to a wavefront, and the form that shares tokens (65536 rows and more than 16 tokens)
WIDE_SHAPES = [(1, 8200, 128), (6, 8192, 384), (13, 16388, 128), (16, 20000, 256), (24, 16400, 256), (40, 8204, 128),
               (64, 16384, 256), (17, 65540, 128), (33, 65536, 384), (64, 65792, 256), (100, 65536, 128)]


@pytest.mark.parametrize("fmt,group,z", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("m,n,k", WIDE_SHAPES)
def test_matvec_of_many_rows(fmt, group, z, m, n, k):
    require_gpu()
    n = -(-n // 128) * 128 if fmt == "e4m3" else n
    rng = np.random.default_rng(m + n + k)
    w, exact = random_weight(rng, fmt, group, z, n, k)
    x = activations(rng, m, k)
    y = torch.full((m + 2, n), POISON, dtype=torch.int16, device="cuda")
    moe.matvec(dev(x.view(np.int16)), to_gpu(w), out=y[1:m + 1])
    xv = values(x)
    check(values(host_u16(y[1:m + 1])), xv @ exact[0].T, fp32_error(w, 0, xv, exact[0]),
          f"matvec {fmt} g{group} {m}x{n}x{k}")
    assert (y[[0, m + 1]] == POISON).all()


@pytest.mark.parametrize("fmt,group,z", FORMATS, ids=FORMAT_IDS)
def test_matvec_picks_every_element(fmt, group, z):
    """x = unit vectors: y is column j of the weight, rounded once, for every j."""
    require_gpu()
    rng = np.random.default_rng(3)
    n, k = 128, 256
    w, exact = random_weight(rng, fmt, group, z, n, k)
    eye = obf16.from_f32(np.eye(k, dtype=np.float32))
    got = host_u16(moe.matvec(dev(eye.view(np.int16)), to_gpu(w)))
    want = obf16.from_f32(exact[0].T.astype(np.float32))
    np.testing.assert_array_equal(values(got), values(want))


@pytest.mark.parametrize("fmt,group,z", [FORMATS[0], FORMATS[2], FORMATS[4]], ids=["e4m3", "e2m1", "int4"])
@pytest.mark.parametrize("m", [1, 5, 40, 67])
def test_matvec_strides(fmt, group, z, m):
    """Rows of x and y inside wider tensors: the gaps are neither read nor written."""
    require_gpu()
    rng = np.random.default_rng(m)
    n, k = 128, 384
    w, exact = random_weight(rng, fmt, group, z, n, k)
    x = activations(rng, m, k)
    wide = torch.full((m, k + 24), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + k] = dev(x.view(np.int16)).view(torch.bfloat16)
    y = torch.full((m + 1, n + 20), POISON, dtype=torch.int16, device="cuda")
    moe.matvec(wide[:, 8:8 + k], to_gpu(w), out=y[:m, 4:4 + n])
    y = y.cpu().numpy().view(np.uint16)
    assert (y[:, :4] == POISON).all() and (y[:, 4 + n:] == POISON).all() and (y[m] == POISON).all()
    xv = values(x)
    check(values(y[:m, 4:4 + n]), xv @ exact[0].T, fp32_error(w, 0, xv, exact[0]), f"strided {fmt} m={m}")


def test_matvec_transposed_rows_are_refused():
    require_gpu()
    rng = np.random.default_rng(0)
    w = to_gpu(random_weight(rng, "e2m1_mx", 32, False, 128, 128)[0])
    x = torch.zeros((128, 2), dtype=torch.bfloat16, device="cuda")
    for bad in (x.t(), x, x.t().contiguous().float(), x.t().contiguous().half(), x.t().contiguous()[:, :64]):
        with pytest.raises(ValueError):
            moe.matvec(bad, w)
    with pytest.raises(moe.MoeError):       # rows that start off a 16-byte boundary
        moe.matvec(torch.zeros((2, 129), dtype=torch.bfloat16, device="cuda")[:, 1:], w)
    with pytest.raises(ValueError):
        moe.matvec(torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda"), w,
                   out=torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda"))


def test_matvec_no_rows():
    require_gpu()
    w = to_gpu(random_weight(np.random.default_rng(0), "e2m1_mx", 32, False, 128, 128)[0])
    assert moe.matvec(torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda"), w).shape == (0, 128)


def test_matvec_one_bad_row_stays_alone():
    """An infinity or a NaN in one row of x leaves the other rows as they are."""
    require_gpu()
    rng = np.random.default_rng(8)
    for fmt, group, z in FORMATS:
        w, _ = random_weight(rng, fmt, group, z, 128, 256)
        g = to_gpu(w)
        x = dev(activations(rng, 20, 256).view(np.int16)).view(torch.bfloat16)
        ref = moe.matvec(x, g)
        bad = x.clone()
        bad[3, 7], bad[17, 100] = math.inf, math.nan
        got = moe.matvec(bad, g)
        keep = [i for i in range(20) if i not in (3, 17)]
        assert torch.equal(got[keep], ref[keep])
        assert not torch.isfinite(got[3]).all() and torch.isnan(got[17]).all()


def test_e8m0_range():
    """Scales from 2^-100 to 2^100 (values inside bf16's range)."""
    require_gpu()
    rng = np.random.default_rng(4)
    n, k = 64, 256
    for fmt in ("e4m3_mx", "e2m1_mx"):
        w, _ = random_weight(rng, fmt, 32, False, n, k)
        codes = np.repeat(rng.integers(27, 228, (1, 1, n, 1)), 4, 3).repeat(k // 128, 1).astype(np.uint8)
        from oracle import mx
        w["scale"] = mx.pack_codes(codes)[..., 0]
        exact = oft.dequant(fmt, w["data"][0], w["scale"][0])
        x = activations(rng, 2, k)
        xv = values(x)
        got = values(host_u16(moe.matvec(dev(x.view(np.int16)), to_gpu(w))))
        check(got, xv @ exact.T, fp32_error(w, 0, xv, exact), f"{fmt} wide scales")


def test_matvec_past_32_bits():
    """A weight of more than 2^31 bytes and an output that starts past 2^31 elements: the last rows are what they are."""
    require_gpu()
    n, k, m = (1 << 17) + 128, 1 << 14, 2
    rng = np.random.default_rng(0)
    tail, exact = random_weight(rng, "e4m3_mx", 32, False, 128, k)
    data = torch.zeros((n, k), dtype=torch.uint8, device="cuda")
    data[-128:] = dev(tail["data"][0])
    scale = torch.zeros((k // 128, n), dtype=torch.int32, device="cuda")
    scale[:, -128:] = dev(tail["scale"][0].view(np.int32))
    x = activations(rng, m, k)
    got = moe.matvec(dev(x.view(np.int16)), moe.Weight("e4m3_mx", n, k, data, scale))
    xv = values(x)
    check(values(host_u16(got[:, -128:])), xv @ exact[0].T, fp32_error(tail, 0, xv, exact[0]), "far rows")
    assert not got[:, :-128].any()
    wide = torch.empty(((1 << 31) // 8192 + 8, 8192), dtype=torch.bfloat16, device="cuda")
    view = wide[-4:, :128]
    x4 = activations(rng, 4, 128)
    w, exact = random_weight(rng, "e2m1_mx", 32, False, 128, 128)
    moe.matvec(dev(x4.view(np.int16)), to_gpu(w), out=view)
    check(values(host_u16(view)), values(x4) @ exact[0].T, fp32_error(w, 0, values(x4), exact[0]), "far output")


# ---------------------------------------------------------------- the layer
def make_layer(rng, T, E, e0, L, k, H, I, f1, f2=None):
    w1, x1 = random_weight(rng, *f1, 2 * I, H, L)
    w2, x2 = random_weight(rng, *(f2 or f1), H, I, L)
    x = activations(rng, T, H)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    tw = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    return dict(d=moe.Dims(S=1, Ts=T, k=k, E=E, e0=e0, L=L, H=H), I=I, w1=w1, x1=x1, w2=w2, x2=x2, x=x, ids=ids, tw=tw)


def run_layer(c, **kw):
    return moe.few_token_layer(c["d"], c["I"], dev(c["x"].view(np.int16)), dev(c["ids"]), dev(c["tw"]),
                               to_gpu(c["w1"]), to_gpu(c["w2"]), **kw)


def check_layer(c, got, what):
    """The bound: gate and up carry fp32_error; h = silu(gate) up w carries |silu'| <= 1.1 of gate's and |silu| of
    up's, sixteen fp32 roundings (the hardware exponential is good to a few, and its argument's own rounding, up to
    |gate| of them, is counted at |gate| < 88), and one rounding to bf16; the second product adds fp32_error over all
    k experts' terms."""
    d, I, x = c["d"], c["I"], values(c["x"])
    out, bound = np.zeros((d.T, d.H)), np.zeros((d.T, d.H))
    for e in range(d.L):
        rows = np.nonzero((c["ids"] == d.e0 + e).any(1))[0]
        if not len(rows):
            continue
        wt = np.where(c["ids"][rows] == d.e0 + e, c["tw"][rows].astype(np.float64), 0).sum(1)[:, None]
        gu, eg = x[rows] @ c["x1"][e].T, fp32_error(c["w1"], e, x[rows], c["x1"][e])
        gate, up = gu[:, :I], gu[:, I:]
        silu = gate / (1 + np.exp(-gate))
        h = silu * up * wt
        eh = np.abs(wt) * (1.1 * eg[:, :I] * (np.abs(up) + eg[:, I:]) + np.abs(silu) * eg[:, I:])
        eh += (16 + np.minimum(np.abs(gate), 88)) * 2 * F32_HALF * np.abs(h)
        eh += BF16_HALF * (np.abs(h) + eh)
        out[rows] += h @ c["x2"][e].T
        bound[rows] += eh @ np.abs(c["x2"][e]).T + d.k * fp32_error(c["w2"], e, np.abs(h) + eh, c["x2"][e])
    check(values(host_u16(got)), out, bound, what)


LAYERS = [  # T, E, e0, L, k, H, I
    (1, 8, 0, 8, 2, 256, 128), (1, 16, 4, 8, 8, 128, 256), (2, 8, 0, 8, 1, 384, 128), (7, 64, 32, 32, 8, 256, 384),
    (16, 8, 0, 8, 3, 128, 128), (17, 40, 3, 33, 5, 256, 128), (33, 8, 0, 8, 2, 128, 256), (64, 8, 2, 5, 2, 256, 128),
    (64, 300, 0, 300, 4, 128, 128), (65, 8, 0, 8, 2, 128, 128), (150, 16, 8, 8, 4, 128, 128),
    # many busy row tiles (two and four to a wavefront) and hidden sizes from 6144 (two in the down projection)
    (8, 32, 0, 32, 8, 128, 384), (8, 32, 0, 32, 8, 128, 512), (30, 40, 0, 40, 4, 128, 512), (64, 64, 0, 64, 8, 128, 256),
    (1, 2, 0, 2, 2, 6144, 128), (12, 2, 0, 2, 1, 6272, 128), (21, 3, 1, 2, 2, 6144, 128), (64, 2, 0, 2, 1, 6144, 128)]


@pytest.mark.parametrize("fmt,group,z", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: "T%d_E%d_e%d_L%d_k%d_H%d_I%d" % s)
def test_layer(fmt, group, z, shape):
    require_gpu()
    c = make_layer(np.random.default_rng(sum(shape)), *shape, (fmt, group, z))
    check_layer(c, run_layer(c), f"layer {fmt} g{group} {shape}")


@pytest.mark.parametrize("f1,f2", [(0, 2), (2, 4), (7, 1), (3, 0)])
def test_layer_of_two_formats(f1, f2):
    require_gpu()
    c = make_layer(np.random.default_rng(f1), 9, 12, 2, 9, 4, 256, 256, FORMATS[f1], FORMATS[f2])
    check_layer(c, run_layer(c), f"layer {FORMATS[f1]} {FORMATS[f2]}")


def test_layer_odd_ids():
    """Padding (-1), ids of other ranks, ids far outside, and a token that names one expert more than once."""
    require_gpu()
    c = make_layer(np.random.default_rng(2), 20, 16, 4, 8, 4, 128, 128, FORMATS[0])
    ids = c["ids"]
    ids[0] = -1
    ids[1] = 15
    ids[2] = 5
    ids[3] = [6, 7, 6, -1]
    ids[4] = [2 ** 31 - 1, -2 ** 31, 4, 11]
    ids[5] = [3, 12, 3, 12]
    c["tw"][2] = [0.5, -0.25, 0.125, 0.0]
    got = run_layer(c)
    check_layer(c, got, "odd ids")
    assert not got[[0, 1, 5]].any()


@pytest.mark.parametrize("fmt,group,z", FORMATS, ids=FORMAT_IDS)
@pytest.mark.parametrize("E", [2, 64], ids=["E2", "E64"])
def test_layer_every_token_names_one_expert(fmt, group, z, E):
    """64 tokens for one expert, where 32 or 2 are expected: further passes over its weights."""
    require_gpu()
    c = make_layer(np.random.default_rng(E), 64, E, 0, 2, 1, 128, 256, (fmt, group, z))
    c["ids"][:] = 1
    check_layer(c, run_layer(c), f"one expert of {E}")
    c["ids"][::3] = 0
    c["ids"][5:9] = -1
    check_layer(c, run_layer(c), f"two experts of {E}")


@pytest.mark.parametrize("f", [0, 2, 4], ids=lambda f: FORMAT_IDS[f])
@pytest.mark.parametrize("shape", [(64, 64, 0, 64, 64, 128, 128), (64, 64, 3, 2, 64, 6144, 128), (64, 64, 3, 2, 64, 128, 128),
                                   (32, 64, 3, 2, 64, 128, 128), (16, 1024, 0, 1024, 64, 128, 128)],
                         ids=lambda s: "T%d_E%d_e%d_L%d_k%d_H%d_I%d" % s)
def test_layer_at_the_largest_top_k(f, shape):
    require_gpu()
    c = make_layer(np.random.default_rng(sum(shape)), *shape, FORMATS[f])
    check_layer(c, run_layer(c), f"top-64 {FORMATS[f]} {shape}")


@pytest.mark.parametrize("T,k", [(1, 64), (17, 5), (64, 64)])
def test_layer_one_expert_in_every_slot(T, k):
    """Every slot of every token names the same expert: one product a token, with the summed weights."""
    require_gpu()
    c = make_layer(np.random.default_rng(T), T, 64, 5, 3, k, 128, 128, FORMATS[2])
    c["ids"][:] = 6
    c["tw"] /= k
    check_layer(c, run_layer(c), f"T={T} k={k}")


def test_layer_of_a_far_expert():
    """The last of 1024 experts, whose weights start past 2^31 bytes."""
    require_gpu()
    rng = np.random.default_rng(1)
    L, H, I = 1024, 4224, 256
    c = make_layer(rng, 3, L, L - 1, 1, 2, H, I, FORMATS[1])
    c["ids"][:, 0] = L - 1
    whole = []
    for w in (c["w1"], c["w2"]):
        data = torch.zeros((L, w["n"], w["k"]), dtype=torch.uint8, device="cuda")
        scale = torch.zeros((L, w["k"] // 128, w["n"]), dtype=torch.int32, device="cuda")
        data[-1], scale[-1] = dev(w["data"][0]), dev(w["scale"][0].view(np.int32))
        whole.append(moe.Weight("e4m3_mx", w["n"], w["k"], data, scale, experts=L))
    assert whole[0].data[:-1].numel() > 1 << 31
    d = moe.Dims(S=1, Ts=3, k=2, E=L, e0=0, L=L, H=H)
    got = moe.few_token_layer(d, I, dev(c["x"].view(np.int16)), dev(c["ids"]), dev(c["tw"]), *whole)
    check_layer(c, got, "far expert")       # the other ids name experts of zeros


def test_layer_nothing_local():
    require_gpu()
    c = make_layer(np.random.default_rng(2), 40, 16, 4, 8, 4, 128, 128, FORMATS[2])
    c["ids"][:] = -1
    out = torch.full((40, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    assert not run_layer(c, out=out).any()


def test_layer_no_tokens():
    require_gpu()
    c = make_layer(np.random.default_rng(2), 0, 16, 4, 8, 4, 128, 128, FORMATS[2])
    c["x"], c["ids"], c["tw"] = np.zeros((1, 128), np.uint16), np.zeros((1, 4), np.int32), np.zeros((1, 4), np.float32)
    assert run_layer(c).shape == (0, 128)


def test_layer_one_bad_token_stays_alone():
    """A NaN token, and NaN weights of an expert that only it names, leave the other tokens as they are."""
    require_gpu()
    for f in (0, 2, 4):
        c = make_layer(np.random.default_rng(5), 24, 8, 0, 8, 2, 128, 128, FORMATS[f])
        c["ids"][c["ids"] == 7] = 6
        c["ids"][5] = [7, 1]
        ref = run_layer(c)
        c["x"][5] = 0x7FC0
        got = run_layer(c)
        keep = [i for i in range(24) if i != 5]
        assert torch.equal(got[keep], ref[keep]) and torch.isnan(got[5]).all()


def test_layer_batches_and_stale_workspace():
    """Each token's output does not depend on the batch it came in, nor on what the workspace held."""
    require_gpu()
    c = make_layer(np.random.default_rng(6), 70, 8, 0, 8, 2, 256, 128, FORMATS[2])
    d = c["d"]
    ws = moe.alloc_few_token_workspace(d, c["I"])
    ws.fill_(0xFF)                              # NaN patterns
    whole = run_layer(c, ws=ws)
    check_layer(c, whole, "70 tokens")
    ws.fill_(0x7F)
    assert torch.equal(run_layer(c, ws=ws), whole)
    out = torch.full((72, 256), POISON, dtype=torch.int16, device="cuda")
    run_layer(c, out=out[1:71], ws=ws)
    assert torch.equal(out[1:71].view(torch.bfloat16), whole)
    assert (out[[0, 71]] == POISON).all()       # rows around the output


def test_layer_binding_refusals():
    require_gpu()
    c = make_layer(np.random.default_rng(1), 4, 8, 0, 8, 2, 128, 128, FORMATS[2])
    d, I = c["d"], c["I"]
    x, ids, tw = dev(c["x"].view(np.int16)), dev(c["ids"]), dev(c["tw"])
    w1, w2 = to_gpu(c["w1"]), to_gpu(c["w2"])
    for bad in ((d, I, x.float(), ids, tw, w1, w2), (d, I, x, ids.long(), tw, w1, w2), (d, I, x, ids, tw.half(), w1, w2),
                (d, I, x, ids, tw, w2, w1), (d, I, x[:2], ids, tw, w1, w2), (d, I, x, ids[:2], tw, w1, w2),
                (d, I, x, ids, tw[:2], w1, w2), (d, I, x, ids.cpu(), tw, w1, w2),
                (moe.Dims(S=1, Ts=4, k=2, E=8, e0=0, L=7, H=128), I, x, ids, tw, w1, w2)):
        with pytest.raises(ValueError):
            moe.few_token_layer(*bad)
    with pytest.raises(moe.MoeError):
        moe.few_token_layer(d, I, x, ids, tw, w1, w2, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        moe.few_token_layer(d, I, x, ids, tw, w1, w2, out=torch.empty((3, 128), dtype=torch.bfloat16, device="cuda"))


# ---------------------------------------------------------------- the router
def check_route(x, k, renormalise, scale=1.0, stride=None):
    """ids exact; weights: an exponential's few fp32 roundings (the argument's own rounding among them, up to the
    distance from the top), a sum of at most E terms and a division."""
    T, E = x.shape
    want_ids, want_w = oft.route_topk(x.float().numpy(), k, renormalise, scale)
    g = x.cuda()
    if stride:
        wide = torch.full((T, stride), math.inf, dtype=x.dtype, device="cuda")
        wide[:, :E] = g
        g = wide[:, :E]
    d = moe.Dims(S=1, Ts=T, k=k, E=E, e0=0, L=E)
    ids, w = moe.route_topk(d, g, renormalise=renormalise, scale=scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    w = w.cpu().double().numpy()
    assert np.isfinite(w).all()
    err, allowed = np.abs(w - want_w), (E + 120) * 2 * F32_HALF * np.abs(want_w) + 2.0 ** -126
    assert (err <= allowed).all(), float((err / allowed).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("renormalise", [True, False], ids=["chosen", "all"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 7, 7), (5, 64, 6), (4, 65, 1), (33, 160, 6), (9, 200, 64),
                                   (6, 300, 16), (7, 513, 8), (2, 1024, 64), (501, 128, 8), (130, 17, 3)])
def test_route(dtype, renormalise, T, E, k):
    require_gpu()
    g = torch.Generator().manual_seed(T * E + k)
    check_route((3 * torch.randn((T, E), generator=g)).to(dtype), k, renormalise)


@pytest.mark.parametrize("renormalise", [True, False], ids=["chosen", "all"])
def test_route_ties_masks_and_infinities(renormalise):
    require_gpu()
    g = torch.Generator().manual_seed(9)
    for E in (8, 70, 256, 700):
        for dtype in (torch.float32, torch.bfloat16):
            x = torch.randint(-2, 3, (64, E), generator=g).to(dtype)             # ties everywhere
            x[1] = 0.0
            x[2, ::2], x[2, 1::2] = 0.0, -0.0
            x[3] = -math.inf
            x[4] = math.nan
            x[5] = -math.inf
            x[5, E // 2] = -3.0
            x[6, 1::3] = -math.inf
            x[7, ::3] = math.nan
            x[8, 2], x[8, E - 1] = math.inf, math.inf
            x[9] = torch.finfo(dtype).min
            x[10] = torch.finfo(dtype).max
            x[11, 1] = torch.finfo(dtype).max
            x[12] = -math.inf
            x[12, 3] = torch.finfo(dtype).min
            x[13] = math.inf
            check_route(x, 8 if E >= 8 else E, renormalise)


def test_route_strides_scale_and_dtypes():
    require_gpu()
    g = torch.Generator().manual_seed(2)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn((37, 65), generator=g).to(dtype)
        check_route(x, 6, True, scale=2.5, stride=71)
        check_route(x, 6, False, scale=-0.5, stride=65)
    d = moe.Dims(S=1, Ts=2, k=2, E=8, e0=0, L=8)
    x = torch.zeros((2, 8), device="cuda")
    for bad in (x.half(), x.double(), x[:1], x[:, :7], torch.zeros((8, 2), device="cuda").t()):
        with pytest.raises(ValueError):
            moe.route_topk(d, bad)
    with pytest.raises(ValueError):
        moe.route_topk(d, x, topk_ids=torch.zeros((2, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        moe.route_topk(d, x, topk_w=torch.zeros((2, 2), dtype=torch.float64, device="cuda"))
    assert moe.route_topk(moe.Dims(S=1, Ts=0, k=2, E=8, e0=0, L=8), x[:0])[0].shape == (0, 2)


def test_route_of_a_large_batch_matches_sorting():
    require_gpu()
    g = torch.Generator().manual_seed(3)
    x = torch.randn((16384, 256), generator=g).cuda()
    ids, w = moe.route_topk(moe.Dims(S=8, Ts=2048, k=8, E=256, e0=0, L=256), x)
    top, want = torch.sort(x.double(), dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), want[:, :8])
    torch.testing.assert_close(w.double(), torch.softmax(top[:, :8], 1), rtol=400 * F32_HALF, atol=0)


# ---------------------------------------------------------------- together
def make_block(rng, T):
    """A decode step's MoE block: router logits from a product, the choice, the experts, and a shared expert."""
    c = make_layer(rng, T, 16, 0, 16, 4, 256, 128, FORMATS[2])
    gate, gate_exact = random_weight(rng, "int4", 128, True, 16, 256)
    shared, shared_exact = random_weight(rng, "int4", 64, True, 256, 256)
    return c, (gate, gate_exact), (shared, shared_exact)


def test_the_calls_together_captured_and_replayed():
    """Router product -> choice -> expert layer, with a shared expert's product beside it, on a side stream: eager,
    then captured once and replayed with new tokens and eager work in between."""
    require_gpu()
    rng = np.random.default_rng(12)
    T = 13
    c, (gate, gate_exact), (shared, shared_exact) = make_block(rng, T)
    d, I = c["d"], c["I"]
    g_gate, g_shared, w1, w2 = to_gpu(gate), to_gpu(shared), to_gpu(c["w1"]), to_gpu(c["w2"])
    x = dev(c["x"].view(np.int16)).view(torch.bfloat16)
    logits = torch.empty((T, 16), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((T, 4), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, 4), dtype=torch.float32, device="cuda")
    out = torch.empty((T, 256), dtype=torch.bfloat16, device="cuda")
    side = torch.empty((T, 256), dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_few_token_workspace(d, I)

    def step():
        moe.matvec(x, g_gate, out=logits)
        moe.route_topk(d, logits, renormalise=True, topk_ids=ids, topk_w=tw)
        moe.few_token_layer(d, I, x, ids, tw, w1, w2, out=out, ws=ws)
        moe.matvec(x, g_shared, out=side)

    def check_step(what):
        xv = values(host_u16(x))
        check(values(host_u16(logits)), xv @ gate_exact[0].T, fp32_error(gate, 0, xv, gate_exact[0]), what + " logits")
        want_ids, want_w = oft.route_topk(logits.float().cpu().numpy(), 4, True)
        np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
        np.testing.assert_allclose(tw.cpu().numpy(), want_w, rtol=300 * F32_HALF)
        c["x"], c["ids"], c["tw"] = host_u16(x), ids.cpu().numpy(), tw.cpu().numpy()
        check_layer(c, out, what + " layer")
        check(values(host_u16(side)), xv @ shared_exact[0].T, fp32_error(shared, 0, xv, shared_exact[0]),
              what + " shared")

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    check_step("eager")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step()
    for rep in range(3):
        x.copy_(dev(activations(rng, T, 256).view(np.int16)).view(torch.bfloat16))
        for t in (logits, out, side):
            t.fill_(math.nan)
        ids.fill_(-7)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        check_step(f"replay {rep}")
        kept = [t.clone() for t in (logits, ids, tw, out, side)]
        step()                                              # the eager pass on the default stream: the same bits
        torch.cuda.synchronize()
        for a, b in zip(kept, (logits, ids, tw, out, side)):
            assert torch.equal(a, b)


def test_two_calls_at_once():
    """Two streams, each with its own workspace and output, over the same weights."""
    require_gpu()
    c = make_layer(np.random.default_rng(15), 16, 16, 0, 16, 4, 512, 256, FORMATS[2])
    d, I = c["d"], c["I"]
    x, ids, tw = dev(c["x"].view(np.int16)), dev(c["ids"]), dev(c["tw"])
    w1, w2 = to_gpu(c["w1"]), to_gpu(c["w2"])
    ref = moe.few_token_layer(d, I, x, ids, tw, w1, w2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(ref) for _ in range(2)]
    wss = [moe.alloc_few_token_workspace(d, I) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, out, ws in zip(streams, outs, wss):
            with torch.cuda.stream(s):
                moe.few_token_layer(d, I, x, ids, tw, w1, w2, out=out, ws=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_the_layer_agrees_with_the_staged_calls():
    """The few-token layer on the staged calls' own weights: layout, quant, GEMM1, act, GEMM2 and combine quantise the
    activations to fp8 twice, so the two agree to fp8's resolution."""
    require_gpu()
    import workloads
    w = workloads.get("tiny_t64_h256_e8")
    ids, wts = workloads.routing(w)
    x = dev(workloads.activations(w).view(np.int16))
    (q1, s1), (q2, s2) = workloads.weights(w), workloads.weights2(w)
    d, I = moe.Dims(S=w.S, Ts=w.Ts, k=w.k, E=w.E, e0=w.e0, L=w.L, H=w.H), w.N // 2
    ids_d, wts_d = dev(ids), dev(wts)
    q1, s1, q2, s2 = dev(q1), dev(s1), dev(q2), dev(s2)
    got = moe.few_token_layer(d, I, x, ids_d, wts_d, moe.Weight("e4m3", w.N, w.H, q1, s1, experts=w.L),
                              moe.Weight("e4m3", w.H, I, q2, s2, experts=w.L))
    lay = moe.route_layout(d, ids_d)
    q, qs = moe.quant_dispatch(d, x, lay)
    y = moe.grouped_gemm1(d, w.N, q, qs, lay, q1, s1)
    h, hs = moe.silu_mul_quant(d, I, y, lay)
    y2 = moe.grouped_gemm2(d, I, h, hs, lay, wts_d, q2, s2)
    staged = moe.combine(d, w.H, y2, lay["assign_row"], torch.ones_like(wts_d))
    a, s = got.double(), staged.double()
    rel = float((a - s).norm() / s.norm())
    # rms errors relative to a sum's own rms: each e4m3 rounding of an operand is at most 2^-4 of it and independent
    # of the others, so two quantised operands (x enters gate and up) leave at most sqrt(3) 2^-4 = 0.108
    say(f"few-token layer against the staged calls: rel-L2 {rel:.4f}")
    assert rel <= math.sqrt(3) * 2.0 ** -4
