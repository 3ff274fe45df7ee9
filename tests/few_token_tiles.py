"""Strict comparison of the few-token products with float64, tile by tile, and inputs of real depth for it.

A tile is one token's sixteen neighbouring outputs (a row tile of the kernels).  For each, the norm of the error has to
stay within

  2^-8 |y| + (1 + 2^-8) 6 s

where the first term is the one rounding of each output to bf16 (at most half a step, so it holds for any part of the
output), and s is the size of all roundings before it: s^2 sums, over the tile, the squares of the single roundings'
bounds.  Roundings of sums over random data have independent signs, and then (Hoeffding) a sum of errors bounded by s_i
passes 6 sqrt(sum s_i^2) once in 3e7 times; a tile's norm joins sixteen.  Unlike a bound that adds the roundings up,
s grows with the root of k as the outputs do, so it stays below a hundredth of them at any depth: a wrong sign, another
token's or tile's values or a K block left out show in every tile, a scale group of 32 left out in nearly every one (the
CPU tests plant them in the reference).
"""
from __future__ import annotations

import numpy as np

from few_token_helpers import BF16_HALF, F32_HALF, random_weight, scale_elements

SIGMAS = 6.0
TILE = 16
STEP = 2 * F32_HALF         # a matrix instruction may truncate where it aligns its products: twice a rounding


def tiled_weight(rng, fmt, group, with_zero, n, k, experts=1, rows=0, distinct=0):
    """A weight of n rows (and `experts` matrices) that repeats `rows` random rows and `distinct` random matrices, so that
    the float64 side stays small.  Returns (arguments of moe.Weight, arguments of the part, exact float64 [distinct,
    rows, k], row_of [n], expert_of [experts])."""
    rows, distinct = rows or n, distinct or experts
    part, exact = random_weight(rng, fmt, group, with_zero, rows, k, distinct)
    row_of, expert_of = np.arange(n) % rows, np.arange(experts) % distinct
    whole = dict(part, n=n, experts=experts, data=part["data"][expert_of][:, row_of])
    if fmt == "e4m3":
        whole["scale"] = part["scale"][expert_of][:, row_of[::128] // 128]
    else:
        whole["scale"] = part["scale"][expert_of][:, :, row_of]
        if with_zero:
            whole["zero"] = part["zero"][expert_of][:, :, row_of]
    return whole, part, exact, row_of, expert_of


def variance(w, e, x, exact):
    """Sum of the squares of the fp32 roundings in x @ exact.T, [rows, n].

    e4m3 and the e2m1 forms: k products are added into sums of at most sum |x w|, and eight wavefronts' sums.
    int4: in a group, g products are added into each of two sums of at most 143 scale sum |x| ((128 + q) x against
    (128 + zero) x), which two more operations put together; the groups are added into a sum of at most sum |x w|."""
    size = (np.abs(x) @ np.abs(exact).T) ** 2
    k = x.shape[1]
    if w["fmt"] != "int4":
        return (k + k // 128 + 8) * STEP ** 2 * size
    g = w["group"]
    in_group = np.abs(x).reshape(x.shape[0], -1, g).sum(2)
    scale = scale_elements(w, e)[:, ::g]
    return (2 * g + 2) * (STEP * 143) ** 2 * (in_group ** 2 @ (scale ** 2).T) + (k // g + 8) * STEP ** 2 * size


def ratios(got, exact, var):
    """The tiles' errors over what they may be, [tokens, tiles]; infinite where anything is not finite."""
    pad = (0, 0), (0, -exact.shape[1] % TILE)
    norm = lambda a: np.sqrt(np.pad(a, pad).reshape(a.shape[0], -1, TILE).sum(2))  # noqa: E731
    err = norm((got - exact) ** 2)
    allowed = BF16_HALF * norm(exact ** 2) + (1 + BF16_HALF) * SIGMAS * norm(var) + 2.0 ** -133
    return np.where(np.isfinite(err), err / allowed, np.inf)


# ---------------------------------------------------------------- products: m, n, k
# one, two and four row tiles to a wavefront with several blocks for each of the eight, each column form
DEEP = ([(m, 260, 128 * 41) for m in (1, 6, 16, 24, 64)] + [(m, 8196, 128 * 33) for m in (1, 6, 16, 24, 64)] +
        [(m, 16388, 128 * 33) for m in (1, 3, 6, 16, 24, 64)] + [(m, 16388, 128 * 41) for m in (1, 8, 64)] +
        # the wavefronts share the tokens: every slot of its rings is refilled
        [(m, 65540, 128 * kb) for kb in (5, 9) for m in (17, 64)] + [(32, 65540, 128 * 4), (100, 65540, 128 * 33)])


def product_case(rng, fmt, group, z, m, n, k):
    if fmt == "e4m3":
        n, rows = -(-n // 128) * 128, 1408
    else:
        rows = 1236
    whole, part, exact, row_of, _ = tiled_weight(rng, fmt, group, z, n, k, rows=min(rows, n))
    return whole, part, exact[0], row_of


# ---------------------------------------------------------------- layers: weights (H, I, local experts, distinct ones)
# and (T, E, e0, k) over them
DEEP_LAYERS = [
    # 33 blocks of K in the first launch: two row tiles (1 token) and four, 4 to 32 columns
    ((4224, 512, 16, 3), [(1, 16, 0, 8), (8, 16, 0, 8), (16, 16, 0, 4), (64, 16, 0, 2), (64, 16, 0, 4)]),
    # four row tiles and one token; sixteen wavefronts in the second launch that start and end inside experts
    ((2432, 1024, 13, 3), [(1, 13, 0, 9), (11, 13, 0, 4), (24, 13, 0, 2), (64, 13, 0, 3)]),
    # two row tiles in the second launch, whose wavefronts cross from expert to expert; each of its column forms
    ((6144, 640, 13, 3), [(1, 13, 0, 7), (12, 13, 0, 7), (16, 26, 7, 4), (20, 13, 0, 1), (24, 13, 0, 2), (64, 13, 0, 3),
                          (64, 128, 50, 8), (64, 384, 3, 8)]),
]


def layer_weights(rng, fmt, group, z, H, I, L, distinct):
    w1, p1, x1, _, expert_of = tiled_weight(rng, fmt, group, z, 2 * I, H, L, distinct=distinct)
    w2, p2, x2, _, _ = tiled_weight(rng, fmt, group, z, H, I, L, distinct=distinct)
    return dict(w1=w1, p1=p1, x1=x1, w2=w2, p2=p2, x2=x2, expert_of=expert_of, H=H, I=I, L=L)


def layer_reference(c, x, ids, tw, e0, keep_x=None, keep_h=None):
    """The layer in float64 and the squares of its roundings, [T, H] each.  The plants of the CPU tests: keep_x and keep_h
    are masks over the inputs and over the intermediate values.

    gate and up carry the roundings of their products; |silu'| <= 1.1; the activation, whose exponential is good to a few
    roundings and whose argument's own rounding counts |gate| times (to 88), sixteen and |gate| of them; the weighted row
    one to bf16.  The second product adds its own."""
    x = x if keep_x is None else x * keep_x
    out, var = np.zeros((x.shape[0], c["H"])), np.zeros((x.shape[0], c["H"]))
    for le in range(c["L"]):
        rows = np.nonzero((ids == e0 + le).any(1))[0]
        if not len(rows):
            continue
        b = c["expert_of"][le]
        wt = np.where(ids[rows] == e0 + le, tw[rows].astype(np.float64), 0).sum(1)[:, None]
        gu, vg = x[rows] @ c["x1"][b].T, variance(c["p1"], b, x[rows], c["x1"][b])
        gate, up = gu[:, :c["I"]], gu[:, c["I"]:]
        silu = gate / (1 + np.exp(-gate))
        h = silu * up * wt
        if keep_h is not None:
            h = h * keep_h
        vh = wt ** 2 * ((1.1 * up) ** 2 * vg[:, :c["I"]] + silu ** 2 * vg[:, c["I"]:])
        vh += (((16 + np.minimum(np.abs(gate), 88)) * STEP) ** 2 + BF16_HALF ** 2) * h ** 2
        out[rows] += h @ c["x2"][b].T
        var[rows] += vh @ (c["x2"][b] ** 2).T + variance(c["p2"], b, h, c["x2"][b])
    return out, var


def layer_tokens(rng, c, T, E, k):
    from few_token_helpers import activations
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    return activations(rng, T, c["H"]), ids, rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
