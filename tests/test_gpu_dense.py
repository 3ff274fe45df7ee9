"""GPU: the linear and gated linear layers, forward and backward, against float64.  Whole-numbered inputs make every sum
exact, so those tests ask for the exact result rounded once, bit for bit; the others hold bounds that count roundings."""
import math

import pytest
import torch

import combine_expert_histogram_amd as moe
from dense_helpers import (ACTS, HALF, Output, act64, check_gated, check_gated_backward, check_linear, check_linear_backward,
                           generator, ids, inside, integers, linear_sizes, normal, same)
from gpu_helpers import require_gpu, say

pytestmark = pytest.mark.gpu

# how the matrices lie: (elements before a row, after it); (0, 0) takes what rows of whole 16 bytes allow
PLACES = [(0, 0), (8, 16), (0, 3), (1, 0)]


def placed(t, place):
    return t if place == (0, 0) else inside(t, place[1], place[0])


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("place", PLACES, ids=ids)
@pytest.mark.parametrize("size", linear_sizes(), ids=ids)
def test_linear_exact(size, place, dtype):
    require_gpu()
    m, n, k = size
    say(f"linear {size} {place} {dtype}")
    g = generator(m + 10 * n + 100 * k)
    x, w = integers(g, m, k, dtype), integers(g, n, k, dtype)
    bias, res = integers(g, 1, n, dtype, 9)[0], integers(g, m, n, dtype, 9)
    z64 = x.double() @ w.double().T
    y, z = Output(m, n, dtype, place[1], place[0]), Output(m, n, dtype, place[0], place[1])
    xp, wp = placed(x, place), placed(w, place)
    moe.linear(xp, wp, out=y.view)
    same(y.view, z64, "plain")
    moe.linear(xp, wp, bias=bias, act="relu", residual=placed(res, place), z=z.view, out=y.view)
    same(z.view, z64 + bias.double(), "z")
    same(y.view, act64(z64 + bias.double(), "relu")[0] + res.double(), "y")
    y.check_surroundings()
    z.check_surroundings()


# Few rows and many columns: the ones where a workgroup takes one, two or four tiles of 16 (of 2 x 8 gated), and where rows
# that start anywhere change over to square tiles; one tile short of each bound, and past it.
@pytest.mark.parametrize("place", PLACES, ids=ids)
@pytest.mark.parametrize("n", [4095, 8176, 8200, 16368, 16391])
@pytest.mark.parametrize("m", [1, 16, 17, 33, 49, 64])
def test_few_rows_exact(m, n, place):
    require_gpu()
    dtype = HALF[(m + n) % 2]
    say(f"few rows {m} {n} {place} {dtype}")
    g = generator(m + 10 * n)
    k, inter = 200, n // 2
    x, w = integers(g, m, k, dtype), integers(g, n, k, dtype)
    bias, res = integers(g, 1, n, dtype, 9)[0], integers(g, m, n, dtype, 9)
    z64 = x.double() @ w.double().T
    y, h = Output(m, n, dtype, place[1], place[0]), Output(m, inter, dtype, place[1], place[0])
    xp, wp = placed(x, place), placed(w, place)
    moe.linear(xp, wp, bias=bias, act="relu", residual=placed(res, place), out=y.view)
    same(y.view, act64(z64 + bias.double(), "relu")[0] + res.double(), "y")
    y.check_surroundings()
    h64 = act64(z64[:, :inter], "relu")[0] * z64[:, inter:2 * inter]
    assert float(h64.abs().max()) < 2 ** 16
    moe.gated_linear(xp, wp[:2 * inter], act="relu", out=h.view)
    same(h.view, h64, "h")
    h.check_surroundings()


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("place", PLACES, ids=ids)
@pytest.mark.parametrize("size", linear_sizes(), ids=ids)
def test_linear_backward_exact(size, place, dtype):
    require_gpu()
    m, n, k = size
    say(f"linear backward {size} {place} {dtype}")
    g = generator(m + 10 * n + 100 * k + 1)
    x, w, dy = integers(g, m, k, dtype), integers(g, n, k, dtype), integers(g, m, n, dtype)
    z = integers(g, m, n, dtype, 2)
    dx, dw = Output(m, k, dtype, place[1], place[0]), Output(n, k, dtype, place[0], place[1])
    xp, wp, dyp = placed(x, place), placed(w, place), placed(dy, place)
    for act in ("none", "relu"):
        dz = dy.double() * act64(z.double(), act)[1]
        _, _, db = moe.linear_backward(dyp, xp, wp, act=act, z=None if act == "none" else placed(z, place), dx=dx.view,
                                       dw=dw.view)
        same(dx.view, dz @ w.double(), act + " dx")
        same(dw.view, dz.T @ x.double(), act + " dw")
        same(db, dz.sum(0), act + " dbias")
    dx.check_surroundings()
    dw.check_surroundings()


def gated_sizes():
    return [(1, 1, 1), (1, 8, 8), (1, 2048, 7168), (2, 9, 65), (16, 64, 128), (17, 100, 1000), (33, 17, 127), (64, 136, 520),
            (65, 8, 8), (66, 31, 72), (100, 1, 37), (127, 65, 63), (128, 64, 64), (129, 72, 65), (200, 200, 1160),
            (256, 128, 2048), (70, 40, 8200), (300, 517, 257), (1000, 264, 136), (4096, 1800, 200)]


# dz and its column sums where the rows of a workgroup change: up to 64 rows, sixteen to a workgroup, and 128 workgroups
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("n", [8, 259, 520])
@pytest.mark.parametrize("m", [1, 15, 16, 17, 63, 64, 65, 80, 81, 2047, 2048, 2049, 4100])
def test_bias_gradient_exact(m, n, act):
    require_gpu()
    dtype = HALF[(m + n) % 2]
    say(f"bias gradient {m} {n} {act} {dtype}")
    g = generator(m + 10 * n)
    k = 24
    x, w, dy, z = integers(g, m, k, dtype), integers(g, n, k, dtype), integers(g, m, n, dtype), integers(g, m, n, dtype, 2)
    dz = dy.double() * act64(z.double(), act)[1]
    dx, dw, db = moe.linear_backward(dy, x, w, act=act, z=z)
    same(db, dz.sum(0), "dbias")
    same(dx, dz @ w.double(), "dx")
    same(dw, dz.T @ x.double(), "dw")


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("place", PLACES, ids=ids)
@pytest.mark.parametrize("size", gated_sizes(), ids=ids)
def test_gated_exact(size, place, dtype):
    require_gpu()
    m, inter, k = size
    say(f"gated {size} {place} {dtype}")
    g = generator(m + 10 * inter + 100 * k)
    x = integers(g, m, k, dtype) * (torch.rand((m, k), generator=g, device="cuda") < min(1.0, 600 / k)).to(dtype)
    w = integers(g, 2 * inter, k, dtype)
    gu64 = x.double() @ w.double().T
    h64 = act64(gu64[:, :inter], "relu")[0] * gu64[:, inter:]
    assert float(h64.abs().max()) < 2 ** 16
    h, gu = Output(m, inter, dtype, place[1], place[0]), Output(m, 2 * inter, dtype, place[0], place[1])
    xp, wp = placed(x, place), placed(w, place)
    moe.gated_linear(xp, wp, act="relu", out=h.view)
    same(h.view, h64, "h alone")
    h.view.fill_(5)
    moe.gated_linear(xp, wp, act="relu", out=h.view, gu=gu.view)
    same(h.view, h64, "h")
    same(gu.view, gu64, "gu")
    h.check_surroundings()
    gu.check_surroundings()


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("place", PLACES, ids=ids)
@pytest.mark.parametrize("size", gated_sizes(), ids=ids)
def test_gated_backward_exact(size, place, dtype):
    require_gpu()
    m, inter, k = size
    say(f"gated backward {size} {place} {dtype}")
    g = generator(m + 10 * inter + 100 * k + 1)
    x, w, dh = integers(g, m, k, dtype), integers(g, 2 * inter, k, dtype), integers(g, m, inter, dtype)
    gu = integers(g, m, 2 * inter, dtype, 3)
    a, da = act64(gu[:, :inter].double(), "relu")
    d = torch.cat((dh.double() * gu[:, inter:].double() * da, dh.double() * a), 1)
    dx, dw = Output(m, k, dtype, place[1], place[0]), Output(2 * inter, k, dtype, place[0], place[1])
    moe.gated_linear_backward(placed(dh, place), placed(x, place), placed(w, place), placed(gu, place), act="relu",
                              dx=dx.view, dw=dw.view)
    same(dx.view, d @ w.double(), "dx")
    same(dw.view, d.T @ x.double(), "dw")
    dx.check_surroundings()
    dw.check_surroundings()


REAL = [(1, 40, 200), (19, 72, 520), (64, 33, 47), (65, 64, 64), (130, 136, 264), (97, 131, 301)]


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", REAL, ids=ids)
def test_linear_activations(size, act, dtype):
    require_gpu()
    m, n, k = size
    g = generator(m + n)
    x, w = normal(g, m, k, dtype), normal(g, n, k, dtype, 3 / math.sqrt(k))
    bias, res = normal(g, 1, n, dtype)[0], normal(g, m, n, dtype)
    z = torch.empty((m, n), dtype=dtype, device="cuda")
    y = moe.linear(x, w, bias=bias, act=act, residual=res, z=z)
    say(f"linear {size} {act} {dtype}", check_linear(x, w, bias, act, res, z, y))


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", REAL, ids=ids)
def test_linear_backward_activations(size, act, dtype):
    require_gpu()
    m, n, k = size
    g = generator(m + n + 1)
    x, w, dy = normal(g, m, k, dtype), normal(g, n, k, dtype, 1 / math.sqrt(k)), normal(g, m, n, dtype)
    z = normal(g, m, n, dtype, 3)
    got = moe.linear_backward(dy, x, w, act=act, z=z)
    say(f"linear backward {size} {act} {dtype}", check_linear_backward(dy, x, w, act, z, *got))


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", REAL, ids=ids)
def test_gated_activations(size, act, dtype):
    require_gpu()
    m, inter, k = size
    g = generator(m + inter + 2)
    x, w = normal(g, m, k, dtype), normal(g, 2 * inter, k, dtype, 2 / math.sqrt(k))
    gu = torch.empty((m, 2 * inter), dtype=dtype, device="cuda")
    h = moe.gated_linear(x, w, act=act, gu=gu)
    say(f"gated {size} {act} {dtype}", check_gated(x, w, act, gu, h))
    dh = normal(g, m, inter, dtype)
    say(f"gated backward {size} {act} {dtype}",
        check_gated_backward(dh, x, w, gu, act, *moe.gated_linear_backward(dh, x, w, gu, act=act)))
