"""GPU: layer norm, forward and backward, against float64, with bounds that count roundings."""
import math

import pytest
import torch

import combine_expert_histogram_amd as moe
from dense_helpers import F32_HALF as F
from dense_helpers import (Output, check_norm, check_norm_backward, generator, ids, inside, normal)
from gpu_helpers import require_gpu, say

pytestmark = pytest.mark.gpu

TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32), (torch.float32, torch.float32)]
# one, two, four and eight wavefronts' rows, every number of pieces, whole and ragged ones, rows read again
SIZES = [(1, 1), (1, 7), (3, 8), (5, 63), (9, 512), (4, 513), (6, 1024), (1, 1111), (13, 1536), (7, 2048), (3, 2049), (2, 4096),
         (5, 5000), (1, 7168), (6, 8192), (3, 8193), (2, 16384), (3, 16385), (2, 40000), (777, 1111), (1030, 72), (2100, 136),
         (600, 4104)]
EPS = 1e-5
# rows to change the number of the backward pass's workgroups
LONG = [(512, 2049), (513, 2049), (8191, 520), (8192, 520), (8192, 2560)]


def stream(g, rows, cols, dtype):
    """rows of different size with an offset, and a few large channels"""
    channel = torch.ones(cols, device="cuda")
    channel[:: 97] = 12.0
    x = (torch.randn((rows, cols), generator=g, device="cuda") * channel + 0.5)
    return (x * torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))).to(dtype)


def parameters(g, cols, p):
    return (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(p), torch.randn(cols, generator=g, device="cuda").to(p)


@pytest.mark.parametrize("types", TYPES, ids=lambda t: ids(t))
@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_forward(size, types):
    require_gpu()
    rows, cols = size
    T, P = types
    g = generator(rows + cols)
    x = stream(g, rows, cols, T)
    w, b = parameters(g, cols, P)
    mean = torch.full((rows,), math.nan, device="cuda")
    rstd = torch.full((rows,), math.nan, device="cuda")
    y = moe.layer_norm(x, w, b, eps=EPS, mean=mean, rstd=rstd)
    worst = check_norm(x, w, b, EPS, y, mean, rstd, str(size))
    say(f"norm {size} {types}: {worst:.3f} of the bound")
    for lead, pad in ((0, 3), (1, 0), (8, 8)):
        out = Output(rows, cols, T, pad, lead)
        moe.layer_norm(inside(x, pad, lead), w, b, eps=EPS, out=out.view)
        assert torch.equal(out.view, y)
        out.check_surroundings()
    check_norm(x, None, None, EPS, moe.layer_norm(x, eps=EPS), None, None, "no parameters")
    check_norm(x, w, None, 0.5, moe.layer_norm(x, w, eps=0.5), None, None, "no bias")
    check_norm(x, None, b, EPS, moe.layer_norm(x, None, b, eps=EPS), None, None, "no weight")
    same = x.clone()
    moe.layer_norm(same, w, b, eps=EPS, out=same)
    assert torch.equal(same, y), "in place"


@pytest.mark.parametrize("types", TYPES, ids=lambda t: ids(t))
@pytest.mark.parametrize("size", SIZES + LONG, ids=ids)
def test_backward(size, types):
    require_gpu()
    rows, cols = size
    T, P = types
    g = generator(rows + cols + 1)
    say(f"norm backward {size} {types}")
    x, dy = stream(g, rows, cols, T), normal(g, rows, cols, T)
    w, b = parameters(g, cols, P)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    moe.layer_norm(x, w, b, eps=EPS, mean=mean, rstd=rstd)
    ws = moe.alloc_layer_norm_backward_workspace(rows, cols).fill_(0xFF)
    dx, dw, db = moe.layer_norm_backward(dy, x, w, mean, rstd, ws=ws)
    assert dw.dtype == P and db.dtype == P and dx.dtype == T
    check_norm_backward(dy, x, w, mean, rstd, dx, dw, db, str(size))
    for lead, pad in ((0, 3), (1, 0), (8, 8)):
        out = Output(rows, cols, T, pad, lead)
        again = moe.layer_norm_backward(inside(dy, lead, pad), inside(x, pad, lead), w, mean, rstd, dx=out.view)
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))
        out.check_surroundings()
    none = moe.layer_norm_backward(dy, x, None, mean, rstd, bias=False)
    assert none[1] is None and none[2] is None
    check_norm_backward(dy, x, None, mean, rstd, none[0], None, None, "no weight")
    only = moe.layer_norm_backward(dy, x, None, mean, rstd)
    assert torch.equal(only[0], none[0]) and only[2].dtype == T
    check_norm_backward(dy, x, None, mean, rstd, None, None, only[2], "bias alone")
    part = torch.empty_like(dw)
    moe.moe_layer_norm_backward(dy, x, w, mean, rstd, None, part, None, ws)
    assert torch.equal(part, dw), "dweight alone"
    for which in (0, 1):
        both = [dy.clone(), x.clone()]
        got = moe.layer_norm_backward(both[0], both[1], w, mean, rstd, dx=both[which])
        assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db))), "in place"


def test_gradients_are_the_slopes():
    """Differences of the float32 forward pass, over a loss sum(y * t)."""
    require_gpu()
    rows, cols, h = 6, 37, 2.0 ** -7
    g = generator(4)
    x, t = normal(g, rows, cols, torch.float32), normal(g, rows, cols, torch.float32)
    w, b = parameters(g, cols, torch.float32)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    moe.layer_norm(x, w, b, mean=mean, rstd=rstd)
    grads = moe.layer_norm_backward(t, x, w, mean, rstd)

    def loss(*p):
        return float((moe.layer_norm(*p).double() * t.double()).sum())

    values = [x, w, b]
    for which, grad in enumerate(grads):
        for at in [(0,) * grad.dim(), tuple(s - 1 for s in grad.shape), tuple(s // 2 for s in grad.shape)]:
            moved = []
            for s in (h, -h):
                v = [p.clone() for p in values]
                v[which][at] += s
                moved.append(loss(*v))
            # the third derivative of a norm of 37 values of size 1 is below 10 |t| |w|: h^2 / 6 of it; the loss, rows * cols
            # terms of size 1 with relative errors of 64 half steps, over 2 h
            slack = 10 * h * h / 6 * 8 + rows * cols * 64 * F / h
            assert abs((moved[0] - moved[1]) / (2 * h) - float(grad[at])) <= slack, (which, at)


def test_a_constant_row_and_large_offsets():
    """No spread: y is the bias.  An offset of 1000 spreads: the variance comes from centred values."""
    require_gpu()
    g = generator(5)
    w, b = parameters(g, 4096, torch.float32)
    x = torch.full((3, 4096), 7.25, device="cuda")
    assert torch.equal(moe.layer_norm(x, w, b), b.expand(3, -1))
    x = 1000.0 + torch.randn((5, 4096), generator=g, device="cuda")
    check_norm(x, w, b, EPS, moe.layer_norm(x, w, b), None, None, "offset")


def test_bad_rows_stay_alone():
    require_gpu()
    for cols in (64, 5000, 16384, 20000):
        g = generator(cols)
        x = normal(g, 9, cols, torch.bfloat16)
        ref = moe.layer_norm(x)
        bad = x.clone()
        bad[3, 5], bad[7, cols - 1], bad[8, 0] = math.nan, math.inf, -math.inf
        got = moe.layer_norm(bad)
        keep = [0, 1, 2, 4, 5, 6]
        assert torch.equal(got[keep], ref[keep])
        assert bool(torch.isnan(got[[3, 7, 8]]).all())


def test_no_rows():
    require_gpu()
    for T, P in TYPES:
        x = torch.zeros((0, 24), dtype=T, device="cuda")
        w = torch.ones(24, dtype=P, device="cuda")
        s = torch.zeros(0, device="cuda")
        assert moe.layer_norm(x, w, mean=s, rstd=s).shape == (0, 24)
        dw, db = torch.full((24,), 3.0, dtype=P, device="cuda"), torch.full((24,), 3.0, dtype=P, device="cuda")
        dx, _, _ = moe.layer_norm_backward(x, x, w, s, s, dweight=dw, dbias=db)
        assert dx.shape == (0, 24) and not dw.any() and not db.any()


def test_far_rows():
    """The last rows start past 2^31 elements."""
    require_gpu()
    g = generator(6)
    rows, cols, step = 5, 640, 1 << 30
    wide = torch.empty(step * 4 // 2 + 4096, dtype=torch.float32, device="cuda").view(torch.bfloat16)
    far = wide.as_strided((rows, cols), (step, 1))
    x = normal(g, rows, cols, torch.bfloat16)
    w, b = parameters(g, cols, torch.float32)
    ref = moe.layer_norm(x, w, b)
    far.copy_(x)
    assert torch.equal(moe.layer_norm(far, w, b), ref)
    moe.layer_norm(x, w, b, out=far)
    assert torch.equal(far, ref)


@pytest.mark.parametrize("rows,cols", [((1 << 22) + 5, 3), ((1 << 20) + 3, 2056), ((1 << 20) + 3, 16392)], ids=ids)
def test_many_rows(rows, cols):
    """More rows than one launch has workgroups for."""
    require_gpu()
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    g = generator(rows)
    at = torch.tensor([0, 1, 1 << 20, rows - 2, rows - 1], device="cuda")
    x[at] = normal(g, 5, cols, torch.bfloat16)
    mean, rstd = torch.full((rows,), math.nan, device="cuda"), torch.full((rows,), math.nan, device="cuda")
    moe.layer_norm(x, out=x, mean=mean, rstd=rstd)
    g = generator(rows)
    small = normal(g, 5, cols, torch.bfloat16)
    m, r = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    assert torch.equal(x[at], moe.layer_norm(small, mean=m, rstd=r))
    assert torch.equal(mean[at], m) and torch.equal(rstd[at], r)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[at] = False
    assert not x.any(1)[keep].any() and not mean[keep].any()
    assert bool((rstd[keep] == rstd[2]).all()) and abs(float(rstd[2]) * math.sqrt(EPS) - 1) < 8 * F


@pytest.mark.parametrize("cols", [1 << 25, (1 << 25) + 36, 1 << 29], ids=ids)
def test_many_columns(cols):
    """More columns' sums than one launch has workgroups for: 2^20 of 64, and past 2^32 threads.  With a mean of 0 and an
    rstd of 1 a single row's gradients are products of two 16-bit numbers, exact in fp32."""
    require_gpu()
    say(f"columns {cols}")
    g = generator(cols % 1000)
    x = torch.randint(-128, 129, (1, cols), generator=g, device="cuda", dtype=torch.int16).to(torch.bfloat16)
    dy = torch.randint(-128, 129, (1, cols), generator=g, device="cuda", dtype=torch.int16).to(torch.bfloat16)
    dw, db = torch.full((cols,), math.nan, device="cuda"), torch.full((cols,), math.nan, device="cuda")
    ws = moe.alloc_layer_norm_backward_workspace(1, cols)
    moe.moe_layer_norm_backward(dy, x, None, torch.zeros(1, device="cuda"), torch.ones(1, device="cuda"), None, dw, db, ws)
    assert torch.equal(dw, x[0].float() * dy[0].float())
    assert torch.equal(db, dy[0].float())
