"""GPU: the dense layers as a program uses them: a block of them with the routed experts beside it, forward and backward,
captured and replayed; streams; large and far operands; rows and columns that spoil nothing but themselves; refusals."""
import math

import pytest
import torch

import combine_expert_histogram_amd as moe
from dense_helpers import (HALF, Output, act64, check_gated, check_gated_backward, check_linear, check_linear_backward,
                           check_norm, check_norm_backward, generator, ids, integers, normal, same)
from gpu_helpers import require_gpu, say

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- a block, forward and backward
class Block:
    """norm -> shared expert (gate and up, down) added to the routed experts' combined output, and back."""

    def __init__(self, g, T, H, I, dtype, act):
        self.T, self.H, self.I, self.dtype, self.act = T, H, I, dtype, act
        new = lambda *shape, t=dtype: torch.full(shape, math.nan, dtype=t, device="cuda")  # noqa: E731
        self.nw, self.nb = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")), 0.1 * torch.randn(H, generator=g, device="cuda")
        self.w1, self.w2 = normal(g, 2 * I, H, dtype, 1 / math.sqrt(H)), normal(g, H, I, dtype, 1 / math.sqrt(I))
        self.b2 = normal(g, 1, H, dtype, 0.1)[0]
        self.x, self.dout, self.routed = new(T, H), new(T, H), new(T, H)
        self.n, self.mean, self.rstd = new(T, H), new(T, t=torch.float32), new(T, t=torch.float32)
        self.gu, self.h, self.out = new(T, 2 * I), new(T, I), new(T, H)
        self.dh, self.dw2, self.db2 = new(T, I), new(H, I), new(H)
        self.dn, self.dw1 = new(T, H), new(2 * I, H)
        self.dx, self.dnw, self.dnb = new(T, H), new(H, t=torch.float32), new(H, t=torch.float32)
        self.ws = torch.full((max(moe.moe_linear_workspace(T, H, I), moe.moe_gated_linear_workspace(T, I, H),
                                  moe.moe_linear_backward_workspace(T, H, I, "none"),
                                  moe.moe_gated_linear_backward_workspace(T, I, H),
                                  moe.moe_layer_norm_backward_workspace(T, H)),), 0xFF, dtype=torch.uint8, device="cuda")

    def outputs(self):
        return [self.n, self.mean, self.rstd, self.gu, self.h, self.out, self.dh, self.dw2, self.db2, self.dn, self.dw1, self.dx,
                self.dnw, self.dnb]

    def new_inputs(self, g):
        self.x.copy_(torch.randn((self.T, self.H), generator=g, device="cuda") + 0.3)
        self.dout.copy_(torch.randn((self.T, self.H), generator=g, device="cuda"))
        self.routed.copy_(torch.randn((self.T, self.H), generator=g, device="cuda"))

    def step(self):
        """One workspace for all of them: one stream, one after the other."""
        moe.layer_norm(self.x, self.nw, self.nb, out=self.n, mean=self.mean, rstd=self.rstd)
        moe.gated_linear(self.n, self.w1, act=self.act, gu=self.gu, out=self.h, ws=self.ws)
        moe.linear(self.h, self.w2, bias=self.b2, residual=self.routed, out=self.out, ws=self.ws)
        moe.linear_backward(self.dout, self.h, self.w2, dx=self.dh, dw=self.dw2, dbias=self.db2, ws=self.ws)
        moe.gated_linear_backward(self.dh, self.n, self.w1, self.gu, act=self.act, dx=self.dn, dw=self.dw1, ws=self.ws)
        moe.layer_norm_backward(self.dn, self.x, self.nw, self.mean, self.rstd, dx=self.dx, dweight=self.dnw, dbias=self.dnb,
                                ws=self.ws)

    def check(self, what):
        check_norm(self.x, self.nw, self.nb, 1e-5, self.n, self.mean, self.rstd, what)
        check_gated(self.n, self.w1, self.act, self.gu, self.h)
        check_linear(self.h, self.w2, self.b2, "none", self.routed, None, self.out)
        check_linear_backward(self.dout, self.h, self.w2, "none", None, self.dh, self.dw2, self.db2)
        check_gated_backward(self.dh, self.n, self.w1, self.gu, self.act, self.dn, self.dw1)
        check_norm_backward(self.dn, self.x, self.nw, self.mean, self.rstd, self.dx, self.dnw, self.dnb, what)
        say(f"{what}: every step within its bound")


@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("shape", [(1, 136, 72), (37, 256, 128), (150, 333, 201), (700, 512, 264)], ids=ids)
def test_block_captured_and_replayed(shape, dtype):
    """Eager on a side stream, then captured once and replayed with new inputs and eager work in between; every replay is
    the eager pass bit for bit."""
    require_gpu()
    g = generator(sum(shape))
    b = Block(g, *shape, dtype, "silu")
    b.new_inputs(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.step()
    torch.cuda.synchronize()
    b.check(f"eager {shape}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            b.step()
    for rep in range(3):
        b.new_inputs(g)
        for t in b.outputs():
            t.fill_(math.nan)
        b.ws.fill_(0xFF)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in b.outputs()]
        b.check(f"replay {rep}")
        for t in b.outputs():
            t.fill_(math.nan)
        b.step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, b.outputs()))


def test_block_beside_the_routed_experts():
    """The shared expert's output added to what moe_combine gives: the staged calls and the dense layers on one batch."""
    require_gpu()
    import workloads
    from gpu_helpers import dev
    import numpy as np
    w = workloads.get("tiny_t64_h256_e8")
    id_, wts = workloads.routing(w)
    x = dev(workloads.activations(w).view(np.int16)).view(torch.bfloat16)
    (q1, s1), (q2, s2) = workloads.weights(w), workloads.weights2(w)
    d, I = moe.Dims(S=w.S, Ts=w.Ts, k=w.k, E=w.E, e0=w.e0, L=w.L, H=w.H), w.N // 2
    g = generator(3)
    nw, nb = torch.ones(w.H, device="cuda"), torch.zeros(w.H, device="cuda")
    n = moe.layer_norm(x, nw, nb)
    lay = moe.route_layout(d, dev(id_))
    q, qs = moe.quant_dispatch(d, n, lay)
    y = moe.grouped_gemm1(d, w.N, q, qs, lay, dev(q1), dev(s1))
    h, hs = moe.silu_mul_quant(d, I, y, lay)
    y2 = moe.grouped_gemm2(d, I, h, hs, lay, dev(wts), dev(q2), dev(s2))
    routed = moe.combine(d, w.H, y2, lay["assign_row"], torch.ones_like(dev(wts)))
    ws1, ws2 = normal(g, 2 * I, w.H, torch.bfloat16, 0.05), normal(g, w.H, I, torch.bfloat16, 0.05)
    shared = moe.gated_linear(n, ws1)
    out = moe.linear(shared, ws2, residual=routed)
    check_norm(x, nw, nb, 1e-5, n, None, None, "norm")
    check_gated(n, ws1, "silu", None, shared)
    check_linear(shared, ws2, None, "none", routed, None, out)


# ---------------------------------------------------------------- slopes
@pytest.mark.parametrize("m", [3, 70])
def test_gradients_are_the_slopes(m):
    """Differences of the forward pass, over a loss sum(y * t).  Without an activation the linear layer is linear and the
    gated one quadratic in each of its arguments, and whole numbers this small are exact: so are central differences."""
    require_gpu()
    g = generator(m)
    k, n = 5, 6
    x, w, t = (integers(g, *s, torch.bfloat16, 2) for s in ((m, k), (n, k), (m, n)))
    wg, tg = integers(g, 2 * n, k, torch.bfloat16, 1), integers(g, m, n, torch.bfloat16, 2)
    dx, dw, db = moe.linear_backward(t, x, w)
    gu = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda")
    moe.gated_linear(x, wg, act="none", gu=gu)
    dxg, dwg = moe.gated_linear_backward(tg, x, wg, gu, act="none")
    bias = torch.zeros(n, dtype=torch.bfloat16, device="cuda")

    def slope(f, value, at):
        up, down = value.clone(), value.clone()
        up[at] += 1
        down[at] -= 1
        return (f(up) - f(down)) / 2

    linear = lambda x, w, b: float((moe.linear(x, w, bias=b).double() * t.double()).sum())  # noqa: E731
    gated = lambda x, w: float((moe.gated_linear(x, w, act="none").double() * tg.double()).sum())  # noqa: E731
    for at in [(0, 0), (m - 1, k - 1), (m // 2, 2)]:
        assert slope(lambda v: linear(v, w, bias), x, at) == float(dx[at])
        assert slope(lambda v: gated(v, wg), x, at) == float(dxg[at])
    for at in [(0, 0), (n - 1, k - 1), (3, 2)]:
        assert slope(lambda v: linear(x, v, bias), w, at) == float(dw[at])
    for at in [(0, 0), (2 * n - 1, k - 1), (n, 2), (n - 1, 4)]:
        assert slope(lambda v: gated(x, v), wg, at) == float(dwg[at])
    for at in (0, n - 1):
        assert slope(lambda v: linear(x, w, v), bias, at) == float(db[at])


# ---------------------------------------------------------------- large, deep and far
@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("size", [(4096, 4096, 7168), (2048, 7168, 2112), (2049, 7176, 2056)], ids=ids)
def test_real_sizes_exact(size, dtype):
    """256 x 256 tiles, several of them to a workgroup, at real depths: whole numbers, the exact result rounded once."""
    require_gpu()
    m, n, k = size
    g = generator(k)
    x, w, dy = integers(g, m, k, dtype), integers(g, n, k, dtype), integers(g, m, n, dtype)
    ws = moe.alloc_linear_backward_workspace(m, n, k).fill_(0xFF)
    res = integers(g, m, n, dtype, 50)
    y = Output(m, n, dtype)
    moe.linear(x, w, residual=res, out=y.view)
    same(y.view, x.double() @ w.double().T + res.double(), "y")
    y.check_surroundings()
    dx, dw = Output(m, k, dtype), Output(n, k, dtype)
    _, _, db = moe.linear_backward(dy, x, w, dx=dx.view, dw=dw.view, ws=ws)
    same(dx.view, dy.double() @ w.double(), "dx")
    same(dw.view, dy.double().T @ x.double(), "dw")
    same(db, dy.double().sum(0), "dbias")
    dx.check_surroundings()
    dw.check_surroundings()
    inter = n // 2
    sparse = x * (torch.rand((m, k), generator=g, device="cuda") < 0.05).to(dtype)
    h, gu = Output(m, inter, dtype), Output(m, 2 * inter, dtype)
    moe.gated_linear(sparse, w, act="relu", out=h.view, gu=gu.view)
    gu64 = sparse.double() @ w.double().T
    same(gu.view, gu64, "gu")
    same(h.view, act64(gu64[:, :inter], "relu")[0] * gu64[:, inter:], "h")
    h.check_surroundings()
    gu.check_surroundings()


def test_far_operands():
    """Rows that start past 2^31 elements, in and out, with few rows and with tiles."""
    require_gpu()
    g = generator(9)
    step, n, k = (1 << 22) - 8, 40, 72
    for m in (60, 600):
        space = torch.empty(step * (m - 1) + 256, dtype=torch.bfloat16, device="cuda")
        far = space.as_strided((m, k), (step, 1))
        assert m < 512 or step * (m - 1) > 1 << 31
        x, w, dy = integers(g, m, k, torch.bfloat16), integers(g, n, k, torch.bfloat16), integers(g, m, n, torch.bfloat16)
        far.copy_(x)
        same(moe.linear(far, w), x.double() @ w.double().T, "x far")
        same(moe.linear_backward(dy, far, w)[1], dy.double().T @ x.double(), "dw of a far x")
        moe.linear_backward(dy, x, w, dx=far)
        same(far, dy.double() @ w.double(), "dx far")
        out = space.as_strided((m, n), (step, 1))
        moe.linear(x, w, residual=dy, out=out)
        same(out, x.double() @ w.double().T + dy.double(), "y far")
        out.copy_(dy)
        moe.linear(x, w, residual=out, out=out)
        same(out, x.double() @ w.double().T + dy.double(), "in place")
        del space, far, out


def test_many_weight_rows():
    """A vocabulary's worth of them for one token and for a few, and weights of more than 2^31 bytes."""
    require_gpu()
    g = generator(10)
    n, k = 1 << 19, 2056
    w = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
    w[-100:] = integers(g, 100, k, torch.bfloat16)
    for m in (1, 20, 70):
        x = integers(g, m, k, torch.bfloat16)
        y = moe.linear(x, w)
        same(y[:, -100:], x.double() @ w[-100:].double().T, "far rows")
        assert not y[:, :-100].any()


# ---------------------------------------------------------------- what spoils what
@pytest.mark.parametrize("m", [20, 300])
@pytest.mark.parametrize("k", [264, 201])
def test_bad_rows_and_columns_stay_alone(m, k):
    require_gpu()
    g = generator(m + k)
    n = 72
    x, w, dy = normal(g, m, k, torch.bfloat16), normal(g, n, k, torch.bfloat16), normal(g, m, n, torch.bfloat16)
    z = normal(g, m, n, torch.bfloat16)
    ref, gref = moe.linear(x, w), moe.gated_linear(x, w)
    rb = moe.linear_backward(dy, x, w, act="gelu", z=z)
    bad = x.clone()
    bad[3, 5], bad[m - 1, k - 1] = math.nan, math.inf
    keep = [i for i in range(m) if i not in (3, m - 1)]
    y, h = moe.linear(bad, w), moe.gated_linear(bad, w)
    assert torch.equal(y[keep], ref[keep]) and torch.equal(h[keep], gref[keep])
    assert bool(torch.isnan(y[3]).all()) and not bool(torch.isfinite(y[m - 1]).any())
    worse = w.clone()
    worse[7, 0] = math.nan
    y, h = moe.linear(x, worse), moe.gated_linear(x, worse)
    cols = [i for i in range(n) if i != 7]
    assert torch.equal(y[:, cols], ref[:, cols]) and bool(torch.isnan(y[:, 7]).all())
    cols = [i for i in range(n // 2) if i != 7]
    assert torch.equal(h[:, cols], gref[:, cols]) and bool(torch.isnan(h[:, 7]).all())
    # a spoiled gradient: its token's dx, its column's dw and dbias
    sick = dy.clone()
    sick[4, 9] = math.nan
    dx, dw, db = moe.linear_backward(sick, x, w, act="gelu", z=z)
    rows, cols = [i for i in range(m) if i != 4], [i for i in range(n) if i != 9]
    assert torch.equal(dx[rows], rb[0][rows]) and bool(torch.isnan(dx[4]).all())
    assert torch.equal(dw[cols], rb[1][cols]) and bool(torch.isnan(dw[9]).all())
    assert torch.equal(db[cols], rb[2][cols]) and bool(torch.isnan(db[9]))


def test_infinite_gradients_stay_infinite():
    """Not turned into NaNs by the two terms in which up to 64 tokens' gradients are held."""
    require_gpu()
    x, w = torch.ones((2, 8), dtype=torch.bfloat16, device="cuda"), torch.ones((8, 8), dtype=torch.bfloat16, device="cuda")
    dy, z = torch.ones((2, 8), dtype=torch.bfloat16, device="cuda"), torch.full((2, 8), 50.0, dtype=torch.bfloat16, device="cuda")
    dy[1, 3] = math.inf
    dx, dw, db = moe.linear_backward(dy, x, w, act="silu", z=z)
    assert bool((dx[1] == math.inf).all()) and bool(torch.isfinite(dx[0]).all())
    assert bool((dw[3] == math.inf).all()) and float(db[3]) == math.inf
    x = torch.ones((2, 8), dtype=torch.float16, device="cuda")
    gu = torch.full((2, 8), 300.0, dtype=torch.float16, device="cuda")       # 300 * 300 does not fit
    dx, dw = moe.gated_linear_backward(torch.full((2, 4), 300.0, dtype=torch.float16, device="cuda"), x, x.new_ones((8, 8)), gu)
    assert bool((dx == math.inf).all()) and bool((dw == math.inf).all())


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activations_of_extreme_values(act):
    """+-0, the type's largest and smallest values: no NaN where the formula has none."""
    require_gpu()
    f = torch.finfo(torch.bfloat16)
    v = torch.tensor([0.0, -0.0, f.tiny, -f.tiny, 1e-30, -1e-30, 88.0, -88.0, 200.0, -200.0, 1e10, -1e10, 1e25, -1e25, f.max / 4,
                      -f.max / 4], dtype=torch.bfloat16, device="cuda")[:, None]
    one = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda")
    y, dx = moe.linear(v, one, act=act), moe.linear_backward(torch.ones_like(v), v, one, act=act, z=v, bias=False)[0]
    a, d = act64(v.double(), act)
    # where z^3 overflows, the reference's z * s * (1 - s) * z^2 is inf * 0: the derivative there is 0 or 1
    d = torch.where(v.double().abs() > 1e3, (v > 0).double(), d)
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(dx).all())
    assert bool(((y.double() - a).abs() <= a.abs() * 2.0 ** -8 + 1e-20).all())
    assert bool(((dx.double() - d).abs() <= d.abs() * 2.0 ** -8 + 1e-20).all())


# ---------------------------------------------------------------- calls beside each other
def test_two_streams():
    require_gpu()
    g = generator(12)
    m, n, k = 300, 264, 2048
    x, w, dy, z = (normal(g, *s, torch.bfloat16) for s in ((m, k), (n, k), (m, n), (m, n)))
    run = lambda ws: (moe.linear(x, w, act="silu", ws=ws), moe.gated_linear(x, w, ws=ws),  # noqa: E731
                      *moe.linear_backward(dy, x, w, act="silu", z=z, ws=ws))
    size = max(moe.moe_linear_backward_workspace(m, n, k, "silu"), moe.moe_linear_workspace(m, n, k),
               moe.moe_gated_linear_workspace(m, n // 2, k))
    wss = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ref = run(wss[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    kept = []
    for _ in range(10):
        for s, ws in zip(streams, wss):
            with torch.cuda.stream(s):
                kept.append(run(ws))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for out in kept for p, q in zip(out, ref))


@pytest.mark.parametrize("m", [5, 200])
def test_parts_of_the_gradients(m):
    """Each gradient alone is the one that the whole call gives; the operands that it does not need may be missing."""
    require_gpu()
    g = generator(m)
    n, k = 96, 136
    x, w, dy, z = (normal(g, *s, torch.float16) for s in ((m, k), (n, k), (m, n), (m, n)))
    dx, dw, db = moe.linear_backward(dy, x, w, act="gelu", z=z)
    ws = moe.alloc_linear_backward_workspace(m, n, k, "gelu").fill_(0xFF)
    a, b, c = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    moe.moe_linear_backward(dy, None, w, "gelu", z, a, None, None, ws)
    moe.moe_linear_backward(dy, x, None, "gelu", z, None, b, None, ws)
    moe.moe_linear_backward(dy, None, None, "gelu", z, None, None, c, ws)
    assert torch.equal(a, dx) and torch.equal(b, dw) and torch.equal(c, db)
    assert moe.linear_backward(dy, x, w, act="gelu", z=z, bias=False)[2] is None
    dh, gu = dy[:, :48].contiguous(), z
    dx, dw = moe.gated_linear_backward(dh, x, w, gu)
    ws = moe.alloc_gated_linear_backward_workspace(m, 48, k).fill_(0xFF)
    moe.moe_gated_linear_backward(dh, None, w, gu, "silu", a, None, ws)
    moe.moe_gated_linear_backward(dh, x, None, gu, "silu", None, b, ws)
    assert torch.equal(a, dx) and torch.equal(b, dw)


def test_no_rows():
    require_gpu()
    for dtype in HALF:
        x, w = torch.zeros((0, 24), dtype=dtype, device="cuda"), torch.ones((10, 24), dtype=dtype, device="cuda")
        y, gu = torch.zeros((0, 10), dtype=dtype, device="cuda"), torch.zeros((0, 10), dtype=dtype, device="cuda")
        assert moe.linear(x, w).shape == (0, 10) and moe.gated_linear(x, w).shape == (0, 5)
        dw, db = Output(10, 24, dtype, 3), torch.full((10,), 3.0, dtype=dtype, device="cuda")
        dx, _, _ = moe.linear_backward(y, x, w, dw=dw.view, dbias=db)
        assert dx.shape == (0, 24) and not dw.view.any() and not db.any()
        dw.check_surroundings()
        dx, dw = moe.gated_linear_backward(y[:, :5], x, w, gu)
        assert dx.shape == (0, 24) and dw.shape == (10, 24) and not dw.any()


def test_the_same_call_gives_the_same_bits():
    require_gpu()
    g = generator(14)
    m, n, k = 777, 392, 4104
    x, w, dy, z = (normal(g, *s, torch.bfloat16) for s in ((m, k), (n, k), (m, n), (m, n)))
    ref = (moe.linear(x, w), *moe.linear_backward(dy, x, w, act="gelu_tanh", z=z))
    for _ in range(5):
        got = (moe.linear(x, w), *moe.linear_backward(dy, x, w, act="gelu_tanh", z=z))
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


# ---------------------------------------------------------------- refusals
def test_refusals():
    require_gpu()
    x, w = torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda"), torch.zeros((6, 16), dtype=torch.bfloat16, device="cuda")
    y, v = torch.zeros((4, 6), dtype=torch.bfloat16, device="cuda"), torch.zeros(6, dtype=torch.bfloat16, device="cuda")
    s, wide = torch.zeros(4, device="cuda"), torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    for f in (lambda: moe.linear(x, w.half()), lambda: moe.linear(x.float(), w.float()), lambda: moe.linear(x, w.cpu()),
              lambda: moe.linear(x[0], w), lambda: moe.linear(x, w[:, :8]), lambda: moe.linear(wide[:, ::2], w),
              lambda: moe.linear(x, w, bias=v[:3]), lambda: moe.linear(x, w, bias=v.float()), lambda: moe.linear(x, w, act="swish"),
              lambda: moe.linear(x, w, residual=y[:2]), lambda: moe.linear(x, w, z=y.half()), lambda: moe.linear(x, w, out=y.t()),
              lambda: moe.linear(x, w, bias=torch.zeros((6, 2), dtype=torch.bfloat16, device="cuda")[:, 0]),
              lambda: moe.gated_linear(x, w[:5]), lambda: moe.gated_linear(x, w[:0]), lambda: moe.gated_linear(x, w, gu=y[:, :3]),
              lambda: moe.gated_linear(x, w, out=y), lambda: moe.linear_backward(y, x[:2], w),
              lambda: moe.linear_backward(y, x, w, dx=y), lambda: moe.linear_backward(y, x, w, dbias=v[:2]),
              lambda: moe.gated_linear_backward(y[:, :3], x, w, y[:2]), lambda: moe.layer_norm(x, v),
              lambda: moe.layer_norm(x, torch.zeros(16, dtype=torch.float16, device="cuda")),
              lambda: moe.layer_norm(x, torch.zeros(16, dtype=torch.float64, device="cuda")),
              lambda: moe.layer_norm(x, torch.zeros(16, device="cuda"), torch.zeros(16, dtype=torch.bfloat16, device="cuda")),
              lambda: moe.layer_norm(x.double()), lambda: moe.layer_norm(x, mean=s[:2]), lambda: moe.layer_norm(x, rstd=s.half()),
              lambda: moe.layer_norm_backward(x[:2], x, None, s, s), lambda: moe.linear(x, w, ws=torch.zeros(64))):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.moe_linear_backward(y, x, w, "silu", None, x.clone(), None, None, torch.zeros(1 << 20, device="cuda")),
              lambda: moe.moe_linear_backward(y, x, w, "none", None, x.clone(), None, None, None),
              lambda: moe.moe_linear_backward(y, None, w, "none", None, None, w.clone(), None, torch.zeros(1 << 20, device="cuda")),
              lambda: moe.layer_norm(x, eps=-1.0), lambda: moe.layer_norm(x, eps=math.nan),
              lambda: moe.linear(torch.empty_strided((2, 16), (1 << 22, 1), dtype=torch.bfloat16, device="cuda"), w),
              lambda: moe.linear(torch.zeros(32, dtype=torch.bfloat16, device="cuda").as_strided((3, 16), (8, 1)), w)):
        with pytest.raises(moe.MoeError):
            f()


def test_tensors_of_one_device():
    require_gpu()
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    x, w = torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda:1"), torch.ones((6, 16), dtype=torch.bfloat16, device="cuda:1")
    assert moe.linear(x, w).device == x.device           # the current device is the other one
    with pytest.raises(ValueError):
        moe.linear(x, w.to("cuda:0"))
