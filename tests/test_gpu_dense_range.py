"""GPU: gradients of any size through the linear and gated linear layers' backward passes, fp16's small and large ones among
them, against float64."""
import math

import pytest
import torch

import combine_expert_histogram_amd as moe
from dense_helpers import (F32_HALF, HALF, act64, act_error, close, generator, grad_error, ids, normal, sum_error)
from gpu_helpers import require_gpu, say
from test_kernel_registers import found  # noqa: F401  (the fixture)

# (m, n, k): two terms and one, 64, 128 and 256 tiles, rows that start anywhere
SIZES = [(1, 8, 24), (40, 24, 72), (64, 136, 264), (65, 136, 264), (97, 131, 301), (300, 264, 136), (2048, 1024, 2048)]


def operand_error(d, m, dtype, most):
    """What 16 bits leave of computed gradients d: half a step of each, or of what the first of two terms left (a step of the
    first, so that the second's half steps are 2^-16 of d in bf16, 2^-22 in fp16).  fp16: scaled so that `most`, the largest
    (of dy in the linear layer) is 2^14 and more, the smallest half step is 2^-25, which is 2^-39 of it.  bf16: half of its
    smallest step is 2^-134."""
    if dtype == torch.bfloat16:
        return d * (2.0 ** -16 if m <= 64 else 2.0 ** -8) + 2.0 ** -134
    return d * (2.0 ** -22 if m <= 64 else 2.0 ** -11) + most * 2.0 ** -39


def largest(t):
    return float(t.abs().max())


def check_products(d, ed, x, w, m, dx, dw, most, what):
    er = ed + operand_error(d.abs() + ed, m, dx.dtype, most)
    size, n = d.abs() + er, d.shape[1]
    x64, w64 = x.double(), w.double()
    a = close(dx, d @ w64, er @ w64.abs() + sum_error(2 * n, size @ w64.abs()), what + " dx")
    b = close(dw, d.T @ x64, er.T @ x64.abs() + sum_error(2 * m, size.T @ x64.abs()), what + " dw")
    return a, b


def linear_case(g, size, dtype, scale, act, dense):
    m, n, k = size
    dy = normal(g, m, n, dtype, scale)
    if not dense:              # few terms to a sum, so that a bound on it is near what one term may be off
        dy *= (torch.rand((m, n), generator=g, device="cuda") < 3 / max(m, n)).to(dtype)
        dy[m // 2, n // 2] = scale
    # outputs are normal numbers of fp16
    one = max(1.0, 1e-2 / scale)
    x, w, z = normal(g, m, k, dtype, min(one, 100.0)), normal(g, n, k, dtype, min(one, 100.0)), normal(g, m, n, dtype, 2)
    dz = dy.double() * act64(z.double(), act)[1]
    return dy, x, w, z, dz, dy.double().abs() * grad_error(z.double(), act) + 2 * F32_HALF * dz.abs()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("scale", [1.0, 1e-3, 1e-5, 2e-7])
@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_small_linear_gradients(size, scale, dtype):
    require_gpu()
    m = size[0]
    for act, dense in (("silu", False), ("gelu", True)):
        g = generator(sum(size))
        dy, x, w, z, dz, ed = linear_case(g, size, dtype, scale, act, dense)
        dx, dw, db = moe.linear_backward(dy, x, w, act=act, z=z)
        what = f"linear {size} {scale} {act} {dtype}"
        say(what, check_products(dz, ed, x, w, m, dx, dw, largest(dy), what))
        close(db, dz.sum(0), ed.sum(0) + sum_error(m, dz.abs().sum(0)), what + " dbias")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("scale", [1.0, 1e-3, 1e-5])
@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_small_gated_gradients(size, scale, dtype):
    require_gpu()
    m, inter, k = size[0], size[1] // 2, size[2]
    for act, dense in (("silu", False), ("gelu_tanh", True)):
        g = generator(sum(size) + 1)
        dh = normal(g, m, inter, dtype, scale)
        if not dense:
            dh *= (torch.rand((m, inter), generator=g, device="cuda") < 3 / max(m, inter)).to(dtype)
            dh[m // 2, inter // 2] = scale
        one = min(max(1.0, 1e-2 / scale), 100.0)
        x, w, gu = normal(g, m, k, dtype, one), normal(g, 2 * inter, k, dtype, one), normal(g, m, 2 * inter, dtype)
        gate, up, dh64 = gu[:, :inter].double(), gu[:, inter:2 * inter].double(), dh.double()
        a, da = act64(gate, act)
        d = torch.cat((dh64 * up * da, dh64 * a), 1)
        ed = torch.cat(((dh64 * up).abs() * grad_error(gate, act), dh64.abs() * act_error(gate, 0.0, act)), 1)
        dx, dw = moe.gated_linear_backward(dh, x, w, gu, act=act)
        what = f"gated {size} {scale} {act} {dtype}"
        say(what, check_products(d, ed + 3 * F32_HALF * d.abs(), x, w, m, dx, dw, largest(d), what))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 40, 65, 300])
def test_gradients_past_the_largest_number(m):
    """dh u = 90000 has no place in fp16; the products with small weights and tokens have."""
    require_gpu()
    g = generator(m)
    inter, k = 16, 40
    sign = lambda *s: torch.randint(0, 2, s, generator=g, device="cuda").half() * 2 - 1  # noqa: E731
    dh, gu = 300 * sign(m, inter), 300 * sign(m, 2 * inter)
    gu[:, :inter] = gu[:, :inter].abs()                      # silu(300) is 300 and its slope 1
    x, w = sign(m, k) * 2.0 ** -10, sign(2 * inter, k) * 2.0 ** -10
    d = torch.cat((dh.double() * gu[:, inter:].double(), dh.double() * 300), 1)
    dx, dw = moe.gated_linear_backward(dh, x, w, gu)
    check_products(d, torch.zeros_like(d), x, w, m, dx, dw, largest(d), f"large {m}")
    dy, z = 60000 * sign(m, 24), torch.full((m, 24), 1.5, dtype=torch.float16, device="cuda")
    w = sign(24, k) * 2.0 ** -10
    slope = act64(z.double(), "gelu")[1]
    assert float(slope.min()) > 65504 / 60000
    dx, dw, _ = moe.linear_backward(dy, x, w, act="gelu", z=z)
    d = dy.double() * slope
    ed = dy.double().abs() * grad_error(z.double(), "gelu") + 2 * F32_HALF * d.abs()
    check_products(d, ed, x, w, m, dx, dw, largest(dy), f"slope {m}")


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 64, 65, 300])
def test_gradients_of_unlike_size(m):
    """One large gradient beside small ones, none at all, and one that is infinite: the others keep their bits."""
    require_gpu()
    size = (m, 24, 72)
    for dtype in HALF:
        g = generator(m)
        dy, x, w, z, dz, ed = linear_case(g, size, dtype, 1e-3, "silu", True)
        dy[m // 2, 5] = 50000.0
        z[m // 2, 5] = 4.0
        dz = dy.double() * act64(z.double(), "silu")[1]
        ed = dy.double().abs() * grad_error(z.double(), "silu") + 2 * F32_HALF * dz.abs()
        x, w = x * 0.01, w * 0.01
        dx, dw, _ = moe.linear_backward(dy, x, w, act="silu", z=z)
        check_products(dz, ed, x, w, m, dx, dw, largest(dy), f"unlike {m} {dtype}")
        dx, dw, db = moe.linear_backward(torch.zeros_like(dy), x, w, act="silu", z=z)
        assert not dx.any() and not dw.any() and not db.any()
        dy[m // 2, 5] = math.inf
        got = moe.linear_backward(dy, x, w, act="silu", z=z)
        dy[m // 2, 5] = 0
        ref = moe.linear_backward(dy, x, w, act="silu", z=z)
        rows, cols = [i for i in range(m) if i != m // 2], [i for i in range(24) if i != 5]
        assert torch.equal(got[0][rows], ref[0][rows]) and torch.equal(got[1][cols], ref[1][cols])
        assert not torch.isfinite(got[0][m // 2]).any() and not torch.isfinite(got[1][5]).any()


def same_infinities(got, want, what):
    """Infinities and NaNs where the formula has them."""
    for f in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(f(got), f(want)), what


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("m", [1, 5, 64, 65])
def test_infinite_weights_and_tokens(m, act, dtype):
    """They meet gradients of 16 bits (whole numbers) and of more."""
    require_gpu()
    g = generator(m)
    n, k = 24, 40
    dy = torch.randint(1, 9, (m, n), generator=g, device="cuda").to(dtype)
    dy = dy * (torch.randint(0, 2, (m, n), generator=g, device="cuda") * 2 - 1).to(dtype)
    z = torch.randint(1, 4, (m, n), generator=g, device="cuda").to(dtype)
    x, w = normal(g, m, k, dtype), normal(g, n, k, dtype)
    x[m // 2, 5], w[3, 7], w[4, 9] = math.inf, math.inf, -math.inf
    for t, u in ((dy, z), (torch.zeros_like(dy), z)):
        dz = t.double() * act64(u.double(), act)[1]
        dx, dw, _ = moe.linear_backward(t, x, w, act=act, z=u)
        same_infinities(dx, dz @ w.double(), f"dx {m} {act}")
        same_infinities(dw, dz.T @ x.double(), f"dw {m} {act}")
    gu = torch.cat((z[:, :n // 2], dy[:, :n // 2]), 1)
    dh = dy[:, n // 2:]
    a, da = act64(gu[:, :n // 2].double(), act)
    d = torch.cat((dh.double() * gu[:, n // 2:].double() * da, dh.double() * a), 1)
    dx, dw = moe.gated_linear_backward(dh, x, w, gu, act=act)
    same_infinities(dx, d @ w.double(), f"gated dx {m} {act}")
    same_infinities(dw, d.T @ x.double(), f"gated dw {m} {act}")


@pytest.mark.gpu
@pytest.mark.parametrize("m", [8, 200])
def test_each_replay_takes_its_own_scale(m):
    """Captured once; replayed with gradients of other sizes: the eager call's results, and the formula's."""
    require_gpu()
    size = (m, 40, 72)
    g = generator(m)
    dy, x, w, z, _, _ = linear_case(g, size, torch.float16, 1.0, "silu", True)
    ws = moe.alloc_linear_backward_workspace(*size, "silu").fill_(0xFF)
    dx, dw, db = moe.linear_backward(dy, x, w, act="silu", z=z, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            moe.linear_backward(dy, x, w, act="silu", z=z, dx=dx, dw=dw, dbias=db, ws=ws)
    for scale in (1e-5, 1000.0, 0.0, 1e-3):
        dy.copy_(normal(g, m, 40, torch.float16, scale))
        ws.fill_(0xFF)
        for t in (dx, dw, db):
            t.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = moe.linear_backward(dy, x, w, act="silu", z=z)
        assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), ref)), scale
        dz = dy.double() * act64(z.double(), "silu")[1]
        ed = dy.double().abs() * grad_error(z.double(), "silu") + 2 * F32_HALF * dz.abs()
        check_products(dz, ed, x, w, m, dx, dw, largest(dy), f"replay {scale}")


@pytest.mark.parametrize("kernel", ["gate_peak_kernel", "dz_peak_kernel"])
def test_no_peak_kernel_spills(found, kernel):  # noqa: F811
    these = [k for k in found if kernel in k[".name"]]
    assert these and not any(k[".vgpr_spill_count"] for k in these)
