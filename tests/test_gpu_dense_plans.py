"""GPU: the linear and gated linear layers at the sizes where large tiles take K in parts, and where a backward pass's two
products share a launch.  Whole-numbered inputs: the exact result rounded once."""
import pytest
import torch

import combine_expert_histogram_amd as moe
from dense_helpers import HALF, Output, act64, generator, ids, inside, integers, same
from gpu_helpers import require_gpu, say

# (m, n, k), and which products are cut into parts there: x w^T, dx or dw; ragged ones, and two of whole tiles
PARTS = [((520, 4104, 4104), "y dx"),            # 128 x 128 tiles
         ((264, 4104, 4104), "y dx"),
         ((384, 2048, 4096), "y"),
         ((768, 4096, 8192), "y"),               # 256 x 256
         ((4104, 1032, 4104), "y dw"),           # 256 x 256, both
         ((4104, 4104, 1032), "dx"),             # 256 x 256
         ((8200, 264, 4104), "y dw")]            # 128 x 128, both
# a joint launch of 256 x 256 tiles with ragged edges: dw's tiles take 1, 2 and 4 times as long as dx's, and its last round
# is a whole one on most XCDs (the last)
JOINT = [(2056, 2056, 4104), (4104, 2056, 5640), (4104, 1032, 7176), (8200, 4104, 3592)]
PLACES = [(0, 0), (8, 16), (0, 3)]


def placed(t, place):
    return t if place == (0, 0) else inside(t, place[1], place[0])


@pytest.mark.parametrize("size,parts", PARTS, ids=ids)
def test_these_sizes_take_parts(size, parts):
    m, n, k = size
    assert (moe.moe_linear_workspace(m, n, k) >= 2 * m * n * 4) == ("y" in parts.split())
    assert (moe.moe_gated_linear_workspace(m, n // 2, k) >= 2 * m * n * 4) == ("y" in parts.split())
    rows = moe.moe_linear_backward_workspace(m, n, k, "none")
    for name, most in (("dx", m * k), ("dw", n * k)):
        assert name not in parts.split() or rows >= 2 * most * 4
    assert "d" in parts or rows < 2 * 4 * min(m * k, n * k)


def check_forward(size, place, dtype):
    m, n, k = size
    g = generator(m + 10 * n + 100 * k)
    x, w = integers(g, m, k, dtype), integers(g, n, k, dtype)
    bias, res = integers(g, 1, n, dtype, 9)[0], integers(g, m, n, dtype, 9)
    xp, wp = placed(x, place), placed(w, place)
    y, z = Output(m, n, dtype, place[1], place[0]), Output(m, n, dtype)
    moe.linear(xp, wp, bias=bias, act="relu", residual=placed(res, place), z=z.view, out=y.view)
    z64 = x.double() @ w.double().T + bias.double()
    same(z.view, z64, "z")
    same(y.view, act64(z64, "relu")[0] + res.double(), "y")
    y.check_surroundings()
    z.check_surroundings()
    sparse = x * (torch.rand((m, k), generator=g, device="cuda") < 0.05).to(dtype)
    gu64 = sparse.double() @ w.double().T
    h64 = act64(gu64[:, :n // 2], "relu")[0] * gu64[:, n // 2:]
    assert float(h64.abs().max()) < 2 ** 16
    h, gu = Output(m, n // 2, dtype, place[1], place[0]), Output(m, n, dtype)
    moe.gated_linear(placed(sparse, place), wp, act="relu", out=h.view, gu=gu.view)
    same(gu.view, gu64, "gu")
    same(h.view, h64, "h")
    h.check_surroundings()
    gu.check_surroundings()


def check_backward(size, place, dtype):
    m, n, k = size
    g = generator(m + 10 * n + 100 * k + 1)
    x, w, dy, z = (integers(g, *s, dtype, most) for *s, most in ((m, k, 1), (n, k, 1), (m, n, 1), (m, n, 2)))
    xp, wp, dyp, zp = (placed(t, place) for t in (x, w, dy, z))
    dx, dw = Output(m, k, dtype, place[1], place[0]), Output(n, k, dtype, place[1], place[0])
    ws = torch.full((max(moe.moe_linear_backward_workspace(m, n, k, "relu"),
                         moe.moe_gated_linear_backward_workspace(m, n // 2, k)),), 0xFF, dtype=torch.uint8, device="cuda")
    for act in ("none", "relu"):
        dz = dy.double() * act64(z.double(), act)[1]
        dx.view.fill_(5)
        dw.view.fill_(5)
        _, _, db = moe.linear_backward(dyp, xp, wp, act=act, z=zp, dx=dx.view, dw=dw.view, ws=ws)
        same(dx.view, dz @ w.double(), act + " dx")
        same(dw.view, dz.T @ x.double(), act + " dw")
        same(db, dz.sum(0), act + " dbias")
    inter = n // 2
    a, da = act64(z[:, :inter].double(), "relu")
    d = torch.cat((dy[:, :inter].double() * z[:, inter:].double() * da, dy[:, :inter].double() * a), 1)
    dx.view.fill_(5)
    dw.view.fill_(5)
    moe.gated_linear_backward(placed(dy[:, :inter], place), xp, wp, zp, act="relu", dx=dx.view, dw=dw.view, ws=ws)
    same(dx.view, d @ w.double(), "gated dx")
    same(dw.view, d.T @ x.double(), "gated dw")
    dx.check_surroundings()
    dw.check_surroundings()


@pytest.mark.gpu
@pytest.mark.parametrize("place", PLACES, ids=ids)
@pytest.mark.parametrize("size,parts", PARTS, ids=ids)
def test_parts_of_large_tiles(size, parts, place):
    require_gpu()
    dtype = HALF[(size[0] // 8 + place[1]) % 2]
    say(f"parts {size} {place} {dtype}")
    check_forward(size, place, dtype)
    check_backward(size, place, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF, ids=ids)
@pytest.mark.parametrize("size", JOINT, ids=ids)
def test_joint_launches(size, dtype):
    require_gpu()
    say(f"joint {size} {dtype}")
    check_backward(size, (0, 0), dtype)
    check_backward(size, (8, 16), dtype)
