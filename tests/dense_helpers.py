"""Inputs, references and error bounds shared by the dense layers' tests.  References are float64 torch on the inputs' own
device, written from the formulas."""
from __future__ import annotations

import math

import torch

import combine_expert_histogram_amd as moe

F32_HALF = 2.0 ** -24        # one rounding to fp32, relative
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
HALF = (torch.bfloat16, torch.float16)


def generator(seed: int, device="cuda") -> torch.Generator:
    return torch.Generator(device=device).manual_seed(seed)


def integers(g, rows, cols, dtype, most=1):
    """Whole numbers in -most .. most: every product and sum of a test below 2^24 is exact in fp32."""
    return torch.randint(-most, most + 1, (rows, cols), generator=g, device=g.device).to(dtype)


def normal(g, rows, cols, dtype, scale=1.0):
    return (torch.randn((rows, cols), generator=g, device=g.device) * scale).to(dtype)


def inside(t, pad, lead=0, fill=math.nan):
    """t as a slice of a wider tensor: `lead` elements before each row, `pad` after it, all of them `fill`."""
    rows, cols = t.shape
    wide = torch.full((rows, lead + cols + pad), fill, dtype=t.dtype, device=t.device)
    wide[:, lead:lead + cols] = t
    return wide[:, lead:lead + cols]


class Output:
    """A [rows, cols] output inside a poisoned buffer, with rows of poison before and behind."""

    def __init__(self, rows, cols, dtype, pad=0, lead=0, device="cuda"):
        self.wide = torch.full((rows + 2, lead + cols + pad), -77.0, dtype=dtype, device=device)
        self.view = self.wide[1:rows + 1, lead:lead + cols]
        self.keep = torch.ones_like(self.wide, dtype=torch.bool)
        self.keep[1:rows + 1, lead:lead + cols] = False

    def check_surroundings(self):
        assert bool((self.wide[self.keep] == -77.0).all()), "written outside the output"


def act64(z, act):
    """(act(z), act'(z)) in float64"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c, a = math.sqrt(2 / math.pi), 0.044715
    s = torch.sigmoid(2 * c * (z + a * z ** 3))
    return z * s, s + z * s * (1 - s) * 2 * c * (1 + 3 * a * z * z)


# Bounds.  A sum of K products in fp32 is off by at most 2 (K + 4) half steps of sum |a b| (a matrix instruction may cut
# off where it aligns its products: at most twice a rounding).  Every activation has |act'| < 1.2 and |act''| < 1.2 (silu's
# and both gelus' largest second derivative is 2 phi(0) = 0.80).  Evaluated in fp32 an activation takes under 16 roundings
# and hardware approximations of two half steps each, and one exponential (erfc holds one) whose argument of size a is
# rounded up to four times, which moves it by 4 a half steps relatively; past a = 100 both sides are 0 or z.
# Its derivative's terms are each at most 1 + |z| in size.  2^-126: fp32's smallest normal, below which results may be 0.
def sum_error(k, magnitude):
    return 2 * F32_HALF * (k + 4) * magnitude


def argument(z, act):
    if act == "gelu":
        return 0.5 * z * z
    if act == "gelu_tanh":
        return 2 * math.sqrt(2 / math.pi) * (z.abs() + 0.044715 * z.abs() ** 3)
    return z.abs()


def act_error(z, ez, act):
    """Bound on |computed act(z') - act(z)|, |z' - z| <= ez."""
    a, _ = act64(z, act)
    own = 0.0 if act in ("none", "relu") else (32 + 4 * argument(z, act).clamp(max=100)) * F32_HALF
    return 1.2 * ez + own * (a.abs() + 1.2 * ez) + 2.0 ** -126


def grad_error(z, act):
    """Bound on |computed act'(z) - act'(z)| for an exact z."""
    if act in ("none", "relu"):
        return torch.zeros_like(z)
    return (32 + 4 * argument(z, act).clamp(max=100)) * F32_HALF * (1 + z.abs().clamp(max=15)) + 2.0 ** -126


def rounding(value, dtype):
    """Half a step of `dtype` around values of this magnitude."""
    f = torch.finfo(dtype)
    return value * (f.eps / 2) + f.tiny * f.eps / 2


def close(got, want, bound, what=""):
    """|got - want| <= bound and one rounding to got's type"""
    assert got.shape == want.shape, what
    err = (got.double() - want).abs()
    allowed = bound + rounding(want.abs() + bound, got.dtype)
    assert bool(torch.isfinite(got).all()), what + ": not finite"
    worst = float((err / allowed).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    return worst


def same(got, want, what=""):
    """got is want (float64, exact) rounded once."""
    want = want.to(got.dtype)
    assert got.shape == want.shape, what
    if not torch.equal(got, want):
        at = torch.nonzero(got != want)[0].tolist()
        bad = int((got != want).sum())
        raise AssertionError(f"{what}: {bad} of {got.numel()} differ, first at {at}: {got[tuple(at)]} for {want[tuple(at)]}")


def linear_sizes():
    """(m, n, k): few rows, one and more tiles, odd sizes, K cut in parts, large tiles"""
    return [(1, 1, 1), (1, 16, 8), (1, 7168, 2048), (2, 33, 65), (15, 24, 136), (16, 128, 128), (17, 100, 1000),
            (33, 17, 127), (48, 64, 320), (49, 8, 64), (64, 264, 520), (65, 8, 8), (65, 130, 72), (100, 1, 37),
            (127, 129, 63), (128, 128, 64), (129, 128, 65), (200, 392, 1160), (256, 256, 2048), (70, 96, 8200),
            (300, 1031, 257), (1000, 520, 136), (4096, 3400, 200), (130, 5, 200), (131, 200, 5), (67, 9, 11), (300, 259, 333)]


def ids(v):
    return "x".join(str(i) for i in v) if isinstance(v, tuple) else str(v).replace("torch.", "")


def held(value, m, dtype):
    """What the products' 16-bit operand leaves of a gradient of this size: a rounding, or with up to 64 tokens, where a
    second term holds that, its rounding"""
    once = rounding(value, dtype)
    return rounding(once, dtype) if m <= 64 else once


def F(value, error=0.0):
    """One rounding to fp32 of a value within `error` of this one"""
    return F32_HALF * (value.abs() + error)


def check_linear(x, w, bias, act, res, z, y):
    k = x.shape[1]
    x64, w64 = x.double(), w.double()
    b64 = torch.zeros(w.shape[0], dtype=torch.float64, device=x.device) if bias is None else bias.double()
    z64 = x64 @ w64.T + b64
    ez = sum_error(k + 2, x64.abs() @ w64.abs().T + b64.abs())
    if z is not None:
        close(z, z64, ez, "z")
    ea = act_error(z64, ez, act)
    want = act64(z64, act)[0]
    if res is not None:
        want = want + res.double()
        ea = ea + F(want, ea)
    return close(y, want, ea, "y")


def check_linear_backward(dy, x, w, act, z, dx, dw, db):
    m, n = dy.shape
    dy64 = dy.double()
    if act == "none":
        dz, ed = dy64, torch.zeros_like(dy64)
        er = ed
    else:
        z64 = z.double()
        dz = dy64 * act64(z64, act)[1]
        ed = dy64.abs() * grad_error(z64, act) + 2 * F(dz)
        er = ed + held(dz.abs() + ed, m, dy.dtype)
    size, worst = dz.abs() + er, []
    if dx is not None:
        w64 = w.double()
        worst.append(close(dx, dz @ w64, er @ w64.abs() + sum_error(2 * n, size @ w64.abs()), "dx"))
    if dw is not None:
        x64 = x.double()
        worst.append(close(dw, dz.T @ x64, er.T @ x64.abs() + sum_error(2 * m, size.T @ x64.abs()), "dw"))
    if db is not None:
        worst.append(close(db, dz.sum(0), ed.sum(0) + sum_error(m, size.sum(0)), "dbias"))
    return worst


def check_gated(x, w, act, gu, h):
    inter, k = h.shape[1], x.shape[1]
    x64, w64 = x.double(), w.double()
    z64, ez = x64 @ w64.T, sum_error(k, x64.abs() @ w64.abs().T)
    if gu is not None:
        close(gu, z64, ez, "gu")
    gate, up, eg, eu = z64[:, :inter], z64[:, inter:], ez[:, :inter], ez[:, inter:]
    a, ea = act64(gate, act)[0], act_error(gate, eg, act)
    e = ea * (up.abs() + eu) + a.abs() * eu
    return close(h, a * up, e + F(a * up, e), "h")


def check_gated_backward(dh, x, w, gu, act, dx, dw):
    m, inter = dh.shape
    gate, up, dh64 = gu[:, :inter].double(), gu[:, inter:].double(), dh.double()
    a, da = act64(gate, act)
    d = torch.cat((dh64 * up * da, dh64 * a), 1)
    ed = torch.cat(((dh64 * up).abs() * grad_error(gate, act), dh64.abs() * act_error(gate, 0.0, act)), 1) + 3 * F(d)
    ed = ed + held(d.abs() + ed, m, dh.dtype)
    size, worst = d.abs() + ed, []
    if dx is not None:
        w64 = w.double()
        worst.append(close(dx, d @ w64, ed @ w64.abs() + sum_error(4 * inter, size @ w64.abs()), "dx"))
    if dw is not None:
        x64 = x.double()
        worst.append(close(dw, d.T @ x64, ed.T @ x64.abs() + sum_error(2 * m, size.T @ x64.abs()), "dw"))
    return worst


def check_norm(x, w, b, eps, y, mean, rstd, what):
    """mean: a sum of H terms.  c = x - mean carries the mean's error and a rounding; the variance 2 |c| ec from each
    square and the sum's roundings; rstd half the variance's relative error, a division, a root and a sum; y three more."""
    H = x.shape[1]
    x64 = x.double()
    w64 = torch.ones(H, dtype=torch.float64, device=x.device) if w is None else w.double()
    b64 = torch.zeros(H, dtype=torch.float64, device=x.device) if b is None else b.double()
    m = x64.sum(1, keepdim=True) / H
    em = F32_HALF * (H + 4) * x64.abs().sum(1, keepdim=True) / H
    c = x64 - m
    ec = em + F32_HALF * (c.abs() + em)
    v = (c * c).sum(1, keepdim=True) / H
    ev = ((2 * c.abs() * ec + ec * ec).sum(1, keepdim=True) + F32_HALF * (H + 4) * ((c.abs() + ec) ** 2).sum(1, keepdim=True)) / H
    r = 1 / torch.sqrt(v + eps)
    rel = ev / (v + eps)
    assert float(rel.max()) < 0.5
    er = r * (rel + 4 * F32_HALF)                                   # 1/sqrt(1 - t) - 1 <= t for t < 0.5
    want = c * r * w64 + b64
    ey = (ec * (r + er) + c.abs() * er) * w64.abs() + 3 * F32_HALF * ((c * r * w64).abs() + b64.abs())
    worst = close(y, want, ey, what + " y")
    if mean is not None:
        close(mean, m[:, 0], em[:, 0] + F32_HALF * m[:, 0].abs(), what + " mean")
        close(rstd, r[:, 0], er[:, 0], what + " rstd")
    return worst


def check_norm_backward(dy, x, w, mean, rstd, dx, dweight, dbias, what):
    """n = (x - mean) rstd takes two roundings and g = dy w one; the rows' and columns' sums a rounding a term."""
    rows, H = x.shape
    w64 = torch.ones(H, dtype=torch.float64, device=x.device) if w is None else w.double()
    m, r, dy64 = mean.double()[:, None], rstd.double()[:, None], dy.double()
    n, g = (x.double() - m) * r, dy64 * w64
    sg, sgn = g.sum(1, keepdim=True) / H, (g * n).sum(1, keepdim=True) / H
    e1 = F32_HALF * (H + 5) * g.abs().sum(1, keepdim=True) / H
    e2 = F32_HALF * (H + 9) * (g * n).abs().sum(1, keepdim=True) / H
    if dx is not None:
        size = g.abs() + sg.abs() + (n * sgn).abs()
        e = r * (e1 + n.abs() * e2 * (1 + 3 * F32_HALF) + 9 * F32_HALF * size)
        close(dx, r * (g - sg - n * sgn), e, what + " dx")
    if dweight is not None:
        close(dweight, (dy64 * n).sum(0), F32_HALF * (rows + 10) * (dy64 * n).abs().sum(0), what + " dweight")
    if dbias is not None:
        close(dbias, dy64.sum(0), F32_HALF * (rows + 4) * dy64.abs().sum(0), what + " dbias")
