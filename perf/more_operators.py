"""Cases that measure the dense half of an MoE block, forward and backward: layer norm, the gated linear layer
(both projections of a shared expert, the activation and the product), and the linear layer with bias, activation
and residual in its epilogue.

Each case runs either in a plain form (elementary torch operations in 32 bits, `own = False`) or through the
framework's entry points (`own = True`).  Rows are tokens.  Weights are [out, in]; a gated weight is [2*I, H], the gate's
rows first.  `pad` is the number of elements between a tensor's rows (a slice of a wider tensor).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
LARGEST = 8 * 16384 * 2048 * 7168          # flops of the largest listed case


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the norm of one decoded token: a launch's latency
        dict(name="norm_one", op="norm", M=1, H=7168, dtype="bf16", params="fp32", bias=True, pad=0),
        # the norm in front of router and experts, prefill of 8 sources x 2048 tokens
        dict(name="norm_prefill", op="norm", M=16384, H=7168, dtype="bf16", params="bf16", bias=True, pad=0),
        # a small odd model in full precision: rows that start anywhere, a ragged number of them
        dict(name="norm_bwd_odd", op="norm_bwd", M=777, H=1111, dtype="fp32", params="fp32", bias=True, pad=0),
        # training step of the same norm
        dict(name="norm_bwd_train", op="norm_bwd", M=16384, H=7168, dtype="bf16", params="fp32", bias=True, pad=0),
        # one decoded token through a shared expert's gate and up projections
        dict(name="gated_one", op="gated", M=1, I=2048, H=7168, dtype="bf16", act="silu", save=False, pad=0),
        # an odd decode batch of a smaller model, fp16
        dict(name="gated_decode", op="gated", M=17, I=1408, H=4096, dtype="fp16", act="gelu_tanh", save=False, pad=0),
        # prefill: 8 sources x 2048 tokens
        dict(name="gated_prefill", op="gated", M=16384, I=2048, H=7168, dtype="bf16", act="silu", save=False, pad=0),
        # training step of the same layer: gradients of the tokens and of both projections
        dict(name="gated_bwd_train", op="gated_bwd", M=16384, I=2048, H=7168, dtype="bf16", act="silu", pad=0),
        # one decoded token through the shared expert's down projection, added to the routed experts' output
        dict(name="linear_one", op="linear", M=1, N=7168, K=2048, dtype="bf16", act="none", bias=False, residual=True,
             save=False, pad=0),
        # odd sizes throughout, every part of the epilogue, the pre-activation kept for training
        dict(name="linear_odd", op="linear", M=1001, N=777, K=1111, dtype="fp16", act="gelu", bias=True, residual=True,
             save=True, pad=0),
        # the down projection of a prefill
        dict(name="linear_prefill", op="linear", M=16384, N=7168, K=2048, dtype="bf16", act="none", bias=False,
             residual=True, save=False, pad=0),
        # training step of a plain (ungated) layer with a bias
        dict(name="linear_bwd_train", op="linear_bwd", M=8192, N=4096, K=7168, dtype="bf16", act="gelu_tanh", bias=True,
             pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _size(rng, lo, hi):
    """Half of the sizes as they come, half rounded to the multiples that models have."""
    v = _log(rng, lo, hi)
    unit = rng.choice((1, 1, 8, 64, 128))
    return max(lo, v // unit * unit)


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "gated", "gated", "gated_bwd", "linear", "linear", "linear_bwd"))
    pad = rng.choice((0, 0, 0, 8, 5))
    if op in ("norm", "norm_bwd"):
        H = _size(rng, 64, 16384)
        return dict(op=op, M=min(_size(rng, 1, 16384), 16384 * 7168 // H), H=H, dtype=rng.choice(tuple(DTYPES)),
                    params=rng.choice(("fp32", "same")), bias=rng.random() < 0.7, pad=pad)
    dtype, M = rng.choice(("bf16", "bf16", "fp16")), _size(rng, 1, 16384)
    act = rng.choice(("silu", "gelu", "gelu_tanh", "relu"))
    if op in ("gated", "gated_bwd"):
        H = _size(rng, 128, 7168)
        I = min(_size(rng, 64, 16384), LARGEST // (8 * M * H))
        case = dict(op=op, M=M, I=I, H=H, dtype=dtype, act=act, pad=pad)
        return dict(case, save=rng.random() < 0.3) if op == "gated" else case
    K = _size(rng, 64, 8192)
    N = min(_size(rng, 64, 32768), LARGEST // (4 * M * K))
    case = dict(op=op, M=M, N=N, K=K, dtype=dtype, act=rng.choice((act, "none")), bias=rng.random() < 0.5, pad=pad)
    return dict(case, residual=rng.random() < 0.5, save=rng.random() < 0.3) if op == "linear" else case


# ---------------------------------------------------------------- inputs
def _normal(gen, rows, cols, dtype, scale=1.0, pad=0):
    """N(0, scale) rows, as a slice of a wider tensor if pad > 0"""
    t = torch.randn((rows, cols), generator=gen, device="cuda").mul_(scale).to(dtype)
    if not pad:
        return t
    wide = torch.zeros((rows, cols + pad), dtype=dtype, device="cuda")
    wide[:, :cols] = t
    return wide[:, :cols]


def _empty(rows, cols, dtype, pad=0):
    return torch.zeros((rows, cols + pad), dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, M, pad, dtype = case["op"], case["M"], case["pad"], DTYPES[case["dtype"]]
    state = dict(case)
    if op in ("norm", "norm_bwd"):
        H = case["H"]
        params = dtype if case["params"] == "same" else DTYPES[case["params"]]
        # a residual stream: rows of different size, a common offset, a few large channels
        size = torch.exp(torch.randn((M, 1), generator=gen, device="cuda") * 0.5)
        channel = torch.ones(H, device="cuda")
        channel[torch.randint(0, H, (max(1, H // 256),), generator=gen, device="cuda")] = 16.0
        x = (torch.randn((M, H), generator=gen, device="cuda") * channel + 0.25) * size
        state["x"] = _empty(M, H, dtype, pad).copy_(x)
        state["w"] = (1.0 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(params)
        state["b"] = (0.1 * torch.randn(H, generator=gen, device="cuda")).to(params) if case["bias"] else None
        state["mean"] = torch.zeros(M, dtype=torch.float32, device="cuda")
        state["rstd"] = torch.zeros(M, dtype=torch.float32, device="cuda")
        if op == "norm":
            state["y"] = _empty(M, H, dtype, pad)
            return state
        v = state["x"].double()
        mean = v.sum(1) / H
        state["mean"].copy_(mean)
        state["rstd"].copy_(1.0 / torch.sqrt(((v - mean[:, None]) ** 2).sum(1) / H + EPS))
        state["dy"] = _normal(gen, M, H, dtype, 1.0, pad)
        state["dx"] = _empty(M, H, dtype, pad)
        state["dw"] = torch.zeros(H, dtype=params, device="cuda")
        state["db"] = torch.zeros(H, dtype=params, device="cuda") if case["bias"] else None
        if own:
            import combine_expert_histogram_amd as moe
            state["ws"] = moe.alloc_layer_norm_backward_workspace(M, H)
        return state
    if op in ("gated", "gated_bwd"):
        I, H = case["I"], case["H"]
        state["x"] = _normal(gen, M, H, dtype, 1.0, pad)
        state["w"] = _normal(gen, 2 * I, H, dtype, 0.02)
        if op == "gated":
            state["h"] = _empty(M, I, dtype, pad)
            state["gu"] = _empty(M, 2 * I, dtype) if case["save"] else None
        else:
            state["gu"] = _normal(gen, M, 2 * I, dtype, 0.02 * math.sqrt(H))     # as x and w give
            state["dh"] = _normal(gen, M, I, dtype, 1.0, pad)
            state["dx"], state["dw"] = _empty(M, H, dtype, pad), _empty(2 * I, H, dtype)
        if own:
            import combine_expert_histogram_amd as moe
            state["ws"] = (moe.alloc_gated_linear_workspace(M, I, H) if op == "gated" else
                           moe.alloc_gated_linear_backward_workspace(M, I, H))
        return state
    N, K = case["N"], case["K"]
    state["x"] = _normal(gen, M, K, dtype, 1.0, pad)
    state["w"] = _normal(gen, N, K, dtype, 0.02)
    if op == "linear":
        state["b"] = _normal(gen, 1, N, dtype, 0.1)[0] if case["bias"] else None
        state["res"] = _normal(gen, M, N, dtype, 1.0, pad) if case["residual"] else None
        state["y"] = _empty(M, N, dtype, pad)
        state["z"] = _empty(M, N, dtype) if case["save"] else None
    else:
        state["dy"] = _normal(gen, M, N, dtype, 1.0, pad)
        state["z"] = None if case["act"] == "none" else _normal(gen, M, N, dtype, 0.02 * math.sqrt(K))
        state["dx"], state["dw"] = _empty(M, K, dtype, pad), _empty(N, K, dtype)
        state["db"] = torch.zeros(N, dtype=dtype, device="cuda") if case["bias"] else None
    if own:
        import combine_expert_histogram_amd as moe
        state["ws"] = (moe.alloc_linear_workspace(M, N, K) if op == "linear" else
                       moe.alloc_linear_backward_workspace(M, N, K, case["act"]))
    return state


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import combine_expert_histogram_amd as moe
    op = s["op"]
    if op == "norm":
        moe.layer_norm(s["x"], s["w"], s["b"], eps=EPS, out=s["y"], mean=s["mean"], rstd=s["rstd"])
        return s["y"], s["mean"], s["rstd"]
    if op == "norm_bwd":
        return moe.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], dx=s["dx"], dweight=s["dw"],
                                       dbias=s["db"], bias=s["bias"], ws=s["ws"])
    if op == "gated":
        h = moe.gated_linear(s["x"], s["w"], act=s["act"], out=s["h"], gu=s["gu"], ws=s["ws"])
        return h, s["gu"]
    if op == "gated_bwd":
        return moe.gated_linear_backward(s["dh"], s["x"], s["w"], s["gu"], act=s["act"], dx=s["dx"], dw=s["dw"],
                                         ws=s["ws"])
    if op == "linear":
        y = moe.linear(s["x"], s["w"], bias=s["b"], act=s["act"], residual=s["res"], out=s["y"], z=s["z"], ws=s["ws"])
        return y, s["z"]
    return moe.linear_backward(s["dy"], s["x"], s["w"], act=s["act"], z=s["z"], bias=s["bias"], dx=s["dx"], dw=s["dw"],
                               dbias=s["db"], ws=s["ws"])


# ---------------------------------------------------------------- plain form
GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z / (1.0 + torch.exp(-2.0 * GELU_C * (z + GELU_A * z * z * z)))


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) +
                z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    s = 1.0 / (1.0 + torch.exp(-2.0 * GELU_C * (z + GELU_A * z * z * z)))
    return s + z * s * (1.0 - s) * (2.0 * GELU_C) * (1.0 + 3.0 * GELU_A * z * z)


def run(state):
    s = state
    if own:
        return _own(s)
    op, x, w = s["op"], s["x"].float(), s["w"].float()
    dtype = s["x"].dtype
    if op == "norm":
        mean = x.sum(1) / s["H"]
        c = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((c * c).sum(1) / s["H"] + EPS)
        y = c * rstd[:, None] * w
        if s["b"] is not None:
            y = y + s["b"].float()
        return y.to(dtype), mean, rstd
    if op == "norm_bwd":
        dy = s["dy"].float()
        xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * w
        dx = s["rstd"][:, None] * (g - g.sum(1, keepdim=True) / s["H"] - xh * ((g * xh).sum(1, keepdim=True) / s["H"]))
        db = dy.sum(0).to(s["w"].dtype) if s["bias"] else None
        return dx.to(dtype), (dy * xh).sum(0).to(s["w"].dtype), db
    if op == "gated":
        gu = x @ w.t()
        g, u = gu[:, :s["I"]], gu[:, s["I"]:]
        return (_act(g, s["act"]) * u).to(dtype), gu.to(dtype) if s["save"] else None
    if op == "gated_bwd":
        gu, dh = s["gu"].float(), s["dh"].float()
        g, u = gu[:, :s["I"]], gu[:, s["I"]:]
        d = torch.cat((dh * u * _act_grad(g, s["act"]), dh * _act(g, s["act"])), 1)
        return (d @ w).to(dtype), (d.t() @ x).to(dtype)
    if op == "linear":
        z = x @ w.t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, s["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return y.to(dtype), z.to(dtype) if s["save"] else None
    d = s["dy"].float()
    if s["act"] != "none":
        d = d * _act_grad(s["z"].float(), s["act"])
    return (d @ w).to(dtype), (d.t() @ x).to(dtype), d.sum(0).to(dtype) if s["bias"] else None


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, M = case["op"], case["M"]
    e = 4 if case["dtype"] == "fp32" else 2
    if op in ("norm", "norm_bwd"):
        H = case["H"]
        p = e if case["params"] == "same" else (4 if case["params"] == "fp32" else 2)
        vectors = (2 if case["bias"] else 1) * H * p
        if op == "norm":
            return {"bytes": 2 * M * H * e + vectors + 8 * M, "flops": 8 * M * H}
        return {"bytes": 3 * M * H * e + vectors + H * p + 8 * M, "flops": 14 * M * H}
    if op in ("gated", "gated_bwd"):
        I, H = case["I"], case["H"]
        if op == "gated":
            return {"bytes": e * (M * H + 2 * I * H + M * I + (2 * M * I if case["save"] else 0)),
                    "flops": 4 * M * I * H}
        return {"bytes": e * (2 * M * H + 4 * I * H + 3 * M * I), "flops": 8 * M * I * H}
    N, K = case["N"], case["K"]
    bias = N if case["bias"] else 0
    if op == "linear":
        return {"bytes": e * (M * K + N * K + bias + M * N * (1 + case["residual"] + case["save"])),
                "flops": 2 * M * N * K}
    return {"bytes": e * (2 * M * K + 2 * N * K + bias + M * N * (1 if case["act"] == "none" else 2)),
            "flops": 4 * M * N * K}


# ---------------------------------------------------------------- 64 bits
def _phi(z):
    return torch.special.erfc(z * -(0.5 ** 0.5)) / 2


def _exact_act(z, act):
    """The activation and its derivative, in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), torch.heaviside(z, torch.zeros_like(z))
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if act == "gelu":
        return z * _phi(z), _phi(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3)))
    d = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z.square())
    return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t.square()) * d / 2


def exact(case, seed):
    s = prepare(case, seed)
    f64 = {k: v.to(torch.float64) for k, v in s.items() if isinstance(v, torch.Tensor) and k != "ws"}
    x, w, op = f64["x"], f64["w"], case["op"]
    if op == "norm":
        mean = x.mean(1)
        rstd = torch.rsqrt((x - mean.unsqueeze(1)).square().mean(1) + EPS)
        y = torch.addcmul(f64["b"] if case["bias"] else torch.zeros_like(w), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), w)
        return y, mean, rstd
    if op == "norm_bwd":
        # the gradient of sum(dy * y) at the given statistics: dx = r (I - 11'/H - xh xh'/H) (w dy)
        r, dy = f64["rstd"].unsqueeze(1), f64["dy"]
        xh = r * (x - f64["mean"].unsqueeze(1))
        g = dy * w
        dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return dx, (dy * xh).sum(0), dy.sum(0) if case["bias"] else None
    if op == "gated":
        g, u = torch.matmul(x, w.mT).chunk(2, dim=1)
        return _exact_act(g, case["act"])[0] * u, torch.cat((g, u), 1) if case["save"] else None
    if op == "gated_bwd":
        g, u = f64["gu"].chunk(2, dim=1)
        a, da = _exact_act(g, case["act"])
        d = torch.cat((f64["dh"] * u * da, f64["dh"] * a), 1)
        return torch.matmul(d, w), torch.matmul(d.mT, x)
    if op == "linear":
        z = torch.matmul(x, w.mT) + (f64["b"] if case["bias"] else 0)
        y = _exact_act(z, case["act"])[0] + (f64["res"] if case["residual"] else 0)
        return y, z if case["save"] else None
    d = f64["dy"]
    if case["act"] != "none":
        d = d * _exact_act(f64["z"], case["act"])[1]
    return torch.matmul(d, w), torch.matmul(d.mT, x), d.sum(0) if case["bias"] else None
