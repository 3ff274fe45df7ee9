"""Cases that measure the few-token serving operators: the router's top-k, the matrix-vector
products over block-scaled weights (4-bit ones above all), and the whole MoE layer for a few tokens.

Each case runs either in a plain form (elementary torch operations in 32 bits, `own = False`) or through
the framework's entry points (`own = True`).  Weight formats, as the framework's header defines them:

  e4m3      uint8 [L, n, K], float32 scale [L, n/128, K/128]
  e4m3_mx   uint8 [L, n, K], four e8m0 codes per int32 [L, K/128, n] (groups of 32 along K)
  e2m1_mx   uint8 [L, n, K/2] (low nibble first), four e8m0 codes per int32 [L, K/128, n]
  int4      uint8 [L, n, K/2], value (q - zero) * scale per group of 32, 64 or 128 along K; bf16 scale
            and optional uint8 zero (8 where absent) [L, K/128, n, 128/group].  Within a block of 128
            elements, element 32s + 8g + j is nibble j//2 + 4(j%2) of little-endian word 4g + s.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the router of one decoded token: a launch's latency and nothing else
        dict(name="route_one", op="route", T=1, E=256, k=8, dtype="f32", renormalise=True, masked=0.0),
        # an odd batch of bf16 logits, softmax over all experts, a third of the experts masked off for each
        # token (node- or group-limited routing) and every 16th token's row masked whole (padding)
        dict(name="route_masked", op="route", T=333, E=160, k=6, dtype="bf16", renormalise=False, masked=0.33),
        # the prefill of 8 sources x 2048 tokens
        dict(name="route_prefill", op="route", T=16384, E=256, k=8, dtype="f32", renormalise=True, masked=0.0),
        # one token through the down projection of a shared expert
        dict(name="matvec_one_mx4", op="matvec", M=1, n=7168, K=2048, fmt="e2m1_mx", group=32, zero=False),
        # one token through an attention-sized projection, int4 with groups of 128
        dict(name="matvec_one_int4", op="matvec", M=1, n=4096, K=7168, fmt="int4", group=128, zero=True),
        # an odd decode batch through a wide projection, the finest int4 groups, with zero points
        dict(name="matvec_17_int4_g32", op="matvec", M=17, n=16388, K=7168, fmt="int4", group=32, zero=True),
        # a full batch through a vocabulary projection
        dict(name="matvec_64_mx4_vocab", op="matvec", M=64, n=131072, K=7168, fmt="e2m1_mx", group=32, zero=False),
        # the tiny layer (64 tokens, 8 experts, top-2): everything in cache
        dict(name="layer_tiny", op="layer", T=64, pad=0, E=8, e0=0, L=8, k=2, H=256, I=128, fmt="e4m3_mx", group=32,
             zero=False),
        # one token of a model whose 32 experts are all on this GPU, 4-bit weights
        dict(name="layer_one_mx4", op="layer", T=1, pad=0, E=32, e0=0, L=32, k=8, H=7168, I=2048, fmt="e2m1_mx",
             group=32, zero=False),
        # one rank of EP8 when each of 8 sources decodes one token: about 7 of its 32 experts are hit
        dict(name="layer_8_ep8", op="layer", T=8, pad=0, E=256, e0=32, L=32, k=8, H=7168, I=2048, fmt="e4m3", group=128,
             zero=False),
        # a captured batch of 16 with 3 padded tokens (their ids are -1), int4 experts
        dict(name="layer_16_int4", op="layer", T=16, pad=3, E=64, e0=0, L=64, k=6, H=4096, I=1408, fmt="int4",
             group=128, zero=True),
        # one rank of EP8 when each source decodes 8 tokens: most experts are hit
        dict(name="layer_64_ep8", op="layer", T=64, pad=0, E=256, e0=0, L=32, k=8, H=7168, I=2048, fmt="e4m3",
             group=128, zero=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _format(rng):
    fmt = rng.choice(("e4m3", "e4m3_mx", "e2m1_mx", "e2m1_mx", "int4", "int4", "int4"))
    if fmt == "int4":
        return dict(fmt=fmt, group=rng.choice((32, 64, 128)), zero=rng.random() < 0.5)
    return dict(fmt=fmt, group=128 if fmt == "e4m3" else 32, zero=False)


def draw(rng):
    op = rng.choice(("route", "matvec", "matvec", "layer", "layer"))
    if op == "route":
        E = _log(rng, 8, 512)
        return dict(op=op, T=min(_log(rng, 1, 16384), (16384 * 256) // E), E=E, k=rng.randint(1, min(8, E)),
                    dtype=rng.choice(("f32", "bf16")), renormalise=rng.random() < 0.5,
                    masked=rng.choice((0.0, 0.25, 0.6)))
    f = _format(rng)
    if op == "matvec":
        K = BLOCK * _log(rng, 1, 96)
        n = _log(rng, 64, min(131072, 131072 * 1792 // K))
        unit = BLOCK if f["fmt"] == "e4m3" else 4
        return dict(op=op, M=_log(rng, 1, 64), n=max(unit, n // unit * unit), K=K, **f)
    H, I = BLOCK * _log(rng, 2, 56), BLOCK * _log(rng, 1, 16)
    E = _log(rng, 8, 256)
    L = max(1, min(rng.choice((E, E // 2, E // 8)), 32 * 7168 * 2048 // (H * I)))
    T = _log(rng, 1, 64)
    return dict(op=op, T=T, pad=rng.choice((0, 0, T // 4)), E=E, e0=rng.randint(0, E - L), L=L,
                k=rng.randint(1, min(8, E)), H=H, I=I, **f)


# ---------------------------------------------------------------- inputs
def _pack_codes(code, L, n, K):
    """e8m0 codes [L, n, K/32] -> four per int32, [L, K/128, n]"""
    c = code.view(L, n, K // BLOCK, 4).to(torch.int64)
    w = c[..., 0] | (c[..., 1] << 8) | (c[..., 2] << 16) | (c[..., 3] << 24)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w)
    return w.to(torch.int32).permute(0, 2, 1).contiguous()


def _quantise(w, fmt, group, zero):
    """One expert's float32 [n, K] weight in a format: (data, scale, zero), each with a leading axis of 1."""
    n, K = w.shape
    nb = K // BLOCK
    if fmt == "e4m3":
        b = w.view(n // BLOCK, BLOCK, nb, BLOCK)
        s = (b.abs().amax(dim=(1, 3)) / 448.0).clamp_min(1e-30)
        q = (b / s[:, None, :, None]).reshape(n, K).to(torch.float8_e4m3fn).view(torch.uint8)
        return q[None], s[None], None
    if fmt in ("e4m3_mx", "e2m1_mx"):
        g = w.view(n, K // 32, 32)
        a = g.abs().amax(dim=2)
        top = 448.0 if fmt == "e4m3_mx" else 6.0
        E = torch.ceil(torch.log2((a / top).clamp_min(2.0 ** -100)))
        v = g * torch.exp2(-E)[:, :, None]
        scale = _pack_codes((E + 127).to(torch.int32)[None], 1, n, K)
        if fmt == "e4m3_mx":
            return v.reshape(n, K).to(torch.float8_e4m3fn).view(torch.uint8)[None], scale, None
        edges = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=w.device)
        c = torch.bucketize(v.abs(), edges).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        c = c.view(n, K // 2, 2)
        return (c[..., 0] | (c[..., 1] << 4))[None], scale, None
    g = w.view(n, K // group, group)
    if zero:
        lo, hi = g.amin(dim=2).clamp_max(0.0), g.amax(dim=2).clamp_min(0.0)
        s = ((hi - lo) / 15.0).clamp_min(1e-8).to(torch.bfloat16)
        z = torch.round(-lo / s.float()).clamp(0, 15)
    else:
        s = (g.abs().amax(dim=2) / 7.0).clamp_min(1e-8).to(torch.bfloat16)
        z = torch.full_like(s, 8.0, dtype=torch.float32)
    q = (torch.round(g / s.float()[:, :, None]) + z[:, :, None]).clamp(0, 15).to(torch.uint8)
    q = q.view(n, nb, 4, 4, 4, 2).permute(0, 1, 3, 2, 5, 4).reshape(n, K // 2, 2)   # words 4g + s, nibbles 4b + h
    data = (q[..., 0] | (q[..., 1] << 4))[None]
    per_block = lambda t: t.view(n, nb, BLOCK // group).permute(1, 0, 2).contiguous()[None]  # noqa: E731
    return data, per_block(s), per_block(z.to(torch.uint8)) if zero else None


def _weights(gen, L, n, K, fmt, group, zero):
    """N(0, 0.02) weights, quantised an expert (and at most 2^26 values) at a time."""
    step = max(BLOCK, min(n, (1 << 26) // K // BLOCK * BLOCK))
    data, scale, zeros = [], [], []
    for _ in range(L):
        parts = []
        for r in range(0, n, step):
            w = torch.randn((min(step, n - r), K), generator=gen, device="cuda") * 0.02
            parts.append(_quantise(w, fmt, group, zero))
        axis = 1 if fmt == "e4m3" else 2
        data.append(torch.cat([p[0] for p in parts], 1))
        scale.append(torch.cat([p[1] for p in parts], axis))
        zeros.append(torch.cat([p[2] for p in parts], 2) if zero else None)
    return dict(fmt=fmt, group=group, L=L, n=n, K=K, data=torch.cat(data), scale=torch.cat(scale),
                zero=torch.cat(zeros) if zero else None)


def _handle(w):
    import combine_expert_histogram_amd as moe
    return moe.Weight(w["fmt"], w["n"], w["K"], w["data"], w["scale"], zero=w["zero"], group=w["group"],
                      experts=w["L"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op = case["op"]
    state = dict(case)
    if op == "route":
        x = torch.randn((case["T"], case["E"]), generator=gen, device="cuda")
        if case["dtype"] == "bf16":
            x = x.to(torch.bfloat16)
        if case["masked"] > 0:
            off = torch.rand((case["T"], case["E"]), generator=gen, device="cuda") < case["masked"]
            off[15::16] = True
            x = x.masked_fill(off, -math.inf)
        state["logits"] = x
        if own:
            import combine_expert_histogram_amd as moe
            state["dims"] = moe.Dims(S=1, Ts=case["T"], k=case["k"], E=case["E"], e0=0, L=case["E"])
        return state
    if op == "matvec":
        state["x"] = torch.randn((case["M"], case["K"]), generator=gen, device="cuda").to(torch.bfloat16)
        state["w"] = _weights(gen, 1, case["n"], case["K"], case["fmt"], case["group"], case["zero"])
        state["out"] = torch.empty((case["M"], case["n"]), dtype=torch.bfloat16, device="cuda")
        if own:
            state["weight"] = _handle(state["w"])
        return state
    T, E, k, H, I = (case[c] for c in ("T", "E", "k", "H", "I"))
    state["x"] = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    top, ids = torch.randn((T, E), generator=gen, device="cuda").topk(k, dim=1)
    if case["pad"]:
        ids[T - case["pad"]:] = -1
    state["ids"] = ids.to(torch.int32).contiguous()
    state["topk_w"] = torch.softmax(top, dim=1).contiguous()
    f = (case["fmt"], case["group"], case["zero"])
    state["w1"] = _weights(gen, case["L"], 2 * I, H, *f)
    state["w2"] = _weights(gen, case["L"], H, I, *f)
    state["out"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    if own:
        import combine_expert_histogram_amd as moe
        state["dims"] = moe.Dims(S=1, Ts=T, k=k, E=E, e0=case["e0"], L=case["L"], H=H)
        state["weight1"], state["weight2"] = _handle(state["w1"]), _handle(state["w2"])
        state["ws"] = moe.alloc_few_token_workspace(state["dims"], I)
    return state


# ---------------------------------------------------------------- the plain form
def _values(w, e):
    """Expert e (a device tensor of one index, or None for the only one) as float32 [n, K]."""
    n, K, fmt = w["n"], w["K"], w["fmt"]
    pick = lambda t: t[0] if e is None else t.index_select(0, e)[0]  # noqa: E731
    data, scale = pick(w["data"]), pick(w["scale"])
    nb = K // BLOCK
    if fmt == "e4m3":
        v = data.view(torch.float8_e4m3fn).to(torch.float32).view(n // BLOCK, BLOCK, nb, BLOCK)
        return (v * scale[:, None, :, None]).view(n, K)
    if fmt in ("e4m3_mx", "e2m1_mx"):
        code = (scale[..., None] >> torch.tensor((0, 8, 16, 24), device=data.device)) & 255      # [nb, n, 4]
        s = torch.ldexp(torch.ones((), device=data.device), code.permute(1, 0, 2) - 127)         # [n, nb, 4]
        if fmt == "e4m3_mx":
            v = data.view(torch.float8_e4m3fn).to(torch.float32)
        else:
            table = torch.tensor(E2M1 + tuple(-t for t in E2M1), device=data.device)
            v = table[torch.stack((data & 15, data >> 4), dim=-1).to(torch.int32)]
        return (v.view(n, nb, 4, 32) * s[..., None]).view(n, K)
    q = torch.stack((data & 15, data >> 4), dim=-1).to(torch.float32)
    q = q.view(n, nb, 4, 4, 2, 4).permute(0, 1, 3, 2, 5, 4)                                      # s, g, h, b
    q = q.reshape(n, nb, BLOCK // w["group"], w["group"])
    s = scale.float().permute(1, 0, 2)[..., None]
    z = 8.0 if w["zero"] is None else pick(w["zero"]).float().permute(1, 0, 2)[..., None]
    return ((q - z) * s).view(n, K)


def _plain_route(state):
    x, k = state["logits"].float(), state["k"]
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    valid = top > -math.inf
    m = torch.where(valid[:, :1], top[:, :1], 0.0)
    p = torch.where(valid, torch.exp(top - m), 0.0)
    total = p.sum(1, keepdim=True) if state["renormalise"] else torch.exp(x - m).sum(1, keepdim=True)
    w = torch.where(valid, p / total, 0.0)
    return torch.where(valid, ids, -1).to(torch.int32), w


def _plain_layer(state):
    x, ids, w = state["x"].float(), state["ids"], state["topk_w"]
    T, k, L, I = state["T"], state["k"], state["L"], state["I"]
    local = ids - state["e0"]
    out = torch.zeros((T, state["H"]), device=x.device)
    if T * k <= L:      # one pass for each assignment, else one for each local expert
        flat = local.reshape(-1).to(torch.int64)
        passes = [(flat[p:p + 1].clamp(0, L - 1), p) for p in range(T * k)]
    else:
        every = torch.arange(L, device=x.device)
        passes = [(every[e:e + 1], None) for e in range(L)]
    for e, p in passes:
        c = torch.where(local == e, w, 0.0)
        if p is not None:
            c = torch.where(torch.arange(T * k, device=x.device).view(T, k) == p, c, 0.0)
        c = c.sum(1, keepdim=True)
        gu = x @ _values(state["w1"], e).t()
        gate, up = gu[:, :I], gu[:, I:]
        h = gate / (1.0 + torch.exp(-gate)) * up
        out += c * (h @ _values(state["w2"], e).t())
    return out.to(torch.bfloat16)


def run(state):
    op = state["op"]
    if own:
        import combine_expert_histogram_amd as moe
        if op == "route":
            return moe.route_topk(state["dims"], state["logits"], renormalise=state["renormalise"])
        if op == "matvec":
            return moe.matvec(state["x"], state["weight"], out=state["out"])
        return moe.few_token_layer(state["dims"], state["I"], state["x"], state["ids"], state["topk_w"],
                                   state["weight1"], state["weight2"], out=state["out"], ws=state["ws"])
    if op == "route":
        return _plain_route(state)
    if op == "matvec":
        return (state["x"].float() @ _values(state["w"], None).t()).to(torch.bfloat16)
    return _plain_layer(state)


# ---------------------------------------------------------------- what a pass cannot do without
def _weight_bytes(case, n, K):
    fmt = case["fmt"]
    if fmt == "e4m3":
        return n * K + 4 * (n // BLOCK) * (K // BLOCK)
    if fmt == "int4":
        return n * K // 2 + n * K // case["group"] * (3 if case["zero"] else 2)
    return n * K // (1 if fmt == "e4m3_mx" else 2) + n * K // 32


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return dict(bytes=T * E * (4 if case["dtype"] == "f32" else 2) + 8 * T * k, flops=T * E)
    if case["op"] == "matvec":
        M, n, K = case["M"], case["n"], case["K"]
        return dict(bytes=_weight_bytes(case, n, K) + 2 * M * (n + K), flops=2 * M * n * K)
    # expectations over the uniform routing: experts hit, and assignments that are local
    T, E, L, k, H, I = (case[c] for c in ("T", "E", "L", "k", "H", "I"))
    real = T - case["pad"]
    hit = L * (1.0 - (1.0 - k / E) ** real)
    weights = _weight_bytes(case, 2 * I, H) + _weight_bytes(case, H, I)
    return dict(bytes=int(hit * weights) + 4 * T * H + 8 * T * k, flops=int(real * k * L / E * 6 * H * I))


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_rows(w, e, r0, r1):
    """Rows r0..r1 of expert e as float64 [r1 - r0, K], element by element from the format's definition."""
    K, fmt = w["K"], w["fmt"]
    dev = w["data"].device
    kk = torch.arange(K, device=dev)
    raw = w["data"][e, r0:r1].to(torch.int64)
    if fmt.startswith("e4m3"):
        sign = 1.0 - 2.0 * (raw >> 7).double()
        ex, man = (raw >> 3) & 15, (raw & 7).double()
        v = sign * torch.where(ex == 0, man * 2.0 ** -9, (1.0 + man / 8.0) * torch.exp2(ex.double() - 7.0))
    else:
        if fmt == "int4":
            i = kk % BLOCK
            s, g, j = i // 32, i % 32 // 8, i % 8
            nib = (kk // BLOCK) * BLOCK + 8 * (4 * g + s) + j // 2 + 4 * (j % 2)
        else:
            nib = kk
        c = (raw[:, nib // 2] >> (4 * (nib % 2))) & 15
        if fmt == "int4":
            v = c.double()
        else:
            ex, man = (c >> 1) & 3, (c & 1).double()
            v = torch.where(ex == 0, man * 0.5, (1.0 + man * 0.5) * torch.exp2(ex.double() - 1.0))
            v = v * (1.0 - 2.0 * (c >> 3).double())
    if fmt == "e4m3":
        rows = torch.arange(r0, r1, device=dev) // BLOCK
        return v * w["scale"][e][rows][:, kk // BLOCK].double()
    if fmt == "int4":
        at = (kk % BLOCK) // w["group"]
        s = w["scale"][e][kk // BLOCK, r0:r1, at].double().t() if r1 - r0 == 1 else \
            w["scale"][e][:, r0:r1][kk // BLOCK, :, at].double().t()
        if w["zero"] is None:
            return (v - 8.0) * s
        return (v - w["zero"][e][:, r0:r1][kk // BLOCK, :, at].double().t()) * s
    word = w["scale"][e][:, r0:r1][kk // BLOCK].to(torch.int64)                                  # [K, rows]
    code = (word >> (8 * ((kk % BLOCK) // 32))[:, None]) & 255
    return v * torch.exp2(code.double() - 127.0).t()


def _exact_product(x, w, e):
    """x float64 [M, K] times expert e's weight, in pieces of its rows."""
    step = max(1, (1 << 24) // w["K"])
    return torch.cat([x @ _exact_rows(w, e, r, min(r + step, w["n"])).t() for r in range(0, w["n"], step)], dim=1)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "route":
        x = state["logits"].double()
        T, E = x.shape
        left, index = x.clone(), torch.arange(E, device=x.device).expand(T, E)
        ids, top = [], []
        for _ in range(case["k"]):      # the largest one left, the lowest index among equals
            m = left.max(dim=1, keepdim=True).values
            i = torch.where(left == m, index, E).min(dim=1, keepdim=True).values
            alive = m > -math.inf
            ids.append(torch.where(alive, i, -1))
            top.append(m)
            left = torch.where(index == i, -math.inf, left)
        ids, top = torch.cat(ids, 1), torch.cat(top, 1)
        first = torch.where(ids[:, :1] >= 0, top[:, :1], 0.0)
        e = torch.exp(top - first)
        total = e.sum(1, keepdim=True) if case["renormalise"] else torch.exp(x - first).sum(1, keepdim=True)
        return ids.to(torch.int32), torch.where(ids >= 0, e / total, 0.0)
    if case["op"] == "matvec":
        return _exact_product(state["x"].double(), state["w"], 0)
    x, ids, w, I = state["x"].double(), state["ids"].cpu(), state["topk_w"].double(), case["I"]
    out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=x.device)
    for e in range(case["L"]):
        hit = (ids == case["e0"] + e).nonzero()
        if not len(hit):
            continue
        t, j = hit[:, 0].to(x.device), hit[:, 1].to(x.device)
        gu = _exact_product(x[t], state["w1"], e)
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        out.index_add_(0, t, w[t, j][:, None] * _exact_product(h, state["w2"], e))
    return out
