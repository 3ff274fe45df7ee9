"""The serving forms for a few tokens: the router's choice, products with block-scaled weights (8 and 4 bits), and
the whole expert layer.

TEST INFRASTRUCTURE (see the package docstring).

Everything is evaluated in float64 from the formats' definitions; nothing is rounded on the way.  The definitions are
plain ones (a gated-MLP expert, a softmax over the chosen or over all experts, a value per code and group scale), so
there is no source to follow beyond them.
  * route_topk: the k largest logits of a row, larger first, ties to the lower id; -inf and NaN are never chosen; the
    slots left over hold id -1 and weight 0.
  * e2m1 codes: bit 3 the sign; exponent field 0 holds 0 and 0.5, else (1 + m/2) * 2^(e-1): 1, 1.5, 2, 3, 4, 6.
  * int4: (q - zero) * scale; the storage order (unpack_int4) puts element 32s + 8g + j of a block of 128 into nibble
    j/2 + 4*(j%2) of little-endian word 4g + s.
"""
from __future__ import annotations

import numpy as np

from . import fp8, mx

BLOCK = 128


def route_topk(logits: np.ndarray, k: int, renormalise: bool, scale: float = 1.0):
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        ok = [e for e in range(E) if x[t, e] > -np.inf]          # NaN compares false
        order = sorted(ok, key=lambda e: (-x[t, e], e))[:k]
        if not order:
            continue
        top = x[t, order[0]]
        term = lambda e: 1.0 if x[t, e] == top else np.exp(x[t, e] - top)  # noqa: E731
        total = sum(term(e) for e in (order if renormalise else ok))
        for j, e in enumerate(order):
            ids[t, j], w[t, j] = e, scale * term(e) / total
    return ids, w


def e2m1_decode(codes: np.ndarray) -> np.ndarray:
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 1) & 3, c & 1
    v = np.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * np.exp2(e - 1.0))
    return np.where(c >> 3 & 1, -v, v)


def unpack_int4(data: np.ndarray) -> np.ndarray:
    """uint8 [n, k/2] -> codes [n, k] in element order"""
    n, half = data.shape
    k = 2 * half
    out = np.zeros((n, k), np.int64)
    for i in range(k):
        b, r = divmod(i, BLOCK)
        s, g, j = r // 32, r % 32 // 8, r % 8
        nibble = b * BLOCK + 8 * (4 * g + s) + j // 2 + 4 * (j % 2)
        out[:, i] = (data[:, nibble // 2] >> (4 * (nibble % 2))) & 15
    return out


def dequant(fmt: str, data: np.ndarray, scale: np.ndarray, zero=None, group: int = 128) -> np.ndarray:
    """One matrix in a weight format -> float64 [n, k].  scale: float32 [n/128, k/128], packed uint32 [k/128, n], or
    (int4) float values [k/128, n, 128/group]; zero like the latter."""
    if fmt == "e4m3":
        v = fp8.decode(data).astype(np.float64)
        return v * np.asarray(scale, np.float64).repeat(128, 0).repeat(128, 1)
    if fmt in ("e4m3_mx", "e2m1_mx"):
        E = mx.unpack_codes(np.ascontiguousarray(np.asarray(scale, np.uint32).T)).astype(np.int64) - 127   # [n, k/32]
        if fmt == "e4m3_mx":
            v = fp8.decode(data).astype(np.float64)
        else:
            v = e2m1_decode(np.stack([data & 15, data >> 4], -1).reshape(data.shape[0], -1))
        return v * np.exp2(E.astype(np.float64)).repeat(32, 1)
    q = unpack_int4(data).astype(np.float64)
    n = q.shape[0]
    flat = lambda t: np.asarray(t, np.float64).transpose(1, 0, 2).reshape(n, -1).repeat(group, 1)  # noqa: E731
    return (q - (8.0 if zero is None else flat(zero))) * flat(scale)


def layer(x: np.ndarray, ids: np.ndarray, topk_w: np.ndarray, e0: int, w1: np.ndarray, w2: np.ndarray):
    """x [T, H], ids and topk_w [T, k], w1 float64 [L, 2I, H], w2 float64 [L, H, I].  Returns (out [T, H], bound
    [T, H]): bound is sum |w| |W2| |h|, the size of the terms that a rounding of h is relative to."""
    x = np.asarray(x, np.float64)
    T, H = x.shape
    I = w2.shape[2]
    out, size = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j]) - e0
            if not 0 <= e < w1.shape[0]:
                continue
            gu = w1[e] @ x[t]
            gate, up = gu[:I], gu[I:]
            with np.errstate(over="ignore"):
                h = gate / (1.0 + np.exp(-gate)) * up
            wt = float(topk_w[t, j])
            out[t] += wt * (w2[e] @ h)
            size[t] += abs(wt) * (np.abs(w2[e]) @ np.abs(h))
    return out, size
