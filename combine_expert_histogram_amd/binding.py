"""ctypes binding of libmoe_hotpath.so (the C ABI in include/moe_hotpath.h).

Argument marshalling only: torch tensors in, device pointers and sizes out to
the C functions of the same names, enqueued on torch's current HIP stream.
Every step of the path runs in the library's HIP kernels; there is no CPU
fallback, and loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_hotpath.so")

MOE_OK = 0
_STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_WORKSPACE",
           -3: "MOE_ERR_UNSUPPORTED", -4: "MOE_ERR_HIP"}

# every symbol include/moe_hotpath.h declares
EXPORTS = ("moe_status_string", "moe_capacity", "moe_route_layout_workspace", "moe_route_layout",
           "moe_route_layout_noalloc",
           "moe_quant_dispatch", "moe_grouped_gemm1_workspace", "moe_grouped_gemm1",
           "moe_quant_dispatch_mx", "moe_grouped_gemm1_mx", "moe_silu_mul_quant",
           "moe_grouped_gemm2_workspace", "moe_grouped_gemm2", "moe_silu_mul_quant_mx",
           "moe_grouped_gemm2_mx", "moe_combine", "moe_route_topk", "moe_matvec",
           "moe_few_token_layer_workspace", "moe_few_token_layer")


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)}")


class moe_dims(ctypes.Structure):
    _fields_ = [("num_sources", ctypes.c_int32), ("tokens_per_source", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("expert_begin", ctypes.c_int32), ("num_local_experts", ctypes.c_int32),
                ("hidden", ctypes.c_int32)]


class moe_weight(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("group", ctypes.c_int32), ("data", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p)]


@dataclass(frozen=True)
class Dims:
    S: int
    Ts: int
    k: int
    E: int
    e0: int
    L: int
    H: int = 128

    @property
    def T(self) -> int:
        return self.S * self.Ts

    def c(self) -> moe_dims:
        return moe_dims(self.S, self.Ts, self.k, self.E, self.e0, self.L, self.H)


_lib = None


def lib() -> ctypes.CDLL:
    """Loads the HIP library (built in-tree by combine_expert_histogram_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m combine_expert_histogram_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        D = ctypes.POINTER(moe_dims)
        sig = {
            "moe_status_string": (ctypes.c_char_p, [I32]),
            "moe_capacity": (I32, [D, ctypes.POINTER(I64), ctypes.POINTER(I64)]),
            "moe_route_layout_workspace": (I32, [D, ctypes.POINTER(SZ)]),
            "moe_route_layout": (I32, [D] + [P] * 10 + [P, SZ, P]),
            "moe_route_layout_noalloc": (I32, [D] + [P] * 10 + [P]),
            "moe_quant_dispatch": (I32, [D, P, P, P, P, P, P]),
            "moe_grouped_gemm1_workspace": (I32, [D, I32, ctypes.POINTER(SZ)]),
            "moe_grouped_gemm1": (I32, [D, I32] + [P] * 8 + [P, SZ, P]),
            "moe_quant_dispatch_mx": (I32, [D, P, P, P, P, P, P]),
            "moe_grouped_gemm1_mx": (I32, [D, I32] + [P] * 7 + [P, SZ, P]),
            "moe_silu_mul_quant": (I32, [D, I32, P, P, P, P, P]),
            "moe_grouped_gemm2_workspace": (I32, [D, I32, ctypes.POINTER(SZ)]),
            "moe_grouped_gemm2": (I32, [D, I32] + [P] * 8 + [P, SZ, P]),
            "moe_silu_mul_quant_mx": (I32, [D, I32, P, P, P, P, P]),
            "moe_grouped_gemm2_mx": (I32, [D, I32] + [P] * 8 + [P, SZ, P]),
            "moe_combine": (I32, [D, I32, P, I64, P, P, P, P]),
            "moe_route_topk": (I32, [D, P, I32, I64, I32, ctypes.c_float, P, P, P]),
            "moe_matvec": (I32, [I32, I32, I32, P, I64, ctypes.POINTER(moe_weight), P, I64, P]),
            "moe_few_token_layer_workspace": (I32, [D, I32, ctypes.POINTER(SZ)]),
            "moe_few_token_layer": (I32, [D, I32, P, P, P, ctypes.POINTER(moe_weight),
                                          ctypes.POINTER(moe_weight), P, P, SZ, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoeError(fn, status)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: torch.Tensor | None, name: str, nbytes_min: int = 0, elt: int | None = None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if elt is not None and t.element_size() != elt:
        raise ValueError(f"{name} must have {elt}-byte elements, got {t.dtype}")
    if t.numel() * t.element_size() < nbytes_min:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, needs {nbytes_min}")
    return t.data_ptr()


def _i32(t, name, n):
    if t is not None and t.dtype != torch.int32:
        raise ValueError(f"{name} must be int32")
    return _ptr(t, name, 4 * n)


# ---------------------------------------------------------------- C ABI, same names
def moe_status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def moe_capacity(d: Dims) -> tuple[int, int]:
    r, s = ctypes.c_int64(), ctypes.c_int64()
    _check("moe_capacity", lib().moe_capacity(ctypes.byref(d.c()), ctypes.byref(r), ctypes.byref(s)))
    return r.value, s.value


def moe_route_layout_workspace(d: Dims) -> int:
    b = ctypes.c_size_t()
    _check("moe_route_layout_workspace", lib().moe_route_layout_workspace(ctypes.byref(d.c()), ctypes.byref(b)))
    return b.value


def moe_grouped_gemm1_workspace(d: Dims, n: int) -> int:
    b = ctypes.c_size_t()
    _check("moe_grouped_gemm1_workspace",
           lib().moe_grouped_gemm1_workspace(ctypes.byref(d.c()), n, ctypes.byref(b)))
    return b.value


def moe_route_layout(d: Dims, topk_ids, expert_counts, expert_offsets, row_slot, row_assign,
                     assign_row, tok_slot, slot_tok, src_slot_offsets, totals, ws) -> None:
    T, k, L, S = d.T, d.k, d.L, d.S
    rows_cap, slots_cap = T * k, T
    ws_need = moe_route_layout_workspace(d)
    st = lib().moe_route_layout(
        ctypes.byref(d.c()), _i32(topk_ids, "topk_ids", T * k), _i32(expert_counts, "expert_counts", L),
        _i32(expert_offsets, "expert_offsets", L + 1), _i32(row_slot, "row_slot", rows_cap),
        _i32(row_assign, "row_assign", rows_cap), _i32(assign_row, "assign_row", T * k),
        _i32(tok_slot, "tok_slot", T), _i32(slot_tok, "slot_tok", slots_cap),
        _i32(src_slot_offsets, "src_slot_offsets", S + 1), _i32(totals, "totals", 2),
        _ptr(ws, "ws", ws_need), 0 if ws is None else ws.numel() * ws.element_size(), _stream())
    _check("moe_route_layout", st)


def moe_route_layout_noalloc(d: Dims, topk_ids, expert_counts, expert_offsets, row_slot, row_assign,
                             assign_row, tok_slot, slot_tok, src_slot_offsets, totals) -> None:
    T, k, L, S = d.T, d.k, d.L, d.S
    rows_cap, slots_cap = T * k, T
    st = lib().moe_route_layout_noalloc(
        ctypes.byref(d.c()), _i32(topk_ids, "topk_ids", T * k), _i32(expert_counts, "expert_counts", L),
        _i32(expert_offsets, "expert_offsets", L + 1), _i32(row_slot, "row_slot", rows_cap),
        _i32(row_assign, "row_assign", rows_cap), _i32(assign_row, "assign_row", T * k),
        _i32(tok_slot, "tok_slot", T), _i32(slot_tok, "slot_tok", slots_cap),
        _i32(src_slot_offsets, "src_slot_offsets", S + 1), _i32(totals, "totals", 2), _stream())
    _check("moe_route_layout_noalloc", st)


def moe_quant_dispatch(d: Dims, x_bf16, slot_tok, totals, q_e4m3, q_scale) -> None:
    T, H = d.T, d.H
    st = lib().moe_quant_dispatch(
        ctypes.byref(d.c()), _ptr(x_bf16, "x_bf16", 2 * T * H, 2), _i32(slot_tok, "slot_tok", T),
        _i32(totals, "totals", 2), _ptr(q_e4m3, "q_e4m3", T * H, 1),
        _ptr(q_scale, "q_scale", 4 * T * (H // 128), 4), _stream())
    _check("moe_quant_dispatch", st)


def moe_grouped_gemm1(d: Dims, n: int, q_e4m3, q_scale, row_slot, expert_offsets, totals,
                      w_e4m3, w_scale, y_bf16, ws=None) -> None:
    T, H, L = d.T, d.H, d.L
    rows_cap = T * d.k
    st = lib().moe_grouped_gemm1(
        ctypes.byref(d.c()), n, _ptr(q_e4m3, "q_e4m3", T * H, 1),
        _ptr(q_scale, "q_scale", 4 * T * (H // 128), 4), _i32(row_slot, "row_slot", rows_cap),
        _i32(expert_offsets, "expert_offsets", L + 1), _i32(totals, "totals", 2),
        _ptr(w_e4m3, "w_e4m3", L * n * H, 1), _ptr(w_scale, "w_scale", 4 * L * (n // 128) * (H // 128), 4),
        _ptr(y_bf16, "y_bf16", 2 * rows_cap * n, 2), _ptr(ws, "ws", moe_grouped_gemm1_workspace(d, n)),
        0 if ws is None else ws.numel() * ws.element_size(), _stream())
    _check("moe_grouped_gemm1", st)


def _u32(t, name, n):
    if t is not None and t.dtype not in (torch.int32, torch.uint32):
        raise ValueError(f"{name} must be a 32-bit integer tensor (packed e8m0 codes)")
    return _ptr(t, name, 4 * n)


def moe_quant_dispatch_mx(d: Dims, x_bf16, slot_tok, totals, q_e4m3, q_scale) -> None:
    T, H = d.T, d.H
    st = lib().moe_quant_dispatch_mx(
        ctypes.byref(d.c()), _ptr(x_bf16, "x_bf16", 2 * T * H, 2), _i32(slot_tok, "slot_tok", T),
        _i32(totals, "totals", 2), _ptr(q_e4m3, "q_e4m3", T * H, 1),
        _u32(q_scale, "q_scale", T * (H // 128)), _stream())
    _check("moe_quant_dispatch_mx", st)


def moe_grouped_gemm1_mx(d: Dims, n: int, q_e4m3, q_scale, row_slot, expert_offsets,
                         w_e4m3, w_scale, y_bf16, ws=None) -> None:
    T, H, L = d.T, d.H, d.L
    rows_cap = T * d.k
    st = lib().moe_grouped_gemm1_mx(
        ctypes.byref(d.c()), n, _ptr(q_e4m3, "q_e4m3", T * H, 1), _u32(q_scale, "q_scale", T * (H // 128)),
        _i32(row_slot, "row_slot", rows_cap), _i32(expert_offsets, "expert_offsets", L + 1),
        _ptr(w_e4m3, "w_e4m3", L * n * H, 1), _u32(w_scale, "w_scale", L * (H // 128) * n),
        _ptr(y_bf16, "y_bf16", 2 * rows_cap * n, 2), _ptr(ws, "ws", moe_grouped_gemm1_workspace(d, n)),
        0 if ws is None else ws.numel() * ws.element_size(), _stream())
    _check("moe_grouped_gemm1_mx", st)


def moe_silu_mul_quant(d: Dims, inter: int, y1_bf16, totals, h_e4m3, h_scale) -> None:
    rows_cap = d.T * d.k
    st = lib().moe_silu_mul_quant(
        ctypes.byref(d.c()), inter, _ptr(y1_bf16, "y1_bf16", 2 * rows_cap * 2 * inter, 2),
        _i32(totals, "totals", 2), _ptr(h_e4m3, "h_e4m3", rows_cap * inter, 1),
        _ptr(h_scale, "h_scale", 4 * rows_cap * (inter // 128), 4), _stream())
    _check("moe_silu_mul_quant", st)


def moe_grouped_gemm2_workspace(d: Dims, inter: int) -> int:
    b = ctypes.c_size_t()
    _check("moe_grouped_gemm2_workspace",
           lib().moe_grouped_gemm2_workspace(ctypes.byref(d.c()), inter, ctypes.byref(b)))
    return b.value


def moe_grouped_gemm2(d: Dims, inter: int, h_e4m3, h_scale, expert_offsets, row_assign, topk_w,
                      w2_e4m3, w2_scale, y2_bf16, ws=None) -> None:
    T, H, L = d.T, d.H, d.L
    rows_cap = T * d.k
    if topk_w is not None and topk_w.dtype != torch.float32:
        raise ValueError("topk_w must be float32")
    st = lib().moe_grouped_gemm2(
        ctypes.byref(d.c()), inter, _ptr(h_e4m3, "h_e4m3", rows_cap * inter, 1),
        _ptr(h_scale, "h_scale", 4 * rows_cap * (inter // 128), 4),
        _i32(expert_offsets, "expert_offsets", L + 1), _i32(row_assign, "row_assign", rows_cap),
        _ptr(topk_w, "topk_w", 4 * T * d.k, 4), _ptr(w2_e4m3, "w2_e4m3", L * H * inter, 1),
        _ptr(w2_scale, "w2_scale", 4 * L * (H // 128) * (inter // 128), 4),
        _ptr(y2_bf16, "y2_bf16", 2 * rows_cap * H, 2), _ptr(ws, "ws", moe_grouped_gemm2_workspace(d, inter)),
        0 if ws is None else ws.numel() * ws.element_size(), _stream())
    _check("moe_grouped_gemm2", st)


def moe_silu_mul_quant_mx(d: Dims, inter: int, y1_bf16, totals, h_e4m3, h_scale) -> None:
    rows_cap = d.T * d.k
    st = lib().moe_silu_mul_quant_mx(
        ctypes.byref(d.c()), inter, _ptr(y1_bf16, "y1_bf16", 2 * rows_cap * 2 * inter, 2),
        _i32(totals, "totals", 2), _ptr(h_e4m3, "h_e4m3", rows_cap * inter, 1),
        _u32(h_scale, "h_scale", rows_cap * (inter // 128)), _stream())
    _check("moe_silu_mul_quant_mx", st)


def moe_grouped_gemm2_mx(d: Dims, inter: int, h_e4m3, h_scale, expert_offsets, row_assign, topk_w,
                         w2_e4m3, w2_scale, y2_bf16, ws=None) -> None:
    T, H, L = d.T, d.H, d.L
    rows_cap = T * d.k
    if topk_w is not None and topk_w.dtype != torch.float32:
        raise ValueError("topk_w must be float32")
    st = lib().moe_grouped_gemm2_mx(
        ctypes.byref(d.c()), inter, _ptr(h_e4m3, "h_e4m3", rows_cap * inter, 1),
        _u32(h_scale, "h_scale", rows_cap * (inter // 128)),
        _i32(expert_offsets, "expert_offsets", L + 1), _i32(row_assign, "row_assign", rows_cap),
        _ptr(topk_w, "topk_w", 4 * T * d.k, 4), _ptr(w2_e4m3, "w2_e4m3", L * H * inter, 1),
        _u32(w2_scale, "w2_scale", L * (inter // 128) * H),
        _ptr(y2_bf16, "y2_bf16", 2 * rows_cap * H, 2), _ptr(ws, "ws", moe_grouped_gemm2_workspace(d, inter)),
        0 if ws is None else ws.numel() * ws.element_size(), _stream())
    _check("moe_grouped_gemm2_mx", st)


def moe_combine(d: Dims, width: int, y_bf16, assign_row, topk_w, out_bf16) -> None:
    T, k = d.T, d.k
    y_rows = 0 if y_bf16 is None else y_bf16.numel() // max(width, 1)
    if topk_w is not None and topk_w.dtype != torch.float32:
        raise ValueError("topk_w must be float32")
    st = lib().moe_combine(
        ctypes.byref(d.c()), width, _ptr(y_bf16, "y_bf16", 0, 2), y_rows,
        _i32(assign_row, "assign_row", T * k), _ptr(topk_w, "topk_w", 4 * T * k, 4),
        _ptr(out_bf16, "out_bf16", 2 * T * width, 2), _stream())
    _check("moe_combine", st)


# ---------------------------------------------------------------- conveniences
LAYOUT_KEYS = ("expert_counts", "expert_offsets", "row_slot", "row_assign", "assign_row",
               "tok_slot", "slot_tok", "src_slot_offsets", "totals")


def alloc_layout(d: Dims, device="cuda") -> dict:
    rows_cap, slots_cap = d.T * d.k, d.T
    sizes = dict(expert_counts=d.L, expert_offsets=d.L + 1, row_slot=rows_cap, row_assign=rows_cap,
                 assign_row=d.T * d.k, tok_slot=d.T, slot_tok=slots_cap, src_slot_offsets=d.S + 1,
                 totals=2)
    out = {k: torch.empty(max(v, 1), dtype=torch.int32, device=device) for k, v in sizes.items()}
    out["ws"] = torch.empty(max(moe_route_layout_workspace(d) // 4, 1), dtype=torch.int32, device=device)
    return out


def route_layout(d: Dims, topk_ids, out: dict | None = None) -> dict:
    out = alloc_layout(d, topk_ids.device) if out is None else out
    moe_route_layout(d, topk_ids, *(out[k] for k in LAYOUT_KEYS), out["ws"])
    return out


def quant_dispatch(d: Dims, x_bf16, lay: dict, q=None, q_scale=None):
    dev = x_bf16.device
    q = torch.empty((max(d.T, 1), d.H), dtype=torch.uint8, device=dev) if q is None else q
    q_scale = (torch.empty((max(d.T, 1), d.H // 128), dtype=torch.float32, device=dev)
               if q_scale is None else q_scale)
    moe_quant_dispatch(d, x_bf16, lay["slot_tok"], lay["totals"], q, q_scale)
    return q, q_scale


def alloc_gemm1_workspace(d: Dims, n: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(moe_grouped_gemm1_workspace(d, n) // 4, 1), dtype=torch.float32, device=device)


def grouped_gemm1(d: Dims, n: int, q, q_scale, lay: dict, w_e4m3, w_scale, y=None, ws=None):
    y = torch.empty((max(d.T * d.k, 1), n), dtype=torch.bfloat16, device=q.device) if y is None else y
    ws = alloc_gemm1_workspace(d, n, q.device) if ws is None else ws
    moe_grouped_gemm1(d, n, q, q_scale, lay["row_slot"], lay["expert_offsets"], lay["totals"],
                      w_e4m3, w_scale, y, ws)
    return y


def quant_dispatch_mx(d: Dims, x_bf16, lay: dict, q=None, q_scale=None):
    dev = x_bf16.device
    q = torch.empty((max(d.T, 1), d.H), dtype=torch.uint8, device=dev) if q is None else q
    q_scale = (torch.empty((max(d.T, 1), d.H // 128), dtype=torch.int32, device=dev)
               if q_scale is None else q_scale)
    moe_quant_dispatch_mx(d, x_bf16, lay["slot_tok"], lay["totals"], q, q_scale)
    return q, q_scale


def grouped_gemm1_mx(d: Dims, n: int, q, q_scale, lay: dict, w_e4m3, w_scale, y=None, ws=None):
    y = torch.empty((max(d.T * d.k, 1), n), dtype=torch.bfloat16, device=q.device) if y is None else y
    ws = alloc_gemm1_workspace(d, n, q.device) if ws is None else ws
    moe_grouped_gemm1_mx(d, n, q, q_scale, lay["row_slot"], lay["expert_offsets"], w_e4m3, w_scale, y, ws)
    return y


def silu_mul_quant(d: Dims, inter: int, y1, lay: dict, h=None, h_scale=None):
    rows = max(d.T * d.k, 1)
    h = torch.empty((rows, inter), dtype=torch.uint8, device=y1.device) if h is None else h
    h_scale = (torch.empty((rows, inter // 128), dtype=torch.float32, device=y1.device)
               if h_scale is None else h_scale)
    moe_silu_mul_quant(d, inter, y1, lay["totals"], h, h_scale)
    return h, h_scale


def alloc_gemm2_workspace(d: Dims, inter: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(moe_grouped_gemm2_workspace(d, inter) // 4, 1), dtype=torch.float32, device=device)


def grouped_gemm2(d: Dims, inter: int, h, h_scale, lay: dict, topk_w, w2_e4m3, w2_scale, y2=None, ws=None):
    y2 = torch.empty((max(d.T * d.k, 1), d.H), dtype=torch.bfloat16, device=h.device) if y2 is None else y2
    ws = alloc_gemm2_workspace(d, inter, h.device) if ws is None else ws
    moe_grouped_gemm2(d, inter, h, h_scale, lay["expert_offsets"], lay["row_assign"], topk_w, w2_e4m3, w2_scale,
                      y2, ws)
    return y2


def silu_mul_quant_mx(d: Dims, inter: int, y1, lay: dict, h=None, h_scale=None):
    rows = max(d.T * d.k, 1)
    h = torch.empty((rows, inter), dtype=torch.uint8, device=y1.device) if h is None else h
    h_scale = (torch.empty((rows, inter // 128), dtype=torch.int32, device=y1.device)
               if h_scale is None else h_scale)
    moe_silu_mul_quant_mx(d, inter, y1, lay["totals"], h, h_scale)
    return h, h_scale


def grouped_gemm2_mx(d: Dims, inter: int, h, h_scale, lay: dict, topk_w, w2_e4m3, w2_scale, y2=None, ws=None):
    y2 = torch.empty((max(d.T * d.k, 1), d.H), dtype=torch.bfloat16, device=h.device) if y2 is None else y2
    ws = alloc_gemm2_workspace(d, inter, h.device) if ws is None else ws
    moe_grouped_gemm2_mx(d, inter, h, h_scale, lay["expert_offsets"], lay["row_assign"], topk_w, w2_e4m3,
                         w2_scale, y2, ws)
    return y2


def combine(d: Dims, width: int, y_bf16, assign_row, topk_w, out=None):
    out = torch.empty((max(d.T, 1), width), dtype=torch.bfloat16, device=y_bf16.device) if out is None else out
    moe_combine(d, width, y_bf16, assign_row, topk_w, out)
    return out


# ---------------------------------------------------------------- few tokens
WEIGHT_FORMATS = {"e4m3": 0, "e4m3_mx": 1, "e2m1_mx": 2, "int4": 3}
_BF16_BITS = (torch.bfloat16, torch.int16, torch.uint16)
_PACKED = (torch.int32, torch.uint32)
_E4M3 = (torch.uint8, torch.float8_e4m3fn)


class Weight:
    """A weight matrix [n, k], or `experts` of them one after the other, in one of the header's formats
    (moe_weight_format): "e4m3", "e4m3_mx", "e2m1_mx" or "int4".  Holds its tensors and checks them once."""

    def __init__(self, fmt: str, n: int, k: int, data, scale, zero=None, group: int = 128, experts: int = 1):
        if fmt not in WEIGHT_FORMATS:
            raise ValueError(f"fmt must be one of {sorted(WEIGHT_FORMATS)}, got {fmt!r}")
        if n < 4 or n % 4 or k < 128 or k % 128 or experts < 1:
            raise ValueError(f"n must be a multiple of 4, k of 128 and experts positive, got {n}, {k}, {experts}")
        if fmt == "e4m3" and n % 128:
            raise ValueError("an e4m3 weight's n must be a multiple of 128")
        if fmt == "int4" and group not in (32, 64, 128):
            raise ValueError(f"group must be 32, 64 or 128, got {group}")
        if fmt != "int4" and zero is not None:
            raise ValueError("zero points belong to int4 weights")
        numel, blocks = experts * n * k, experts * n * (k // 128)
        if fmt in ("e2m1_mx", "int4"):
            self._tensor(data, "data", (torch.uint8,), numel // 2)
        else:
            self._tensor(data, "data", _E4M3, numel)
        if fmt == "e4m3":
            self._tensor(scale, "scale", (torch.float32,), blocks // 128)
        elif fmt == "int4":
            self._tensor(scale, "scale", _BF16_BITS, numel // group)
        else:
            self._tensor(scale, "scale", _PACKED, blocks)
        if zero is not None:
            self._tensor(zero, "zero", (torch.uint8,), numel // group)
        if len({t.device for t in (data, scale, zero) if t is not None}) != 1:
            raise ValueError("data, scale and zero must be on one device")
        self.fmt, self.n, self.k, self.group, self.experts = fmt, n, k, group, experts
        self.data, self.scale, self.zero, self.device = data, scale, zero, data.device
        self._c = moe_weight(WEIGHT_FORMATS[fmt], group if fmt == "int4" else 0, data.data_ptr(), scale.data_ptr(),
                             None if zero is None else zero.data_ptr())
        self._ref = ctypes.byref(self._c)

    @staticmethod
    def _tensor(t, name, dtypes, numel):
        if t.dtype not in dtypes:
            raise ValueError(f"{name} must be one of {dtypes}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.numel() != numel:
            raise ValueError(f"{name} must hold {numel} elements, got {t.numel()}")
        if t.data_ptr() % 16:
            raise ValueError(f"{name} must be 16-byte aligned")

    def c(self):
        return self._ref


def _blocks_first(t: torch.Tensor, per_block: int) -> torch.Tensor:
    """[.., n, k/128 * per_block] -> contiguous [.., k/128, n, per_block], always a copy (with one K block the transposed
    view is contiguous already)"""
    t = t.unflatten(-1, (-1, per_block))
    return t.transpose(-3, -2).clone(memory_format=torch.contiguous_format)


def _pack_nibbles(q: torch.Tensor) -> torch.Tensor:
    q = q.unflatten(-1, (-1, 2))
    return (q[..., 0] | (q[..., 1] << 4)).contiguous()


def int4_weight(q: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor | None = None) -> Weight:
    """Lays out an int4 weight: codes q uint8 [(experts,) n, k] in 0..15, scale [.., n, k/group] (rounded to
    bf16) and, optionally, integer zero points of scale's shape; value = (q - zero) * scale, zero = 8 if absent."""
    if q.dtype != torch.uint8 or q.dim() not in (2, 3) or q.shape[-1] % 128 or not q.numel():
        raise ValueError("q must be uint8 [(experts,) n, k] with k a multiple of 128")
    if scale.shape[:-1] != q.shape[:-1] or (zero is not None and zero.shape != scale.shape):
        raise ValueError("scale (and zero) must be [(experts,) n, k/group]")
    n, k = q.shape[-2:]
    group = k // max(scale.shape[-1], 1)
    if group not in (32, 64, 128) or scale.shape[-1] * group != k:
        raise ValueError("scale must have k/32, k/64 or k/128 columns")
    if int(q.max()) > 15 or (zero is not None and not bool(((zero >= 0) & (zero <= 15) & (zero % 1 == 0)).all())):
        raise ValueError("codes and zero points must be whole numbers in 0..15")
    # k = 32 s + 8 g + 2 h + b of a block is nibble 4 b + h of word 4 g + s
    w = q.unflatten(-1, (k // 128, 4, 4, 4, 2))
    lead = w.dim() - 4
    w = w.permute(*range(lead), lead + 1, lead, lead + 3, lead + 2).reshape(*q.shape)
    return Weight("int4", n, k, _pack_nibbles(w), _blocks_first(scale.to(torch.bfloat16), 128 // group),
                  zero=None if zero is None else _blocks_first(zero.to(torch.uint8), 128 // group), group=group,
                  experts=q.shape[0] if q.dim() == 3 else 1)


def e2m1_weight(codes: torch.Tensor, e8m0: torch.Tensor) -> Weight:
    """Lays out an e2m1 weight: codes uint8 [(experts,) n, k] in 0..15 and the e8m0 codes uint8 [.., n, k/32]."""
    if codes.dtype != torch.uint8 or codes.dim() not in (2, 3) or codes.shape[-1] % 128 or not codes.numel():
        raise ValueError("codes must be uint8 [(experts,) n, k] with k a multiple of 128")
    n, k = codes.shape[-2:]
    if e8m0.dtype != torch.uint8 or e8m0.shape != (*codes.shape[:-1], k // 32):
        raise ValueError("e8m0 must be uint8 [(experts,) n, k/32]")
    if int(codes.max()) > 15:
        raise ValueError("codes must be in 0..15")
    packed = _blocks_first(e8m0, 4).view(torch.int32).squeeze(-1)
    return Weight("e2m1_mx", n, k, _pack_nibbles(codes), packed, experts=codes.shape[0] if codes.dim() == 3 else 1)


def _same_device(*named) -> torch.device:
    """The one device of the tensors, which has to be a GPU."""
    device = named[0][1].device
    if device.type != "cuda":
        raise ValueError(f"{named[0][0]} must be a device tensor")
    for name, t in named[1:]:
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, {named[0][0]} on {device}")
    return device


def _dtype(t: torch.Tensor, name: str, dtypes) -> None:
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {dtypes}, got {t.dtype}")


def _rows(t: torch.Tensor, name: str, rows: int, cols: int) -> int:
    """Row stride (elements) of a [rows, cols] tensor whose rows are contiguous."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")
    step, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return cols if rows <= 1 else step


def _launch(device: torch.device, fn: str, *args) -> None:
    """Calls fn(*args, stream) with `device` current, on its current stream.  The raw handle takes 0.1 us where a
    torch.cuda.Stream object takes 1.9, of the 5 us that a launch costs."""
    call, index = getattr(_lib or lib(), fn), device.index
    if index == torch.cuda.current_device():
        status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != MOE_OK:
        raise MoeError(fn, status)


def moe_route_topk(d: Dims, logits, renormalise: bool, scale: float, topk_ids, topk_w) -> None:
    device = _same_device(("logits", logits), ("topk_ids", topk_ids), ("topk_w", topk_w))
    _dtype(logits, "logits", (torch.float32, torch.bfloat16))
    _dtype(topk_w, "topk_w", (torch.float32,))
    stride = _rows(logits, "logits", d.T, d.E)
    _launch(device, "moe_route_topk", ctypes.byref(d.c()), logits.data_ptr(), int(logits.dtype == torch.bfloat16),
            stride, int(bool(renormalise)), float(scale), _i32(topk_ids, "topk_ids", d.T * d.k),
            _ptr(topk_w, "topk_w", 4 * d.T * d.k))


def moe_matvec(x_bf16, weight: Weight, y_bf16) -> None:
    device = _same_device(("x_bf16", x_bf16), ("weight", weight), ("y_bf16", y_bf16))
    _dtype(x_bf16, "x_bf16", _BF16_BITS)
    _dtype(y_bf16, "y_bf16", _BF16_BITS)
    if weight.experts != 1:
        raise ValueError(f"weight must be one matrix, got {weight.experts}")
    m = x_bf16.shape[0]
    xs, ys = _rows(x_bf16, "x_bf16", m, weight.k), _rows(y_bf16, "y_bf16", m, weight.n)
    _launch(device, "moe_matvec", m, weight.n, weight.k, x_bf16.data_ptr(), xs, weight.c(), y_bf16.data_ptr(), ys)


def moe_few_token_layer_workspace(d: Dims, inter: int) -> int:
    b = ctypes.c_size_t()
    _check("moe_few_token_layer_workspace",
           lib().moe_few_token_layer_workspace(ctypes.byref(d.c()), inter, ctypes.byref(b)))
    return b.value


def moe_few_token_layer(d: Dims, inter: int, x_bf16, topk_ids, topk_w, w1: Weight, w2: Weight, out_bf16, ws) -> None:
    device = _same_device(("x_bf16", x_bf16), ("topk_ids", topk_ids), ("topk_w", topk_w), ("w1", w1), ("w2", w2),
                          ("out_bf16", out_bf16), ("ws", ws))
    _dtype(x_bf16, "x_bf16", _BF16_BITS)
    _dtype(topk_w, "topk_w", (torch.float32,))
    _dtype(out_bf16, "out_bf16", _BF16_BITS)
    for name, w, shape in (("w1", w1, (d.L, 2 * inter, d.H)), ("w2", w2, (d.L, d.H, inter))):
        if (w.experts, w.n, w.k) != shape:
            raise ValueError(f"{name} must be {shape[0]} matrices of [{shape[1]}, {shape[2]}], got {w.experts} of "
                             f"[{w.n}, {w.k}]")
    T = d.T
    _launch(device, "moe_few_token_layer", ctypes.byref(d.c()), inter, _ptr(x_bf16, "x_bf16", 2 * T * d.H),
            _i32(topk_ids, "topk_ids", T * d.k), _ptr(topk_w, "topk_w", 4 * T * d.k), w1.c(), w2.c(),
            _ptr(out_bf16, "out_bf16", 2 * T * d.H), _ptr(ws, "ws"), ws.numel() * ws.element_size())


def route_topk(d: Dims, logits, renormalise: bool = True, scale: float = 1.0, topk_ids=None, topk_w=None):
    """logits [T, E] (float32 or bfloat16) -> (topk_ids int32 [T, k], topk_w float32 [T, k])"""
    topk_ids = (torch.empty((d.T, d.k), dtype=torch.int32, device=logits.device) if topk_ids is None else topk_ids)
    topk_w = torch.empty((d.T, d.k), dtype=torch.float32, device=logits.device) if topk_w is None else topk_w
    moe_route_topk(d, logits, renormalise, scale, topk_ids, topk_w)
    return topk_ids, topk_w


def matvec(x, weight: Weight, out=None):
    """x bf16 [m, k] times a weight [n, k], transposed -> bf16 [m, n]"""
    out = torch.empty((x.shape[0], weight.n), dtype=torch.bfloat16, device=x.device) if out is None else out
    moe_matvec(x, weight, out)
    return out


def alloc_few_token_workspace(d: Dims, inter: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(moe_few_token_layer_workspace(d, inter), 16), dtype=torch.uint8, device=device)


def few_token_layer(d: Dims, inter: int, x, topk_ids, topk_w, w1: Weight, w2: Weight, out=None, ws=None):
    """The expert layer on x bf16 [T, H] -> bf16 [T, H]: w1 the L gate-and-up matrices, w2 the down matrices."""
    out = torch.empty((d.T, d.H), dtype=torch.bfloat16, device=x.device) if out is None else out
    ws = alloc_few_token_workspace(d, inter, x.device) if ws is None else ws
    moe_few_token_layer(d, inter, x, topk_ids, topk_w, w1, w2, out, ws)
    return out
