"""The dense layers' host side (no GPU): workspace sizes and every refusal, with pointers that are never followed."""
import ctypes

import pytest
import torch

import combine_expert_histogram_amd as moe
from combine_expert_histogram_amd import binding as b

OK, INVALID, WORKSPACE, UNSUPPORTED = 0, -1, -2, -3
BF16, FP16, FP32 = 0, 1, 2
HERE = 1 << 20               # an address that no call below follows
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(b.LIB_PATH):
        from combine_expert_histogram_amd import build
        build.build()
    return b.lib()


def call(L, fn, base, **change):
    """fn with its arguments by name, some of them changed"""
    args = dict(base)
    for k, v in change.items():
        assert k in args, k
        args[k] = v
    return getattr(L, fn)(*args.values())


LINEAR = dict(m=300, n=64, k=128, dtype=BF16, x=HERE, x_stride=128, w=HERE, w_stride=128, bias=HERE, act=2, residual=HERE,
              residual_stride=64, z=HERE, z_stride=64, y=HERE, y_stride=64, ws=HERE, ws_bytes=BIG, stream=None)
LINEAR_BACK = dict(m=300, n=64, k=128, dtype=FP16, dy=HERE, dy_stride=64, x=HERE, x_stride=128, w=HERE, w_stride=128, act=2,
                   z=HERE, z_stride=64, dx=HERE, dx_stride=128, dw=HERE, dw_stride=128, dbias=HERE, ws=HERE, ws_bytes=BIG,
                   stream=None)
GATED = dict(m=300, inter=32, hidden=128, dtype=BF16, x=HERE, x_stride=128, w=HERE, w_stride=128, act=2, gu=HERE, gu_stride=64,
             h=HERE, h_stride=32, ws=HERE, ws_bytes=BIG, stream=None)
GATED_BACK = dict(m=300, inter=32, hidden=128, dtype=BF16, dh=HERE, dh_stride=32, gu=HERE, gu_stride=64, x=HERE, x_stride=128,
                  w=HERE, w_stride=128, act=2, dx=HERE, dx_stride=128, dw=HERE, dw_stride=128, ws=HERE, ws_bytes=BIG, stream=None)
NORM = dict(rows=4, cols=32, dtype=BF16, param_dtype=FP32, x=HERE, x_stride=32, weight=HERE, bias=HERE, eps=1e-5, y=HERE,
            y_stride=32, mean=HERE, rstd=HERE, stream=None)
NORM_BACK = dict(rows=4, cols=32, dtype=BF16, param_dtype=FP32, dy=HERE, dy_stride=32, x=HERE, x_stride=32, weight=HERE,
                 mean=HERE, rstd=HERE, dx=HERE, dx_stride=32, dweight=HERE, dbias=HERE, ws=HERE, ws_bytes=BIG, stream=None)

FAR = 1 << 22
REFUSED = [
    ("moe_linear", LINEAR, INVALID, [
        dict(m=-1), dict(n=0), dict(k=0), dict(n=-5), dict(dtype=FP32), dict(dtype=3), dict(dtype=-1), dict(act=-1),
        dict(act=5), dict(x=None), dict(w=None), dict(y=None), dict(x=HERE + 1), dict(w=HERE + 1), dict(y=HERE + 1),
        dict(bias=HERE + 1), dict(residual=HERE + 1), dict(z=HERE + 1), dict(x_stride=127), dict(w_stride=127),
        dict(y_stride=63), dict(residual_stride=63), dict(z_stride=63), dict(ws=HERE + 8, k=4096, x_stride=4096, w_stride=4096)]),
    ("moe_linear", LINEAR, UNSUPPORTED, [
        dict(x_stride=FAR), dict(w_stride=FAR), dict(y_stride=FAR), dict(residual_stride=FAR), dict(z_stride=FAR),
        dict(m=1 << 30), dict(n=1 << 30), dict(k=1 << 30), dict(m=1 << 29, n=1 << 29)]),
    ("moe_linear", LINEAR, WORKSPACE, [
        dict(ws=None, k=4096, x_stride=4096, w_stride=4096), dict(ws_bytes=16, k=4096, x_stride=4096, w_stride=4096)]),
    ("moe_linear_backward", LINEAR_BACK, INVALID, [
        dict(m=-1), dict(n=0), dict(k=0), dict(dtype=FP32), dict(act=5), dict(act=-1), dict(dy=None), dict(x=None),
        dict(w=None), dict(z=None), dict(dy=HERE + 1), dict(x=HERE + 1), dict(w=HERE + 1), dict(z=HERE + 1), dict(dx=HERE + 1),
        dict(dw=HERE + 1), dict(dbias=HERE + 1), dict(dy_stride=63), dict(x_stride=127), dict(w_stride=127), dict(z_stride=63),
        dict(dx_stride=127), dict(dw_stride=127), dict(ws=HERE + 8), dict(m=0, dw_stride=127)]),
    ("moe_linear_backward", LINEAR_BACK, UNSUPPORTED, [
        dict(dy_stride=FAR), dict(x_stride=FAR), dict(w_stride=FAR), dict(z_stride=FAR), dict(dx_stride=FAR),
        dict(dw_stride=FAR), dict(m=1 << 30)]),
    ("moe_linear_backward", LINEAR_BACK, WORKSPACE, [dict(ws=None), dict(ws_bytes=64)]),
    ("moe_gated_linear", GATED, INVALID, [
        dict(m=-1), dict(inter=0), dict(hidden=0), dict(dtype=FP32), dict(act=5), dict(x=None), dict(w=None), dict(h=None),
        dict(x=HERE + 1), dict(w=HERE + 1), dict(h=HERE + 1), dict(gu=HERE + 1), dict(x_stride=127), dict(w_stride=127),
        dict(h_stride=31), dict(gu_stride=63), dict(ws=HERE + 8, hidden=4096, x_stride=4096, w_stride=4096)]),
    ("moe_gated_linear", GATED, UNSUPPORTED, [
        dict(x_stride=FAR), dict(w_stride=FAR), dict(h_stride=FAR), dict(gu_stride=FAR), dict(inter=1 << 29),
        dict(inter=(1 << 31) - 1)]),
    ("moe_gated_linear", GATED, WORKSPACE, [dict(ws_bytes=16, hidden=4096, x_stride=4096, w_stride=4096)]),
    ("moe_gated_linear_backward", GATED_BACK, INVALID, [
        dict(m=-1), dict(inter=0), dict(hidden=-1), dict(dtype=FP32), dict(act=9), dict(dh=None), dict(gu=None), dict(x=None),
        dict(w=None), dict(dh=HERE + 1), dict(gu=HERE + 1), dict(x=HERE + 1), dict(w=HERE + 1), dict(dx=HERE + 1),
        dict(dw=HERE + 1), dict(dh_stride=31), dict(gu_stride=63), dict(x_stride=127), dict(w_stride=127), dict(dx_stride=127),
        dict(dw_stride=127), dict(ws=HERE + 8)]),
    ("moe_gated_linear_backward", GATED_BACK, UNSUPPORTED, [
        dict(dh_stride=FAR), dict(gu_stride=FAR), dict(x_stride=FAR), dict(w_stride=FAR), dict(dx_stride=FAR),
        dict(dw_stride=FAR), dict(inter=(1 << 31) - 1)]),
    ("moe_gated_linear_backward", GATED_BACK, WORKSPACE, [dict(ws=None), dict(ws_bytes=64)]),
    ("moe_layer_norm", NORM, INVALID, [
        dict(rows=-1), dict(cols=0), dict(dtype=3), dict(dtype=-1), dict(param_dtype=FP16), dict(dtype=FP32, param_dtype=BF16),
        dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(y=None), dict(x=HERE + 1), dict(y=HERE + 1),
        dict(weight=HERE + 2), dict(bias=HERE + 2), dict(mean=HERE + 2), dict(rstd=HERE + 2), dict(x_stride=31),
        dict(y_stride=31), dict(dtype=FP32, x=HERE + 2)]),
    ("moe_layer_norm", NORM, UNSUPPORTED, [dict(rows=1 << 30), dict(cols=1 << 30)]),
    ("moe_layer_norm_backward", NORM_BACK, INVALID, [
        dict(rows=-1), dict(cols=0), dict(dtype=3), dict(param_dtype=FP16), dict(dy=None), dict(x=None), dict(mean=None),
        dict(rstd=None), dict(dy=HERE + 1), dict(x=HERE + 1), dict(weight=HERE + 2), dict(mean=HERE + 2), dict(rstd=HERE + 2),
        dict(dx=HERE + 1), dict(dweight=HERE + 2), dict(dbias=HERE + 2), dict(dy_stride=31), dict(x_stride=31),
        dict(dx_stride=31), dict(ws=HERE + 8)]),
    ("moe_layer_norm_backward", NORM_BACK, UNSUPPORTED, [dict(rows=1 << 30), dict(cols=1 << 30)]),
    ("moe_layer_norm_backward", NORM_BACK, WORKSPACE, [dict(ws=None), dict(ws_bytes=64)]),
]


@pytest.mark.parametrize("fn,base,status,change",
                         [(f, base, s, c) for f, base, s, changes in REFUSED for c in changes],
                         ids=lambda v: v if isinstance(v, str) else
                         "_".join(f"{k}={x}" for k, x in v.items()) if isinstance(v, dict) and len(v) < 5 else "")
def test_refused_before_any_launch(L, fn, base, status, change):
    assert call(L, fn, base, **change) == status


def test_nothing_to_do_is_fine(L):
    assert call(L, "moe_linear", LINEAR, m=0, x=None, y=None, ws=None, ws_bytes=0) == OK
    assert call(L, "moe_gated_linear", GATED, m=0, x=None, h=None, ws=None, ws_bytes=0) == OK
    assert call(L, "moe_layer_norm", NORM, rows=0, x=None, y=None) == OK
    assert call(L, "moe_linear_backward", LINEAR_BACK, m=0, dy=None, x=None, z=None, dx=None, dw=None, dbias=None) == OK
    assert call(L, "moe_gated_linear_backward", GATED_BACK, m=0, dh=None, gu=None, x=None, dx=None, dw=None) == OK
    assert call(L, "moe_layer_norm_backward", NORM_BACK, rows=0, dy=None, x=None, dx=None, dweight=None, dbias=None) == OK
    # nothing wanted
    assert call(L, "moe_linear_backward", LINEAR_BACK, dx=None, dw=None, dbias=None, x=None, w=None, ws=None) == OK
    assert call(L, "moe_gated_linear_backward", GATED_BACK, dx=None, dw=None, x=None, w=None, ws=None) == OK
    assert call(L, "moe_layer_norm_backward", NORM_BACK, dx=None, dweight=None, dbias=None, ws=None) == OK


def test_workspaces(L):
    assert b.moe_linear_workspace(1, 7168, 2048) == 0 and b.moe_linear_workspace(16, 4096, 7168) == 0
    assert b.moe_linear_workspace(16384, 7168, 2048) == 0 and b.moe_linear_workspace(0, 8, 8) == 0
    assert b.moe_gated_linear_workspace(16384, 2048, 7168) == 0
    for fn in (b.moe_linear_workspace, b.moe_gated_linear_workspace, b.moe_gated_linear_backward_workspace):
        assert fn(0, 8, 8) >= 0
    assert b.moe_linear_backward_workspace(0, 8, 8, "none") >= 0 and b.moe_linear_backward_workspace(0, 8, 8, "gelu") >= 0
    for m, n, k in ((65, 8, 8200), (300, 200, 4096), (1000, 777, 1111)):
        assert b.moe_linear_workspace(m, n, k) % 256 == 0
    # dz of two bytes an element, rows padded to eight, and something for the sums
    assert b.moe_linear_backward_workspace(100, 9, 33, "silu") >= 100 * 16 * 2 + 9 * 4
    assert b.moe_linear_backward_workspace(100, 9, 33, "none") < b.moe_linear_backward_workspace(100, 9, 33, "silu")
    assert b.moe_gated_linear_backward_workspace(16384, 2048, 7168) >= 16384 * 4096 * 2
    assert b.moe_layer_norm_backward_workspace(0, 64) == 0
    assert b.moe_layer_norm_backward_workspace(1, 64) == 2 * 64 * 4
    for fn in ("moe_linear_workspace", "moe_gated_linear_workspace", "moe_gated_linear_backward_workspace"):
        for bad in ((-1, 8, 8), (8, 0, 8), (8, 8, 0)):
            with pytest.raises(moe.MoeError) as e:
                getattr(b, fn)(*bad)
            assert e.value.status == INVALID
        assert getattr(L, fn)(8, 8, 8, None) == INVALID
    with pytest.raises(moe.MoeError):
        b.moe_layer_norm_backward_workspace(-1, 8)
    assert L.moe_linear_backward_workspace(8, 8, 8, 7, ctypes.byref(ctypes.c_size_t())) == INVALID
    with pytest.raises(ValueError):
        b.moe_linear_backward_workspace(8, 8, 8, "swish")


def test_host_tensors_are_refused():
    x, w, v = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros((6, 8), dtype=torch.bfloat16), torch.zeros(4)
    for f in (lambda: moe.linear(x, w, ws=x), lambda: moe.gated_linear(x, w, ws=x), lambda: moe.layer_norm(x),
              lambda: moe.linear_backward(w[:4, :6], x, w, ws=x), lambda: moe.gated_linear_backward(w[:4, :3], x, w, x, ws=x),
              lambda: moe.layer_norm_backward(x, x, None, v, v, ws=x)):
        with pytest.raises(ValueError):
            f()
