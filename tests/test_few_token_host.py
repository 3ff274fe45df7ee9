"""The few-token calls without a GPU: the oracle's pins, the packers, and every refusal that the library and the
binding make before a launch."""
import ctypes

import numpy as np
import pytest
import torch

import combine_expert_histogram_amd as moe
from combine_expert_histogram_amd import binding as b
from few_token_helpers import FORMATS, FORMAT_IDS, random_weight
from oracle import bf16 as obf16
from oracle import few_token as oft
from oracle import mx


# ---------------------------------------------------------------- the oracle
def test_e2m1_values():
    want = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert oft.e2m1_decode(np.arange(16)).tolist() == want + [-v for v in want]


def test_route_topk_ties_masks_and_infinities():
    inf, nan = np.inf, np.nan
    x = np.array([[1.0, 3.0, 3.0, 2.0], [-inf, nan, -inf, -inf], [nan, 0.0, -0.0, -inf], [inf, 1.0, inf, 0.0]])
    ids, w = oft.route_topk(x, 3, True)
    assert ids.tolist() == [[1, 2, 3], [-1, -1, -1], [1, 2, -1], [0, 2, 1]]
    np.testing.assert_allclose(w[0], np.array([1, 1, np.exp(-1)]) / (2 + np.exp(-1)), rtol=1e-15)
    assert w[1].tolist() == [0, 0, 0] and w[2].tolist() == [0.5, 0.5, 0] and w[3].tolist() == [0.5, 0.5, 0]
    _, w = oft.route_topk(x[:1], 1, False, 2.0)
    np.testing.assert_allclose(w[0, 0], 2 / (2 + np.exp(-1) + np.exp(-2)), rtol=1e-15)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("with_zero", [False, True])
@pytest.mark.parametrize("lead", [(), (3,)])
def test_int4_packer_round_trip(group, with_zero, lead):
    rng = np.random.default_rng(group + with_zero)
    n, k = 12, 384
    q = rng.integers(0, 16, (*lead, n, k)).astype(np.uint8)
    scale = obf16.to_f32(obf16.from_f32(np.exp2(rng.uniform(-8, 2, (*lead, n, k // group))).astype(np.float32)))
    zero = rng.integers(0, 16, scale.shape).astype(np.uint8) if with_zero else None
    w = moe.int4_weight(torch.from_numpy(q), torch.from_numpy(scale),
                        None if zero is None else torch.from_numpy(zero))
    assert (w.n, w.k, w.group, w.experts) == (n, k, group, lead[0] if lead else 1)
    z = 8.0 if zero is None else zero.repeat(group, -1).astype(np.float64)
    want = ((q - z) * scale.astype(np.float64).repeat(group, -1)).reshape(-1, n, k)
    for e in range(w.experts):
        pick = lambda t: t.reshape(w.experts, *t.shape[-3:])[e].float().numpy()  # noqa: E731
        got = oft.dequant("int4", w.data.reshape(w.experts, n, -1)[e].numpy(), pick(w.scale),
                          None if zero is None else pick(w.zero), group)
        np.testing.assert_array_equal(got, want[e])


def test_e2m1_packer_round_trip():
    rng = np.random.default_rng(5)
    codes = rng.integers(0, 16, (2, 8, 256)).astype(np.uint8)
    e8m0 = rng.integers(100, 140, (2, 8, 8)).astype(np.uint8)
    w = moe.e2m1_weight(torch.from_numpy(codes), torch.from_numpy(e8m0))
    assert w.scale.shape == (2, 2, 8)
    for e in range(2):
        got = oft.dequant("e2m1_mx", w.data[e].numpy(), w.scale[e].numpy().view(np.uint32))
        want = oft.e2m1_decode(codes[e]) * np.exp2(e8m0[e].astype(np.float64) - 127).repeat(32, 1)
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("fmt,group,z", FORMATS, ids=FORMAT_IDS)
def test_layer_oracle_matches_a_scalar_loop(fmt, group, z):
    rng = np.random.default_rng(1)
    _, w1 = random_weight(rng, fmt, group, z, 256, 128, 2)
    _, w2 = random_weight(rng, fmt, group, z, 128, 128, 2)
    x = rng.standard_normal((2, 128))
    ids, tw = np.array([[5, 4], [9, -1]], np.int32), np.array([[0.25, 0.75], [1.0, 1.0]])
    out, _ = oft.layer(x, ids, tw, 4, w1, w2)
    assert not out[1].any()
    for c in (0, 77):
        total = 0.0
        for j, e in enumerate((1, 0)):
            for i in range(128):
                gate = sum(w1[e, i, h] * x[0, h] for h in range(128))
                up = sum(w1[e, 128 + i, h] * x[0, h] for h in range(128))
                total += tw[0, j] * w2[e, c, i] * gate / (1 + np.exp(-gate)) * up
        np.testing.assert_allclose(out[0, c], total, rtol=1e-9)


# ---------------------------------------------------------------- refusals of the C ABI (fake pointers, no launch)
P = ctypes.c_void_p
FAKE = 4096


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(b.LIB_PATH):
        from combine_expert_histogram_amd import build
        build.build()
    return b.lib()


def _w(fmt=2, group=0, data=FAKE, scale=FAKE, zero=None):
    return ctypes.byref(b.moe_weight(fmt, group, data, scale, zero))


def test_matvec_refusals(L):
    def call(m=2, n=128, k=256, x=FAKE, xs=256, w=None, y=FAKE, ys=128):
        return L.moe_matvec(m, n, k, x, xs, _w() if w is None else w, y, ys, None)
    assert call(m=0) == 0 and call(m=0, x=None, y=None) == 0
    for bad in (dict(m=-1), dict(n=0), dict(n=-4), dict(n=126), dict(k=0), dict(k=200), dict(k=-128), dict(x=None),
                dict(y=None), dict(x=FAKE + 8), dict(y=FAKE + 4), dict(xs=255), dict(xs=128), dict(xs=260),
                dict(xs=-256), dict(ys=124), dict(ys=130), dict(n=132, ys=132, w=_w(0)), dict(w=_w(7)), dict(w=_w(-1)),
                dict(w=_w(data=None)), dict(w=_w(scale=None)), dict(w=_w(data=FAKE + 1)), dict(w=_w(scale=FAKE + 4)),
                dict(w=_w(zero=FAKE)), dict(w=_w(3, 16)), dict(w=_w(3, 0)), dict(w=_w(3, 256)),
                dict(w=_w(3, 32, zero=FAKE + 2))):
        assert call(**bad) == -1, bad
    assert L.moe_matvec(2, 128, 256, FAKE, 256, None, FAKE, 128, None) == -1
    assert call(xs=1 << 24) == -3
    assert call(m=(1 << 20) + 1) == -3
    assert call(n=(1 << 27) + 4, ys=1 << 28) == -3
    assert L.moe_matvec(0, 128, 256, None, 256, _w(7), None, 128, None) == -1    # a bad weight, even with no rows


def _dims(**kw):
    args = dict(S=1, Ts=4, k=2, E=8, e0=0, L=8, H=256)
    args.update(kw)
    return b.Dims(**args)


def test_layer_refusals(L):
    def call(d=None, inter=128, x=FAKE, ids=FAKE, tw=FAKE, w1=None, w2=None, out=FAKE, ws=FAKE, nbytes=1 << 20):
        d = _dims() if d is None else d
        return L.moe_few_token_layer(ctypes.byref(d.c()), inter, x, ids, tw, w1 or _w(), w2 or _w(), out, ws, nbytes,
                                     None)
    assert call(d=_dims(Ts=0)) == 0 and call(d=_dims(Ts=0), x=None, ids=None, tw=None, out=None, ws=None) == 0
    for bad in (dict(d=_dims(Ts=-1)), dict(d=_dims(k=0)), dict(d=_dims(k=9)), dict(d=_dims(e0=4)), dict(d=_dims(L=0)),
                dict(d=_dims(H=200)), dict(d=_dims(H=0)), dict(inter=0), dict(inter=100), dict(inter=-128),
                dict(x=None), dict(ids=None), dict(tw=None), dict(out=None), dict(x=FAKE + 2), dict(out=FAKE + 2),
                dict(w1=_w(9)), dict(w2=_w(9)), dict(w1=_w(data=None)), dict(w2=_w(scale=None)),
                dict(w1=_w(3, 48)), dict(w2=_w(0, zero=FAKE))):
        assert call(**bad) == -1, bad
    for short in (dict(ws=None), dict(nbytes=4 * 2 * 128 * 2 - 1), dict(ws=FAKE + 8)):
        assert call(**short) == -2, short
    assert call(d=_dims(E=2048, L=2048)) == -3
    assert call(d=_dims(E=256, k=65)) == -3
    assert call(d=_dims(Ts=64, H=1 << 24)) == -3                  # 64 rows of 2^25 bytes
    assert call(inter=1 << 24, nbytes=1 << 40) == -3
    assert call(d=_dims(Ts=64, k=64, E=64, L=64), inter=1 << 18, nbytes=1 << 40) == -3
    assert L.moe_few_token_layer(None, 128, *[FAKE] * 3, _w(), _w(), FAKE, FAKE, 1 << 20, None) == -1
    assert L.moe_few_token_layer(ctypes.byref(_dims().c()), 128, *[FAKE] * 3, None, _w(), FAKE, FAKE, 1 << 20, None) == -1


def test_layer_widest_rows(L):
    """hidden is refused from 2^24 on for one token too, by the workspace query as well."""
    wide, need = _dims(Ts=1, H=1 << 24), ctypes.c_size_t()
    args = (128, *[FAKE] * 3, _w(), _w(), FAKE, FAKE, 1 << 20, None)
    assert L.moe_few_token_layer(ctypes.byref(wide.c()), *args) == -3
    assert L.moe_few_token_layer_workspace(ctypes.byref(wide.c()), 128, ctypes.byref(need)) == -3
    assert L.moe_few_token_layer_workspace(ctypes.byref(_dims(Ts=1, H=(1 << 24) - 128).c()), 128, ctypes.byref(need)) == 0


def test_layer_workspace(L):
    assert b.moe_few_token_layer_workspace(_dims(), 128) == 4 * 2 * 128 * 2
    assert b.moe_few_token_layer_workspace(_dims(Ts=1, k=1), 128) == 256
    big = b.moe_few_token_layer_workspace(_dims(S=8, Ts=2048, k=8), 2048)
    assert big == 64 * 8 * 2048 * 2                               # batches of 64 reuse it
    assert b.moe_few_token_layer_workspace(_dims(Ts=0), 128) == 0
    for inter in (0, 64, -128):
        with pytest.raises(b.MoeError):
            b.moe_few_token_layer_workspace(_dims(), inter)
    assert L.moe_few_token_layer_workspace(ctypes.byref(_dims().c()), 128, None) == -1


def test_route_topk_refusals(L):
    def call(d=None, x=FAKE, stride=8, ids=FAKE, w=FAKE):
        d = _dims() if d is None else d
        return L.moe_route_topk(ctypes.byref(d.c()), x, 0, stride, 1, 1.0, ids, w, None)
    assert call(d=_dims(Ts=0)) == 0 and call(d=_dims(Ts=0), x=None, ids=None, w=None) == 0
    for bad in (dict(x=None), dict(ids=None), dict(w=None), dict(stride=7), dict(stride=-8), dict(d=_dims(k=9)),
                dict(d=_dims(S=0))):
        assert call(**bad) == -1, bad
    assert call(d=_dims(E=1025, L=8), stride=1025) == -3
    assert call(d=_dims(E=1024, k=65), stride=1024) == -3
    assert call(d=_dims(Ts=(1 << 25) + 1)) == -3


# ---------------------------------------------------------------- refusals of the binding
def test_weight_checks():
    data, scale = torch.zeros(128 * 128, dtype=torch.uint8), torch.zeros(128, dtype=torch.int32)
    ok = moe.Weight("e4m3_mx", 128, 128, data, scale)
    assert ok.experts == 1 and ok.device.type == "cpu"
    for bad in (dict(fmt="fp8"), dict(n=126), dict(k=100), dict(k=0), dict(n=0), dict(experts=0), dict(experts=2),
                dict(data=data[:-1]), dict(data=data.view(torch.int8)), dict(scale=scale.float()),
                dict(zero=torch.zeros(128, dtype=torch.uint8)), dict(data=data.view(128, 128).t()),
                dict(fmt="e4m3", n=64), dict(fmt="int4", group=16), dict(scale=torch.zeros(129, dtype=torch.int32)[1:])):
        args = dict(fmt="e4m3_mx", n=128, k=128, data=data, scale=scale)
        args.update(bad)
        with pytest.raises(ValueError):
            moe.Weight(**args)


def test_packer_refusals():
    q, s = torch.zeros((8, 128), dtype=torch.uint8), torch.ones((8, 4))
    moe.int4_weight(q, s)
    for bad in ((q.int(), s), (q[:, :64], s), (q, s[:4]), (q, torch.ones((8, 3))), (q, torch.ones((8, 8))),
                (q + 16, s), (q, s, torch.full((8, 4), 16, dtype=torch.uint8)), (q, s, torch.zeros((8, 2))),
                (q, torch.ones((8, 0)))):
        with pytest.raises(ValueError):
            moe.int4_weight(*bad)
    e = torch.full((8, 4), 127, dtype=torch.uint8)
    for bad in ((q.int(), e), (q, e[:4]), (q, e.int()), (q + 16, e)):
        with pytest.raises(ValueError):
            moe.e2m1_weight(*bad)


def test_host_tensors_are_refused():
    d = moe.Dims(S=1, Ts=2, k=2, E=8, e0=0, L=1, H=128)
    with pytest.raises(ValueError, match="device tensor"):
        moe.route_topk(d, torch.zeros(2, 8))
    w = moe.Weight("e4m3_mx", 128, 128, torch.zeros(128 * 128, dtype=torch.uint8), torch.zeros(128, dtype=torch.int32))
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        moe.matvec(x, w)
    with pytest.raises(ValueError, match="device tensor"):
        moe.few_token_layer(d, 128, x, torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2)), w, w, ws=x)


def test_mx_packing_helper_agrees_with_the_oracle():
    codes = np.arange(2 * 3 * 4, dtype=np.uint8).reshape(2, 3, 4)
    w = b._blocks_first(torch.from_numpy(codes.transpose(1, 0, 2).reshape(3, 8).copy()), 4)
    assert w.view(torch.int32).squeeze(-1).numpy().view(np.uint32).tolist() == mx.pack_codes(codes)[..., 0].tolist()
