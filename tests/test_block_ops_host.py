"""Refusals of the operators around the layer (route, rms_norm), on the CPU: bad
arguments never reach the device, in the C ABI and in the binding. And the
plain routing that the GPU tests compare with, on hand-worked tokens."""
import math

import numpy as np
import pytest
import torch

import fake_device
import route_ref
import sparse_moe_gemm_amd as cm

FAKE = 0x100000  # never dereferenced: validation fails before any use
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture
def dev(monkeypatch):
    return fake_device.Device(monkeypatch)


def tensor(dev, shape, dtype, index=0, stride=None):
    t = fake_device.Tensor(shape, dtype, dev.current, index)
    if stride is not None:
        t.stride = lambda: stride
        t.is_contiguous = lambda: False
    return t


def rule(**kw):
    return cm.RoutingRule(**kw).c


# --- the C ABI -----------------------------------------------------------------------------------


def c_route(logits=FAKE, dtype=cm.F32, stride=64, T=4, E=64, k=4, r=None, bias=None, ids=FAKE, w=FAKE):
    return cm.colibri_moe_route(logits, dtype, stride, T, E, k, r or rule(), bias, ids, w)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), cm.ERR_INVALID_ARG), (dict(ids=None), cm.ERR_INVALID_ARG), (dict(w=None), cm.ERR_INVALID_ARG),
    (dict(dtype=2), cm.ERR_INVALID_ARG), (dict(T=-1), cm.ERR_INVALID_ARG), (dict(E=0), cm.ERR_INVALID_ARG),
    (dict(k=0), cm.ERR_INVALID_ARG), (dict(E=4, k=5), cm.ERR_INVALID_ARG), (dict(stride=63), cm.ERR_INVALID_ARG),
    (dict(stride=1 << 41), cm.ERR_INVALID_ARG), (dict(E=257, stride=300), cm.ERR_UNSUPPORTED),
    (dict(k=9), cm.ERR_UNSUPPORTED), (dict(logits=FAKE + 2), cm.ERR_ALIGNMENT), (dict(bias=FAKE + 2), cm.ERR_ALIGNMENT),
    (dict(logits=FAKE + 1, dtype=cm.BF16), cm.ERR_ALIGNMENT), (dict(ids=FAKE + 1), cm.ERR_ALIGNMENT),
    (dict(w=FAKE + 2), cm.ERR_ALIGNMENT), (dict(T=0, logits=None, ids=None, w=None), cm.OK),
])
def test_route_refusals(kw, status):
    assert c_route(**kw) == status


BAD_RULES = [dict(groups=5), dict(groups=0), dict(groups=128), dict(groups=8, top_groups=9), dict(groups=8, top_groups=0),
             dict(groups=32, top_groups=1), dict(scale=math.inf), dict(scale=math.nan)]


@pytest.mark.parametrize("bad", BAD_RULES, ids=str)
def test_rules_that_do_not_fit(bad):
    assert c_route(r=rule(**bad)) == cm.ERR_INVALID_ARG
    cfg = cm.Config(256, 128, 64, 4, 16, cm.BF16, 0)
    w = cm.Weights(FAKE, None, FAKE, FAKE, FAKE)
    assert cm.colibri_moe_init_rule(cfg, w, rule(**bad), None) == (cm.ERR_INVALID_ARG, None)


def test_rule_fields_and_nulls():
    for field, value in (("scoring", 2), ("group_score", -1), ("normalize", 2)):
        r = rule()
        setattr(r, field, value)
        assert c_route(r=r) == cm.ERR_INVALID_ARG
    assert cm.colibri_moe_route(FAKE, cm.F32, 64, 4, 64, 4, None, None, FAKE, FAKE) == cm.ERR_INVALID_ARG
    cfg = cm.Config(256, 128, 64, 4, 16, cm.BF16, 0)
    w = cm.Weights(FAKE, None, FAKE, FAKE, FAKE)
    assert cm.colibri_moe_init_rule(cfg, w, None, None)[0] == cm.ERR_INVALID_ARG
    assert cm.colibri_moe_init_rule(cfg, w, rule(), FAKE + 2)[0] == cm.ERR_ALIGNMENT
    with pytest.raises(ValueError):
        cm.RoutingRule(scoring="tanh")
    with pytest.raises(ValueError):
        cm.RoutingRule(group_score="mean")


def c_norm(**kw):
    a = dict(x=FAKE, x_stride=64, residual=None, residual_stride=0, weight=FAKE, dtype=cm.BF16, weight_dtype=cm.BF16,
             rows=4, cols=64, eps=1e-6, y=FAKE, residual_out=None, residual_out_stride=0, codes=None, scales=None)
    a.update(kw)
    return cm.colibri_moe_rms_norm(cm.Norm(*a.values()))


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), cm.ERR_INVALID_ARG), (dict(weight=None), cm.ERR_INVALID_ARG), (dict(y=None), cm.ERR_INVALID_ARG),
    (dict(codes=FAKE), cm.ERR_INVALID_ARG), (dict(dtype=2), cm.ERR_INVALID_ARG), (dict(weight_dtype=2), cm.ERR_INVALID_ARG),
    (dict(rows=-1), cm.ERR_INVALID_ARG), (dict(cols=0), cm.ERR_INVALID_ARG), (dict(cols=65), cm.ERR_INVALID_ARG),
    (dict(cols=(1 << 24) + 1, x_stride=1 << 25), cm.ERR_INVALID_ARG), (dict(eps=0.0), cm.ERR_INVALID_ARG),
    (dict(eps=-1.0), cm.ERR_INVALID_ARG), (dict(eps=math.nan), cm.ERR_INVALID_ARG), (dict(eps=math.inf), cm.ERR_INVALID_ARG),
    (dict(x_stride=1 << 41), cm.ERR_INVALID_ARG), (dict(residual=FAKE, residual_stride=63), cm.ERR_INVALID_ARG),
    (dict(residual=FAKE, residual_stride=64, residual_out=FAKE), cm.ERR_INVALID_ARG),
    (dict(x=FAKE + 1), cm.ERR_ALIGNMENT), (dict(y=FAKE + 1), cm.ERR_ALIGNMENT), (dict(weight=FAKE + 1), cm.ERR_ALIGNMENT),
    (dict(residual=FAKE + 1, residual_stride=64), cm.ERR_ALIGNMENT),
    (dict(dtype=cm.F32, x=FAKE + 2), cm.ERR_ALIGNMENT), (dict(weight_dtype=cm.F32, weight=FAKE + 2), cm.ERR_ALIGNMENT),
    (dict(codes=FAKE + 1, scales=FAKE + 2), cm.ERR_ALIGNMENT), (dict(rows=0, x=None, y=None), cm.OK),
])
def test_norm_refusals(kw, status):
    assert c_norm(**kw) == status
    assert cm.colibri_moe_rms_norm(None) == cm.ERR_INVALID_ARG


# --- the binding ---------------------------------------------------------------------------------


def test_route_arguments(dev, monkeypatch):
    calls = []
    monkeypatch.setattr(cm, "colibri_moe_route", lambda *a: calls.append(a) or cm.OK)
    x = tensor(dev, (4, 64), F32)
    for bad in (torch.zeros(4, 64), tensor(dev, (4, 64), I32), tensor(dev, (64,), F32)):
        with pytest.raises(TypeError):
            cm.route(bad, 4)
    for stride in ((64, 2), (63, 1), (0, 1)):
        with pytest.raises(ValueError):
            cm.route(tensor(dev, (4, 64), F32, stride=stride), 4)
    for bad in (tensor(dev, (63,), F32), tensor(dev, (64,), BF16), tensor(dev, (64,), F32, index=1), torch.zeros(64),
                tensor(dev, (64,), F32, stride=(2,))):
        with pytest.raises(TypeError):
            cm.route(x, 4, bias=bad)
    with pytest.raises(ValueError):
        cm.route(x, 4, stream=fake_device.Stream(0x70, index=1))
    assert not calls
    ids, w = cm.route(tensor(dev, (4, 64), BF16, stride=(80, 1)), 4)
    assert calls[-1][1:6] == (cm.BF16, 80, 4, 64, 4) and calls[-1][8:10] == (ids.ptr, w.ptr)
    assert (ids.shape, ids.dtype, w.shape, w.dtype) == ((4, 4), I32, (4, 4), F32)
    s = fake_device.Stream(0x71)
    b = tensor(dev, (64,), F32)
    ids, w = cm.route(x, 4, bias=b, stream=s)
    assert calls[-1][-1] == 0x71 and calls[-1][7] == b.ptr
    assert all(t.pool is s and dev.current in t.recorded for t in (ids, w)) and s in x.recorded and s in b.recorded


def test_norm_arguments(dev, monkeypatch):
    calls = []
    monkeypatch.setattr(cm, "colibri_moe_rms_norm", lambda n, s: calls.append((n, s)) or cm.OK)
    x, w, r = tensor(dev, (4, 64), BF16), tensor(dev, (64,), BF16), tensor(dev, (4, 64), BF16)
    with pytest.raises(TypeError):
        cm.rms_norm(torch.zeros(4, 64), w)
    for bad in (tensor(dev, (4, 64), I32), tensor(dev, (64,), BF16)):
        with pytest.raises(TypeError):
            cm.rms_norm(bad, w)
    for stride in ((64, 2), (63, 1), (0, 1)):
        with pytest.raises(ValueError):
            cm.rms_norm(tensor(dev, (4, 64), BF16, stride=stride), w)
        with pytest.raises(ValueError):
            cm.rms_norm(x, w, residual=tensor(dev, (4, 64), BF16, stride=stride))
        with pytest.raises(ValueError):
            cm.rms_norm(x, w, residual=r, residual_out=tensor(dev, (4, 64), BF16, stride=stride))
    for bad in (tensor(dev, (64,), torch.float16), tensor(dev, (64,), F32, index=1), tensor(dev, (1, 64), BF16)):
        with pytest.raises(TypeError):
            cm.rms_norm(x, bad)
    with pytest.raises(TypeError):
        cm.rms_norm(tensor(dev, (4, 64), F32), w)
    for bad in (tensor(dev, (63,), BF16), tensor(dev, (64,), BF16, stride=(2,))):
        with pytest.raises(ValueError):
            cm.rms_norm(x, bad)
    for bad in (tensor(dev, (4, 63), BF16), tensor(dev, (4, 64), F32), tensor(dev, (4, 64), BF16, index=1)):
        for kw in (dict(residual=bad), dict(residual=r, residual_out=bad), dict(y=bad)):
            with pytest.raises(TypeError):
                cm.rms_norm(x, w, **kw)
    with pytest.raises(TypeError):
        cm.rms_norm(x, w, y=tensor(dev, (4, 64), BF16, stride=(80, 1)))
    for kw in (dict(quantize="mxfp4"), dict(residual_out=r), dict(with_y=False), dict(with_y=False, y=r, quantize="fp8")):
        with pytest.raises(ValueError):
            cm.rms_norm(x, w, **kw)
    with pytest.raises(ValueError):
        cm.rms_norm(x, w, stream=fake_device.Stream(0x72, index=1))
    assert not calls
    got = cm.rms_norm(x, w)
    assert got.residual is None and got.codes is None and got.scales is None
    assert (calls[-1][0].x, calls[-1][0].y, calls[-1][0].residual) == (x.ptr, got.y.ptr, None)
    s = fake_device.Stream(0x73)
    got = cm.rms_norm(x, w, residual=r, quantize="fp8", stream=s)
    n = calls[-1][0]
    assert calls[-1][1] == 0x73
    assert [n.y, n.residual_out, n.codes, n.scales] == [t.ptr for t in got]
    assert all(t.pool is s and dev.current in t.recorded for t in got)
    assert all(s in t.recorded for t in (x, w, r))
    assert (got.codes.dtype, got.scales.shape) == (U8, (4,))


def test_layer_with_a_rule_reaches_the_library(dev, monkeypatch):
    made = []
    monkeypatch.setattr(cm, "colibri_moe_init", lambda *a: made.append(("plain", a)) or (cm.OK, 7))
    monkeypatch.setattr(cm, "colibri_moe_init_rule", lambda *a: made.append(("rule", a)) or (cm.OK, 7))
    monkeypatch.setattr(cm, "colibri_moe_free", lambda h: cm.OK)
    shapes = dict(w_router=(64, 8), w_gate=(8, 128, 64), w_up=(8, 128, 64), w_down=(8, 64, 128))
    w = {n: tensor(dev, v, BF16) for n, v in shapes.items()}
    args = dict(b_router=None, top_k=2, max_tokens=16)
    r, b = cm.RoutingRule(scoring="sigmoid"), tensor(dev, (8,), F32)
    cm.MoELayer(**w, **args, rule=r, select_bias=b)
    assert made[-1][0] == "rule" and made[-1][1][2:4] == (r.c, b.ptr)
    cm.MoELayer(**w, **args, rule=r)
    assert made[-1][0] == "rule" and made[-1][1][3] is None
    with pytest.raises(ValueError):
        cm.MoELayer(**w, **args, select_bias=b)
    for bad in (tensor(dev, (7,), F32), tensor(dev, (8,), BF16), tensor(dev, (8,), F32, index=1)):
        with pytest.raises(TypeError):
            cm.MoELayer(**w, **args, rule=r, select_bias=bad)
    assert len(made) == 2


# --- the plain routing ----------------------------------------------------------------------------


def test_plain_routing_on_hand_worked_tokens():
    ln2 = math.log(2.0)
    ids, w, _, _ = route_ref.route([[0.0, ln2, 2 * ln2, -np.inf]], 2)  # 1 : 2 : 4
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[2 / 3, 1 / 3]])
    ids, w, _, _ = route_ref.route([[0.0, ln2, 2 * ln2, -np.inf]], 2, normalize=False, scale=7.0)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[4, 2]])
    ids, w, _, _ = route_ref.route([[0.0, ln2, 0.0, ln2]], 3, "sigmoid")  # 1/2, 2/3
    assert ids.tolist() == [[1, 3, 0]] and np.allclose(w, np.array([[4, 4, 3]]) / 11)
    # the bias decides the choice, not the weight
    ids, w, _, _ = route_ref.route([[0.0, ln2, 0.0, ln2]], 2, "sigmoid", bias=[0.3, 0.0, 0.0, 0.0], normalize=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[1 / 2, 2 / 3]])
    # groups (0,1) and (2,3): the best expert is in the second, the better pair in the first
    l = [[2.0, 2.0, 3.0, -3.0]]
    assert route_ref.route(l, 2, "sigmoid", 2, 1, "max")[0].tolist() == [[2, 3]]
    assert route_ref.route(l, 2, "sigmoid", 2, 1, "top2")[0].tolist() == [[0, 1]]
    # an expert that is out adds nothing to its group and comes last
    l = [[0.5, -np.inf, -1.0, np.nan]]
    ids, w, _, _ = route_ref.route(l, 2, "sigmoid", 2, 1, "top2")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[1, 0]]
    ids, w, _, _ = route_ref.route([[-np.inf] * 4], 3)
    assert ids.tolist() == [[0, 1, 2]] and w.tolist() == [[0, 0, 0]]


# --- 4-bit integer groups -------------------------------------------------------------------------


def c_quant(w=FAKE, dtype=cm.BF16, rows=4, cols=256, stride=256, group=128, codes=FAKE, scales=FAKE, zeros=FAKE):
    return cm.colibri_moe_quantize_int4(w, dtype, rows, cols, stride, group, codes, scales, zeros)


def c_dequant(codes=FAKE, scales=FAKE, sd=cm.BF16, zeros=FAKE, rows=4, cols=256, group=128, dtype=cm.BF16, out=FAKE):
    return cm.colibri_moe_dequantize_int4(codes, scales, sd, zeros, rows, cols, group, dtype, out)


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), cm.ERR_INVALID_ARG), (dict(codes=None), cm.ERR_INVALID_ARG), (dict(scales=None), cm.ERR_INVALID_ARG),
    (dict(dtype=cm.F16), cm.ERR_INVALID_ARG), (dict(rows=0), cm.ERR_INVALID_ARG), (dict(cols=0), cm.ERR_INVALID_ARG),
    (dict(cols=192, stride=192), cm.ERR_INVALID_ARG), (dict(stride=255), cm.ERR_INVALID_ARG),
    (dict(group=0), cm.ERR_INVALID_ARG), (dict(group=16), cm.ERR_INVALID_ARG), (dict(group=96), cm.ERR_INVALID_ARG),
    (dict(group=512), cm.ERR_INVALID_ARG), (dict(group=-128), cm.ERR_INVALID_ARG),
    (dict(rows=(1 << 40) // 256 + 1), cm.ERR_INVALID_ARG), (dict(stride=1 << 41), cm.ERR_INVALID_ARG),
    (dict(w=FAKE + 1), cm.ERR_ALIGNMENT), (dict(w=FAKE + 2, dtype=cm.F32), cm.ERR_ALIGNMENT),
    (dict(codes=FAKE + 2), cm.ERR_ALIGNMENT), (dict(scales=FAKE + 1), cm.ERR_ALIGNMENT),
])
def test_quantize_int4_refusals(kw, status):
    assert c_quant(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), cm.ERR_INVALID_ARG), (dict(scales=None), cm.ERR_INVALID_ARG), (dict(out=None), cm.ERR_INVALID_ARG),
    (dict(sd=cm.F32), cm.ERR_INVALID_ARG), (dict(dtype=cm.F16), cm.ERR_INVALID_ARG), (dict(rows=0), cm.ERR_INVALID_ARG),
    (dict(group=48), cm.ERR_INVALID_ARG), (dict(cols=384, group=256), cm.ERR_INVALID_ARG),
    (dict(codes=FAKE + 2), cm.ERR_ALIGNMENT), (dict(scales=FAKE + 1), cm.ERR_ALIGNMENT), (dict(out=FAKE + 8), cm.ERR_ALIGNMENT),
])
def test_dequantize_int4_refusals(kw, status):
    assert c_dequant(**kw) == status


def matrix(**kw):
    a = dict(n_experts=4, rows=64, cols=256, group=128, scale_dtype=cm.BF16, swiglu=0)
    a.update(kw)
    return cm.Int4(*a.values())


BAD_MATRICES = [dict(n_experts=0), dict(n_experts=257), dict(rows=0), dict(rows=(1 << 24) + 1), dict(cols=0),
                dict(cols=320), dict(cols=1 << 21), dict(group=16), dict(group=192), dict(scale_dtype=cm.F32),
                dict(swiglu=2), dict(swiglu=1, rows=63), dict(n_experts=256, rows=1 << 24, cols=512)]


def c_linear(m=None, packed=FAKE, x=FAKE, T=4, k=2, per_slot=0, ids=FAKE, weights=None, y=FAKE, dtype=cm.BF16):
    return cm.colibri_moe_int4_linear(m or matrix(), packed, x, T, k, per_slot, ids, weights, y, dtype)


@pytest.mark.parametrize("bad", BAD_MATRICES, ids=str)
def test_matrices_that_are_not_supported(bad):
    m = matrix(**bad)
    assert cm.colibri_moe_int4_bytes(m) == -1
    assert cm.colibri_moe_int4_pack(m, FAKE, FAKE, None, FAKE) == cm.ERR_INVALID_ARG
    assert c_linear(m) == cm.ERR_INVALID_ARG


def test_pack_refusals_and_sizes():
    m = matrix()
    for args in ((None, FAKE, None, FAKE), (FAKE, None, None, FAKE), (FAKE, FAKE, None, None)):
        assert cm.colibri_moe_int4_pack(m, *args) == cm.ERR_INVALID_ARG
    assert cm.colibri_moe_int4_pack(None, FAKE, FAKE, None, FAKE) == cm.ERR_INVALID_ARG
    assert cm.colibri_moe_int4_bytes(None) == -1
    assert cm.colibri_moe_int4_pack(m, FAKE, FAKE + 1, None, FAKE) == cm.ERR_ALIGNMENT
    assert cm.colibri_moe_int4_pack(m, FAKE, FAKE, None, FAKE + 8) == cm.ERR_ALIGNMENT
    # whole tiles: half a byte per code, four bytes per group
    assert cm.colibri_moe_int4_bytes(m) == 4 * 64 * (256 // 2 + 4 * 2)


@pytest.mark.parametrize("kw,status", [
    (dict(packed=None), cm.ERR_INVALID_ARG), (dict(x=None), cm.ERR_INVALID_ARG), (dict(y=None), cm.ERR_INVALID_ARG),
    (dict(T=-1), cm.ERR_INVALID_ARG), (dict(k=0), cm.ERR_INVALID_ARG), (dict(per_slot=2), cm.ERR_INVALID_ARG),
    (dict(dtype=cm.F16), cm.ERR_INVALID_ARG), (dict(ids=None), cm.ERR_INVALID_ARG),
    (dict(m=matrix(n_experts=1), ids=None), cm.ERR_INVALID_ARG),
    (dict(m=matrix(n_experts=1), ids=None, k=1, weights=FAKE), cm.ERR_INVALID_ARG),
    (dict(m=matrix(swiglu=1), weights=FAKE), cm.ERR_INVALID_ARG), (dict(k=9), cm.ERR_UNSUPPORTED),
    (dict(T=65), cm.ERR_TOO_LARGE), (dict(T=1 << 30, k=8), cm.ERR_TOO_LARGE), (dict(packed=FAKE + 8), cm.ERR_ALIGNMENT),
    (dict(x=FAKE + 8), cm.ERR_ALIGNMENT), (dict(ids=FAKE + 2), cm.ERR_ALIGNMENT), (dict(weights=FAKE + 2), cm.ERR_ALIGNMENT),
    (dict(y=FAKE + 1), cm.ERR_ALIGNMENT), (dict(y=FAKE + 2, dtype=cm.F32), cm.ERR_ALIGNMENT),
    (dict(T=0, packed=None, x=None, y=None), cm.OK),
])
def test_int4_linear_refusals(kw, status):
    assert c_linear(**kw) == status
    assert cm.colibri_moe_int4_linear(None, FAKE, FAKE, 4, 2, 0, FAKE, None, FAKE, cm.BF16) == cm.ERR_INVALID_ARG


def test_int4_linear_refuses_y_over_x():
    """x [4][256] bf16 takes 2048 bytes, y [4][2][64] bf16 1024, fp32 2048."""
    for y in (FAKE, FAKE + 2032, FAKE - 1008):
        assert c_linear(x=FAKE, y=y) == cm.ERR_INVALID_ARG
    assert c_linear(x=FAKE, y=FAKE - 2032, dtype=cm.F32) == cm.ERR_INVALID_ARG
    assert c_linear(x=FAKE, y=FAKE + 4080, per_slot=1) == cm.ERR_INVALID_ARG


def test_int4_codec_arguments(dev, monkeypatch):
    calls = []
    for fn in ("colibri_moe_quantize_int4", "colibri_moe_dequantize_int4"):
        monkeypatch.setattr(cm, fn, lambda *a: calls.append(a) or cm.OK)
    for bad in (torch.zeros(4, 256, dtype=BF16), tensor(dev, (4, 256), torch.float16), tensor(dev, (256,), BF16)):
        with pytest.raises(TypeError):
            cm.quantize_int4(bad)
    for bad, group in ((tensor(dev, (4, 256), BF16, stride=(255, 1)), 128), (tensor(dev, (4, 256), BF16, stride=(512, 2)), 128),
                       (tensor(dev, (2, 4, 256), BF16, stride=(2048, 256, 1)), 128), (tensor(dev, (4, 256), BF16), 96),
                       (tensor(dev, (4, 192), BF16), 128), (tensor(dev, (4, 256), BF16), 0)):
        with pytest.raises(ValueError):
            cm.quantize_int4(bad, group)
    s = fake_device.Stream(0x74)
    with pytest.raises(ValueError):
        cm.quantize_int4(tensor(dev, (4, 256), BF16), stream=fake_device.Stream(0x75, index=1))
    assert not calls
    w = tensor(dev, (2, 4, 256), F32)
    codes, scales, zeros = cm.quantize_int4(w, 64, stream=s)
    assert calls[-1] == (w.ptr, cm.F32, 8, 256, 256, 64, codes.ptr, scales.ptr, zeros.ptr, 0x74)
    assert (codes.shape, scales.shape, zeros.shape) == ((2, 4, 128), (2, 4, 4), (2, 4, 4))
    assert all(t.pool is s and dev.current in t.recorded for t in (codes, scales, zeros)) and s in w.recorded
    assert cm.quantize_int4(w, symmetric=True)[2] is None and calls[-1][8] is None
    good = dict(codes=tensor(dev, (4, 128), U8), scales=tensor(dev, (4, 2), BF16), zeros=tensor(dev, (4, 2), U8))
    n = len(calls)
    for name, bad in (("codes", tensor(dev, (4, 128), I32)), ("codes", tensor(dev, (128,), U8)),
                      ("codes", tensor(dev, (4, 128), U8, stride=(256, 1))), ("scales", tensor(dev, (4, 2), F32)),
                      ("scales", tensor(dev, (4, 2), BF16, index=1)), ("zeros", tensor(dev, (4, 2), I32)),
                      ("zeros", tensor(dev, (4, 2), U8, index=1))):
        for fn in (cm.dequantize_int4, cm.Int4Linear):
            with pytest.raises(TypeError):
                fn(**{**good, name: bad})
    for name, bad in (("codes", tensor(dev, (5, 128), U8)), ("scales", tensor(dev, (4, 3), BF16)),
                      ("scales", tensor(dev, (4, 0), BF16)), ("zeros", tensor(dev, (4, 1), U8))):
        for fn in (cm.dequantize_int4, cm.Int4Linear):
            with pytest.raises(ValueError):
                fn(**{**good, name: bad})
    with pytest.raises(TypeError):
        cm.dequantize_int4(**good, dtype=torch.float16)
    assert len(calls) == n
    out = cm.dequantize_int4(**good, stream=s)
    assert calls[-1][-2:] == (out.ptr, 0x74) and out.pool is s and all(s in t.recorded for t in good.values())


def test_int4_linear_arguments(dev, monkeypatch):
    calls = []
    monkeypatch.setattr(cm, "colibri_moe_int4_pack", lambda *a: cm.OK)
    monkeypatch.setattr(cm, "colibri_moe_int4_linear", lambda *a: calls.append(a) or cm.OK)

    def linear(E=4, N=64, K=256, **kw):
        lead = (N,) if E is None else (E, N)
        return cm.Int4Linear(tensor(dev, (*lead, K // 2), U8), tensor(dev, (*lead, K // 128), BF16), **kw)

    with pytest.raises(ValueError):
        linear(N=63, swiglu=True)
    lin, dense = linear(), linear(None)
    x, ids, w = tensor(dev, (5, 256), BF16), tensor(dev, (5, 2), I32), tensor(dev, (5, 2), F32)
    for bad in (tensor(dev, (5, 256), F32), tensor(dev, (5, 255), BF16), tensor(dev, (256,), BF16),
                tensor(dev, (5, 256), BF16, index=1), tensor(dev, (5, 256), BF16, stride=(512, 1))):
        with pytest.raises(TypeError):
            lin.forward(bad, ids)
    for bad in (tensor(dev, (5, 2), torch.int64), tensor(dev, (10,), I32), tensor(dev, (5, 2), I32, index=1),
                tensor(dev, (5, 2), I32, stride=(4, 1))):
        with pytest.raises(TypeError):
            lin.forward(x, bad)
    for bad in (tensor(dev, (5, 2), BF16), tensor(dev, (5, 3), F32), tensor(dev, (5, 2), F32, index=1)):
        with pytest.raises(TypeError):
            lin.forward(x, ids, bad)
    with pytest.raises(ValueError):
        lin.forward(x)
    with pytest.raises(ValueError):
        lin.forward(x, tensor(dev, (4, 2), I32))
    with pytest.raises(ValueError):
        lin.forward(tensor(dev, (5, 3, 256), BF16), ids)
    with pytest.raises(ValueError):
        dense.forward(tensor(dev, (5, 1, 256), BF16))
    with pytest.raises(ValueError):
        dense.forward(x, weights=w)
    with pytest.raises(ValueError):
        linear(swiglu=True).forward(x, ids, w)
    with pytest.raises(TypeError):
        lin.forward(x, ids, dtype=torch.float16)
    for bad in (tensor(dev, (5, 2, 64), F32), tensor(dev, (5, 64), BF16), tensor(dev, (5, 2, 64), BF16, index=1),
                tensor(dev, (5, 2, 64), BF16, stride=(256, 64, 1))):
        with pytest.raises(TypeError):
            lin.forward(x, ids, y=bad)
    with pytest.raises(cm.ColibriError):
        lin.forward(tensor(dev, (65, 256), BF16), tensor(dev, (65, 2), I32))
    with pytest.raises(ValueError):
        lin.forward(x, ids, stream=fake_device.Stream(0x76, index=1))
    assert not calls
    y = lin.forward(x, ids)
    assert y.shape == (5, 2, 64) and calls[-1][2:6] == (x.ptr, 5, 2, 0)
    assert lin.forward(x, ids, w, dtype=F32).shape == (5, 64)
    assert linear(swiglu=True).forward(tensor(dev, (5, 2, 256), BF16), ids).shape == (5, 2, 32) and calls[-1][5] == 1
    assert dense.forward(x).shape == (5, 64)
    s = fake_device.Stream(0x77)
    y = lin.forward(x, ids, w, stream=s)
    assert calls[-1][-1] == 0x77 and y.pool is s and dev.current in y.recorded
    assert all(s in t.recorded for t in (x, ids, w, lin.packed))


def test_plain_int4_on_hand_worked_groups():
    import int4_ref

    w = np.zeros((2, 32))
    w[0, :3] = [-1.0, 2.0, 0.5]       # lo -1, hi 2: s = 0.2 as bf16, z = 5
    w[1, :2] = [7.0, -3.5]
    q, s, z, _ = int4_ref.quantize(w, 32, False)
    assert s[0, 0] == int4_ref.to_bf16(0.2) == 0.2001953125 and z[0, 0] == 5
    assert q[0, :4].tolist() == [0, 15, 7, 5]  # 2 / s = 9.99: 10 steps; 0.5 / s = 2.5 - : 2
    q, s, z, _ = int4_ref.quantize(w, 32, True)
    assert s[1, 0] == 1 and q[1, :3].tolist() == [15, 4, 8]  # -3.5: a tie, to -4
    assert int4_ref.values(q, s, None)[1, :3].tolist() == [7, -4, 0]
    assert (int4_ref.unpack(int4_ref.pack(q)) == q).all()
    y, _ = int4_ref.product64(np.eye(32)[:2], q, s, None)
    assert y[:, 1].tolist() == [7, -4]
