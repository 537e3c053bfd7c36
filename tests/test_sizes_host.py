"""Sizes past 32 bits that the library's arguments don't hold: refused, instead of
being cut to another size that the library would take. On the CPU; tensors are
stand-ins."""
import pytest
import torch

import fake_device
import sparse_moe_gemm_amd as cm

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
WRAP = 1 << 32


@pytest.fixture
def dev(monkeypatch):
    for fn in [n for n in cm.EXPORTS if n not in ("colibri_moe_status_string", "colibri_moe_int4_bytes")]:
        monkeypatch.setattr(cm, fn, lambda *a, n=fn: pytest.fail(f"{n} was called"), raising=False)
    return fake_device.Device(monkeypatch)


def tensor(dev, shape, dtype):
    return fake_device.Tensor(shape, dtype, dev.current)


def refused(fn, *args, **kw):
    with pytest.raises(cm.ColibriError) as e:
        fn(*args, **kw)
    assert e.value.status == cm.ERR_INVALID_ARG


@pytest.mark.parametrize("T,E,k", [(WRAP, 4, 2), (WRAP + 5, 4, 2), (1 << 31, 4, 2), (3, WRAP + 4, 2), (3, 4, WRAP + 2)])
def test_route(dev, T, E, k):
    refused(cm.route, tensor(dev, (T, E), BF16), k)
    assert not dev.made


@pytest.mark.parametrize("d", [WRAP, WRAP + 8, 1 << 31])
def test_rms_norm(dev, d):
    refused(cm.rms_norm, tensor(dev, (1, d), BF16), tensor(dev, (d,), BF16))
    assert not dev.made


@pytest.mark.parametrize("E,N,K,group", [(WRAP + 1, 2, 32, 32), (1, WRAP + 2, 32, 32), (1, 2, WRAP + 32, 32),
                                         (1, 2, WRAP + 128, WRAP + 128), (1, 1 << 31, 32, 32)])
def test_int4_linear(dev, E, N, K, group):
    with pytest.raises(ValueError):
        cm.Int4Linear(tensor(dev, (E, N, K // 2), U8), tensor(dev, (E, N, K // group), BF16))
    assert not dev.made


@pytest.mark.parametrize("kw", [dict(groups=WRAP + 1), dict(groups=1 - WRAP), dict(groups=2, top_groups=WRAP + 1)])
def test_rules(kw):
    with pytest.raises(ValueError):
        cm.RoutingRule(**kw)


@pytest.mark.parametrize("kw", [dict(top_k=WRAP + 2), dict(max_tokens=WRAP + 16)])
def test_layer(dev, kw):
    shapes = dict(w_router=(128, 8), w_gate=(8, 128, 128), w_up=(8, 128, 128), w_down=(8, 128, 128))
    refused(cm.MoELayer, **{n: tensor(dev, v, BF16) for n, v in shapes.items()}, b_router=None,
            **{**dict(top_k=2, max_tokens=16), **kw})


def test_the_largest_sizes_reach_the_library(dev, monkeypatch):
    seen = []
    monkeypatch.setattr(cm, "colibri_moe_route", lambda *a: seen.append(a[3]) or cm.OK)
    monkeypatch.setattr(cm, "colibri_moe_rms_norm", lambda n, s: seen.append(n.cols) or cm.OK)
    cm.route(tensor(dev, ((1 << 31) - 1, 4), BF16), 2)
    cm.rms_norm(tensor(dev, (1, 1 << 24), BF16), tensor(dev, (1 << 24,), BF16))
    assert seen == [(1 << 31) - 1, 1 << 24]
