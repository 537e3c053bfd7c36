"""Tensors that do not fit a call are refused by the binding before their
pointers reach the library, on stand-ins for device tensors."""
import pytest
import torch

import fake_device
import sparse_moe_gemm_amd as cm

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ENTRIES = ["forward", "forward_few"]


@pytest.fixture
def dev(monkeypatch):
    return fake_device.Device(monkeypatch)


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for e in ENTRIES:
        monkeypatch.setattr(cm, f"colibri_moe_{e}", lambda *a: seen.append(a) or cm.OK)
    return seen


def tensor(dev, shape, dtype, index=0, contiguous=True):
    t = fake_device.Tensor(shape, dtype, dev.current, index)
    t.is_contiguous = lambda: contiguous
    return t


@pytest.mark.parametrize("entry", ENTRIES)
def test_x_and_y_that_do_not_fit(dev, calls, entry):
    run = getattr(fake_device.layer(dev), entry)
    x = tensor(dev, (4, 64), BF16)
    with pytest.raises(TypeError):
        run(torch.zeros(4, 64, dtype=BF16))  # not on a GPU
    for bad in (tensor(dev, (4, 64), F32), tensor(dev, (4, 65), BF16), tensor(dev, (4, 1, 64), BF16),
                tensor(dev, (4, 64), BF16, index=1), tensor(dev, (4, 64), BF16, contiguous=False)):
        with pytest.raises(TypeError):
            run(bad)
    with pytest.raises(TypeError):
        run(x, torch.zeros(4, 64, dtype=BF16))
    for bad in (tensor(dev, (4, 64), F32), tensor(dev, (3, 64), BF16), tensor(dev, (4, 64), BF16, index=1),
                tensor(dev, (4, 64), BF16, contiguous=False)):
        with pytest.raises(TypeError):
            run(x, bad)
    assert not calls
    y = tensor(dev, (6, 64), BF16)  # rows behind the call's tokens are left alone
    assert run(x, y) is y and len(calls) == 1


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("name,dtype,size", [
    ("logits", F32, 32), ("topk_ids", I32, 8), ("topk_w", F32, 8), ("expert_counts", I32, 8),
    ("expert_offsets", I32, 9), ("perm", I32, 8), ("perm_slot", I32, 8), ("inv", I32, 8)])
def test_routing_buffers_that_do_not_fit(dev, calls, entry, name, dtype, size):
    run = getattr(fake_device.layer(dev), entry)
    x = tensor(dev, (4, 64), BF16)
    other = I32 if dtype is F32 else F32
    for bad in (tensor(dev, (size - 1,), dtype), tensor(dev, (size,), other), tensor(dev, (size,), dtype, index=1),
                tensor(dev, (size,), dtype, contiguous=False), torch.zeros(size, dtype=dtype)):
        with pytest.raises(TypeError, match=name):
            run(x, None, {name: bad})
    assert not calls
    run(x, None, {name: tensor(dev, (size,), dtype)})
    run(x, None, {"logits": None, "inv": None, "note": "not a routing output"})
    assert len(calls) == 2


def test_the_layers_own_buffers_fit(dev, calls):
    layer = fake_device.layer(dev)
    layer.forward_few(tensor(dev, (4, 64), BF16), None, layer.routing_buffers(4))
    layer.stream = fake_device.Stream(0x60)
    layer.forward_few(tensor(dev, (4, 64), BF16), None, {**layer.routing_buffers(4), "note": "not a routing output"})
    assert len(calls) == 2


def weights(dev, d=64, E=8, f=128, index=0):
    shapes = dict(w_router=(d, E), b_router=(E,), w_gate=(E, f, d), w_up=(E, f, d), w_down=(E, d, f))
    return {n: tensor(dev, v, F32 if n == "b_router" else BF16, index) for n, v in shapes.items()}


def test_weights_that_do_not_belong_together(dev, monkeypatch):
    made = []
    monkeypatch.setattr(cm, "colibri_moe_init", lambda *a: made.append(a) or (cm.OK, 7))
    monkeypatch.setattr(cm, "colibri_moe_free", lambda h: cm.OK)
    for name, shapes in dict(w_gate=[(7, 128, 64), (8, 128, 32)], w_up=[(8, 64, 64), (8, 64, 128), (7, 128, 64)],
                             w_down=[(8, 128, 64), (8, 64, 64)], b_router=[(7,), (16,)]).items():
        for shape in shapes:
            w = weights(dev)
            w[name] = tensor(dev, shape, w[name].dtype)
            with pytest.raises(ValueError):
                cm.MoELayer(**w, top_k=2, max_tokens=16)
    w = weights(dev)
    w["b_router"].is_contiguous = lambda: False
    with pytest.raises(ValueError):
        cm.MoELayer(**w, top_k=2, max_tokens=16)
    assert not made
    cm.MoELayer(**weights(dev), top_k=2, max_tokens=16)
    cm.MoELayer(**{**weights(dev), "b_router": None}, top_k=2, max_tokens=16)
    assert len(made) == 2


def test_layer_lives_on_its_weights_device(dev, monkeypatch):
    made = []
    monkeypatch.setattr(cm, "colibri_moe_init", lambda c, w, s: made.append((dev.index, s)) or (cm.OK, 7))
    monkeypatch.setattr(cm, "colibri_moe_free", lambda h: cm.OK)
    layer = cm.MoELayer(**weights(dev, index=1), top_k=2, max_tokens=16)
    assert made == [(1, 0x1000)] and dev.index == 0
    assert all(t.device.index == 1 for t in layer.routing_buffers(4).values())
    cm.MoELayer(**weights(dev, index=1), top_k=2, max_tokens=16, stream=fake_device.Stream(0x61, index=1))
    assert made[1:] == [(1, 0x61)]
    for name in ("w_gate", "w_up", "w_down", "b_router"):
        w = weights(dev, index=1)
        w[name] = weights(dev)[name]
        with pytest.raises(TypeError):
            cm.MoELayer(**w, top_k=2, max_tokens=16)
    with pytest.raises(ValueError):
        cm.MoELayer(**weights(dev, index=1), top_k=2, max_tokens=16, stream=fake_device.Stream(0x62))
    assert len(made) == 2


@pytest.mark.parametrize("entry", ENTRIES)
def test_a_refused_call_on_another_stream_leaves_its_tensors_alone(dev, calls, entry):
    layer = fake_device.layer(dev, stream=fake_device.Stream(0x63))
    x, ids = tensor(dev, (4, 64), BF16), tensor(dev, (4, 2), I32)
    with pytest.raises(TypeError, match="inv"):
        getattr(layer, entry)(x, None, {"topk_ids": ids, "inv": torch.zeros(8, dtype=I32)})
    assert not calls and not dev.made and not x.recorded and not ids.recorded
