"""Calls that run on another stream than the current one, on stand-ins for
device tensors: memory that the call writes comes from the pool of the stream
it is written on (memory of the current stream's pool may still be in use by
kernels queued there), and every stream that uses a tensor of another pool is
recorded on it."""
import pytest
import torch

import fake_device
import sparse_moe_gemm_amd as cm


@pytest.fixture
def dev(monkeypatch):
    return fake_device.Device(monkeypatch)


def tensor(dev, shape, dtype):
    return fake_device.Tensor(shape, dtype, dev.current)


def check_outputs(dev, outs, s):
    for t in outs:
        assert t.pool is s
        assert s is dev.current or dev.current in t.recorded


def test_quantize_mxfp4_outputs_belong_to_the_stream_that_writes_them(dev, monkeypatch):
    calls = []
    monkeypatch.setattr(cm, "colibri_moe_quantize_mxfp4", lambda *a: calls.append(a) or cm.OK)
    w = tensor(dev, (4, 64), torch.bfloat16)
    s = fake_device.Stream(0x51)
    codes, scales = cm.quantize_mxfp4(w, stream=s)
    assert calls[-1][-3:] == (codes.ptr, scales.ptr, 0x51)
    check_outputs(dev, (codes, scales), s)
    assert s in w.recorded
    codes, scales = cm.quantize_mxfp4(w)
    assert calls[-1][-1] == 0
    check_outputs(dev, (codes, scales), dev.current)


def test_dequantize_mxfp4_outputs_belong_to_the_stream_that_writes_them(dev, monkeypatch):
    calls = []
    monkeypatch.setattr(cm, "colibri_moe_dequantize_mxfp4", lambda *a: calls.append(a) or cm.OK)
    codes, scales = tensor(dev, (4, 32), torch.uint8), tensor(dev, (4, 2), torch.uint8)
    s = fake_device.Stream(0x52)
    out = cm.dequantize_mxfp4(codes, scales, stream=s)
    assert calls[-1][-2:] == (out.ptr, 0x52)
    check_outputs(dev, (out,), s)
    assert s in codes.recorded and s in scales.recorded
    out = cm.dequantize_mxfp4(codes, scales)
    check_outputs(dev, (out,), dev.current)


def test_a_stream_of_another_device_is_refused(dev, monkeypatch):
    for fn in ("colibri_moe_quantize_mxfp4", "colibri_moe_dequantize_mxfp4"):
        monkeypatch.setattr(cm, fn, lambda *a: pytest.fail("reached the library"))
    s = fake_device.Stream(0x53, index=1)
    with pytest.raises(ValueError):
        cm.quantize_mxfp4(tensor(dev, (4, 64), torch.bfloat16), stream=s)
    with pytest.raises(ValueError):
        cm.dequantize_mxfp4(tensor(dev, (4, 32), torch.uint8), tensor(dev, (4, 2), torch.uint8), stream=s)


def test_quantize_fp8_outputs_belong_to_the_stream_that_writes_them(dev, monkeypatch):
    calls = []
    monkeypatch.setattr(cm, "colibri_moe_quantize_fp8", lambda *a: calls.append(a) or cm.OK)
    w = tensor(dev, (4, 64), torch.bfloat16)
    s = fake_device.Stream(0x54)
    codes, scales = cm.quantize_fp8(w, stream=s)
    assert calls[-1][-3:] == (codes.ptr, scales.ptr, 0x54)
    check_outputs(dev, (codes, scales), s)
    assert s in w.recorded
    check_outputs(dev, cm.quantize_fp8(w), dev.current)
    assert calls[-1][-1] == 0
    with pytest.raises(ValueError):
        cm.quantize_fp8(w, stream=fake_device.Stream(0x55, index=1))
    assert len(calls) == 2


@pytest.mark.parametrize("entry", ["forward", "forward_few"])
def test_layer_outputs_belong_to_the_handles_stream(dev, monkeypatch, entry):
    calls = []

    def call(handle, x, T, y, r):
        calls.append(y)
        return cm.OK

    monkeypatch.setattr(cm, f"colibri_moe_{entry}", call)
    layer = fake_device.layer(dev, stream=fake_device.Stream(0x56))
    x = tensor(dev, (4, 64), torch.bfloat16)
    y = getattr(layer, entry)(x)
    assert calls == [y.ptr]
    check_outputs(dev, (y,), layer.stream)
    assert layer.stream in x.recorded
    # a given y and routing buffers stay where they are; their memory too waits for the stream
    mine, ids = tensor(dev, (4, 64), torch.bfloat16), tensor(dev, (4, 2), torch.int32)
    assert getattr(layer, entry)(x, mine, {"topk_ids": ids, "inv": None}) is mine
    assert layer.stream in mine.recorded and layer.stream in ids.recorded
    # on the handle's own stream nothing is recorded
    dev.current = layer.stream
    x = tensor(dev, (4, 64), torch.bfloat16)
    y = getattr(layer, entry)(x)
    assert y.pool is layer.stream and not y.recorded and not x.recorded
