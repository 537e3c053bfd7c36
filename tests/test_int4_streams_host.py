"""The packed weights of an Int4Linear that is used on another stream than it was made
on: their memory is recorded there, so that an Int4Linear that goes out of use does not
free it under a running product. On the CPU, with stand-in tensors."""
import pytest
import torch

import fake_device
import sparse_moe_gemm_amd as cm


@pytest.mark.parametrize("made_on", [None, 0x51])
def test_packed_is_recorded_where_it_is_used(monkeypatch, made_on):
    dev = fake_device.Device(monkeypatch)
    seen = []
    monkeypatch.setattr(cm, "colibri_moe_int4_pack", lambda *a: seen.append(a[-1]) or cm.OK)
    monkeypatch.setattr(cm, "colibri_moe_int4_linear", lambda *a: seen.append(a[-1]) or cm.OK)

    def tensor(shape, dtype):
        return fake_device.Tensor(shape, dtype, dev.current)

    home = dev.current if made_on is None else fake_device.Stream(made_on)
    lin = cm.Int4Linear(tensor((64, 128), torch.uint8), tensor((64, 2), torch.bfloat16),
                        stream=None if made_on is None else home)
    lin.packed.recorded.clear()  # by its allocation for another stream
    x = tensor((3, 256), torch.bfloat16)
    other, given = fake_device.Stream(0x61), fake_device.Stream(0x62)
    with torch.cuda.stream(home):
        lin.forward(x)
        assert not lin.packed.recorded
    with torch.cuda.stream(other):
        lin.forward(x)
        assert lin.packed.recorded == [other]
        lin.forward(x, stream=given)
        assert lin.packed.recorded == [other, given]
        lin.forward(x, stream=home)
        assert lin.packed.recorded == [other, given]
    assert seen == [home.cuda_stream, home.cuda_stream, 0x61, 0x62, home.cuda_stream]
