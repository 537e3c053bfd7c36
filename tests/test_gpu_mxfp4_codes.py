"""The 4-bit code of every fp32 of magnitude at most 6, both signs, under the
scale 1 (each block holds a 6 that fixes it)."""
import pytest

pytestmark = pytest.mark.gpu

SIX = 0x40C00000  # fp32 bits of 6


@pytest.mark.parametrize("sign", [0, 1], ids=["positive", "negative"])
def test_code_of_every_fp32(sign):
    import torch

    import sparse_moe_gemm_amd as cm

    rows = 1 << 20
    per = rows * 31
    x = torch.empty(rows, 32, device="cuda")
    x[:, 31] = 6.0
    for first in range(0, SIX + 1, per):
        bits = torch.arange(first, first + per, device="cuda", dtype=torch.int64).clamp_(max=SIX)
        a = bits.int().view(torch.float32).view(rows, 31)
        x[:, :31] = -a if sign else a
        codes, scales = cm.quantize_mxfp4(x)
        # borders between neighbouring codes; a tie goes to the even code
        want = torch.zeros(rows, 31, dtype=torch.uint8, device="cuda")
        for border, to_upper in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                                 (5.0, False)):
            want += (a >= border) if to_upper else (a > border)
        want += 8 * sign
        got = torch.stack((codes & 15, codes >> 4), dim=2).view(rows, 32)
        assert bool((scales == 127).all()) and bool((got[:, 31] == 7).all()), hex(first)
        same = got[:, :31] == want
        assert bool(same.all()), [hex(int(v)) for v in bits.view(rows, 31)[~same][:4]]
