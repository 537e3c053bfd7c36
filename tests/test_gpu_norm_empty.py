"""Rows without values: rms_norm's outputs are empty, and the scale of such a row
is that of a row of zeros, 1."""
import pytest

pytestmark = pytest.mark.gpu


def test_scales_of_rows_without_values():
    import torch

    import sparse_moe_gemm_amd as cm

    side = torch.cuda.Stream()
    for dtype in (torch.bfloat16, torch.float32):
        x, w = torch.empty(1000, 0, dtype=dtype, device="cuda"), torch.empty(0, dtype=dtype, device="cuda")
        for stream in (None, side):
            torch.cuda.synchronize()
            junk = torch.full((1000,), 7.0, device="cuda")  # memory that the scales may get
            del junk
            got = cm.rms_norm(x, w, residual=x, quantize="fp8", stream=stream)
            torch.cuda.synchronize()
            assert got.y.shape == got.residual.shape == got.codes.shape == (1000, 0)
            assert got.scales.shape == (1000,) and (got.scales == 1).all()
