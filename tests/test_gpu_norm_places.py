"""rms_norm with y and residual_out in the place of x and residual, every way round: the
bits of a call whose buffers lie apart; and overlaps are refused."""
import pytest

from test_gpu_norm import make, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 37])
@pytest.mark.parametrize("d", [5, 96, 519, 1500, 4100, 9000, 17001])
def test_outputs_in_an_inputs_place(d, T, dtype):
    import torch

    import sparse_moe_gemm_amd as cm

    x0, r0 = make(T, d, dtype), make(T, d, dtype, seed=1)
    w = weight(d, x0.dtype)
    want = cm.rms_norm(x0, w, residual=r0, quantize="fp8")
    for y_at, sum_at in ((0, 1), (1, 0), (0, None), (1, None), (None, 0), (None, 1)):
        at = [x0.clone().contiguous(), r0.clone().contiguous()]
        got = cm.rms_norm(at[0], w, residual=at[1], quantize="fp8", y=None if y_at is None else at[y_at],
                          residual_out=None if sum_at is None else at[sum_at])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (y_at, sum_at)


def test_overlaps_are_refused():
    import torch

    import sparse_moe_gemm_amd as cm

    flat = torch.randn(40 * 64, device="cuda").bfloat16()
    x, near, r = flat[: 8 * 64].view(8, 64), flat[8: 8 + 8 * 64].view(8, 64), flat[20 * 64: 28 * 64].view(8, 64)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    before = flat.clone()
    for kw in (dict(y=near), dict(residual=r, residual_out=near), dict(residual=r, y=r, residual_out=r),
               dict(residual=near, y=x), dict(residual=r, y=flat[27 * 64: 35 * 64].view(8, 64))):
        with pytest.raises(cm.ColibriError) as e:
            cm.rms_norm(x, w, **kw)
        assert e.value.status == cm.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(flat, before)
