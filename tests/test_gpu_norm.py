"""rms_norm against its formula in 64 bits.

Errors of the kernel's fp32 before the last rounding, relative to y: v = x + r
by half a step (2^-24), which also moves the mean's root by at most that;
1 / sqrt by half a step, and two products: in all at most 5 * 2^-24, taken as
2^-21. Then one rounding: at most 2^-8 |y| for bf16, 2^-24 |y| for fp32, half a
step of the E4M3 grid for the codes (taken exactly); below the normal range of
the type an absolute half step."""
import numpy as np
import pytest

from moe_case import to_f64

pytestmark = pytest.mark.gpu

FP32 = 2.0 ** -21


def make(T, d, dtype, pad=0, seed=0, std=1.0, offset=0):
    import torch

    g = torch.Generator().manual_seed(seed + 1000 * T + d)
    wide = (torch.randn(T, d + pad + offset, generator=g) * std).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return wide.cuda()[:, offset:offset + d]


def formula(x, w, r, eps):
    v = to_f64(x) + (0 if r is None else to_f64(r))
    return v / np.sqrt((v * v).mean(axis=1, keepdims=True) + np.float64(np.float32(eps))) * to_f64(w)


def check(x, w, r=None, eps=1e-6, rows=None, **kw):
    """Runs rms_norm on x (rows: compare these alone) and checks every output."""
    import torch

    import sparse_moe_gemm_amd as cm

    xin = x.clone()  # outputs may be written over it
    rin = None if r is None else r.clone()
    got = cm.rms_norm(x, w, eps, residual=r, **kw)
    torch.cuda.synchronize()
    y = formula(xin, w, rin, eps)
    pick = slice(None) if rows is None else rows
    if got.y is not None:
        assert got.y.dtype == x.dtype
        half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
        off = np.abs(to_f64(got.y) - y)[pick] - ((half + FP32) * np.abs(y) + 2.0 ** -133)[pick]
        assert (off <= 0).all(), f"y off at {np.argwhere(off > 0)[:3].tolist()}"
    if r is not None:
        want = xin.float() + rin.float()
        assert torch.equal(got.residual, want.to(x.dtype))
    if got.codes is not None:
        scale = to_f64(got.scales)
        amax = np.abs(y).max(axis=1)
        m, e = np.frexp(scale)
        assert (m == 0.5).all()
        some = amax > 0
        assert (amax <= 448 * scale * (1 + FP32))[some].all()
        assert (amax * (1 + FP32) > 224 * scale)[some & (scale > 2.0 ** -126)].all()
        assert (scale[~some] == 1).all()
        u = y / scale[:, None]
        value = to_f64(got.codes.view(torch.float8_e4m3fn).float())
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(u), 2.0 ** -6))) - 3)
        off = np.abs(value - u)[pick] - (step / 2 + FP32 * np.abs(u) + 2.0 ** -149 / scale[:, None])[pick]
        assert (off <= 0).all(), f"codes off at {np.argwhere(off > 0)[:3].tolist()}"
    return got


def weight(d, dtype, seed=3):
    import torch

    return (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


WIDTHS = [1, 5, 7, 8, 9, 15, 31, 64, 500, 511, 512, 513, 520, 1024, 1031, 2048, 2049, 2080, 4095, 4096, 4100, 8192, 8200,
          11111, 16383, 16384, 16385, 20000]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(d, dtype):
    import torch

    for T, pad, offset in ((1, 0, 0), (2, 1, 0), (5, 8, 0), (6, 3, 1)):
        x, r = make(T, d, dtype, pad, offset=offset), make(T, d, dtype, pad + 1, seed=1, std=3.0)
        for w in (weight(d, x.dtype), weight(d, torch.float32)):
            check(x, w)
            check(x, w, r, quantize="fp8")
        check(x, w, quantize="fp8", with_y=False)
        check(x, w, r, with_y=False)


@pytest.mark.parametrize("T", [3, 4, 100, 1023, 20001])
@pytest.mark.parametrize("d", [40, 600, 2048])
def test_row_counts(T, d):
    x, r = make(T, d, "bf16"), make(T, d, "bf16", seed=1)
    check(x, weight(d, x.dtype), r, quantize="fp8")


@pytest.mark.parametrize("d", [96, 1500, 4096, 9000, 17000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(d, dtype):
    """y over x and the sum over the residual, with rows whose last values two
    lanes hold."""
    import torch

    for T in (1, 37):
        x, r = make(T, d + 3, dtype)[:, :d].contiguous(), make(T, d, dtype, pad=5, seed=1)
        w = weight(d, x.dtype)
        apart = check(x.clone(), w, r.clone(), quantize="fp8")
        y, rr = x, r
        got = check(x, w, r, quantize="fp8", y=y, residual_out=rr)
        assert got.y is y and got.residual is rr
        assert all(torch.equal(a, b) for a, b in zip(apart, got))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [8, 600, 3001, 17000])
def test_largest_smallest_and_zero_rows(d, dtype):
    x = make(8, d, dtype)
    for i, s in enumerate((1e38, 3e37, 1e19, 1e-10, 1e-20, 1e-30, 1e-38, 0.0)):
        x[i] = (x[i].float().clamp(-3, 3) * s).to(x.dtype)
    for eps in (1e-6, 1e-30, 1e-5):
        check(x, weight(d, x.dtype), eps=eps, quantize="fp8")


def test_infinities_and_nan_stay_in_their_rows():
    import torch

    import sparse_moe_gemm_amd as cm

    for d in (24, 700, 4096, 17001):
        x = make(5, d, "bf16")
        x[1, d // 2], x[3, d - 1], x[4, 0] = float("nan"), float("inf"), -float("inf")
        got = cm.rms_norm(x, weight(d, x.dtype), quantize="fp8")
        clean = cm.rms_norm(x[[0, 2]], weight(d, x.dtype), quantize="fp8")
        torch.cuda.synchronize()
        for a, b in zip(got, clean):
            assert a is None or torch.equal(a[[0, 2]], b)
        values = got.codes.view(torch.float8_e4m3fn).float()
        assert got.y[1].isnan().all() and values[1].isnan().all() and got.scales[1] == 1
        for i, c in ((3, d - 1), (4, 0)):
            rest = torch.arange(d, device="cuda") != c
            assert got.y[i, c].isnan() and values[i, c].isnan() and (got.y[i][rest] == 0).all()
            assert (values[i][rest] == 0).all() and got.scales[i] == 1
        # infinite weights: infinite y, NaN codes, the others under their own scale
        w = weight(d, torch.float32)
        w[d // 3] = float("inf")
        got = cm.rms_norm(x[:1], w, quantize="fp8")
        w[d // 3] = 0
        clean = cm.rms_norm(x[:1], w, quantize="fp8")
        rest = torch.arange(d, device="cuda") != d // 3
        assert got.y[0, d // 3].isinf() and got.codes[0, d // 3] & 127 == 127
        assert torch.equal(got.codes[0][rest], clean.codes[0][rest]) and torch.equal(got.scales, clean.scales)


def test_codes_are_quantize_fp8s_for_values_that_need_no_rounding():
    """Rows whose y is exact in bf16: the codes and scales of quantize_fp8."""
    import torch

    import sparse_moe_gemm_amd as cm

    d = 1024
    x = torch.zeros(64, d)
    g = torch.Generator().manual_seed(1)
    sign = torch.randint(0, 2, (64, d), generator=g) * 2.0 - 1
    x[:] = sign  # mean square 1: y = w * sign up to 1 / sqrt(1 + eps)
    w = (2.0 ** torch.randint(-9, 9, (d,), generator=g).float()) * (1 + torch.randint(0, 8, (d,), generator=g) / 8)
    got = cm.rms_norm(x.bfloat16().cuda(), w.cuda(), eps=2.0 ** -40, quantize="fp8")
    codes, scales = cm.quantize_fp8(got.y)
    assert torch.equal(got.y.float().cpu(), sign * w) and torch.equal(got.scales, scales)
    assert torch.equal(got.codes, codes)


def test_rows_past_32_bits():
    import torch

    stride = (1 << 31) + 40
    flat = torch.empty(2 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    for d in (96, 2100):
        x = torch.as_strided(flat, (3, d), (stride, 1))
        x.copy_(make(3, d, "bf16"))
        check(x, weight(d, x.dtype), quantize="fp8")
        check(x, weight(d, x.dtype), x, residual_out=x)


def test_memory_around_the_rows_is_left_alone():
    import torch

    import sparse_moe_gemm_amd as cm

    for d in (7, 30, 515, 2050, 4097, 16400):
        wide = torch.full((5, d + 6), 3.0, dtype=torch.bfloat16, device="cuda")
        before = wide.clone()
        flat = torch.full((5 * d + 16,), 5.0, dtype=torch.bfloat16, device="cuda")
        y = flat[:3 * d].view(3, d)
        x, r = make(3, d, "bf16"), make(3, d, "bf16", seed=1)
        cm.rms_norm(x, weight(d, x.dtype), residual=r, residual_out=wide[1:4, 2:2 + d], y=y)
        torch.cuda.synchronize()
        assert (flat[3 * d:] == 5).all() and torch.equal(y, cm.rms_norm(x, weight(d, x.dtype), residual=r).y)
        inside = torch.zeros_like(wide, dtype=torch.bool)
        inside[1:4, 2:2 + d] = True
        assert torch.equal(wide[~inside], before[~inside]) and torch.equal(wide[1:4, 2:2 + d], x + r)


def test_streams_graphs_and_empty_calls():
    import torch

    import sparse_moe_gemm_amd as cm

    x, r = make(200, 4096, "bf16"), make(200, 4096, "bf16", seed=1)
    w = weight(4096, x.dtype)
    want = cm.rms_norm(x, w, residual=r, quantize="fp8")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = cm.rms_norm(x, w, residual=r, quantize="fp8", stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    src = x.clone()
    with torch.cuda.graph(graph):
        out = cm.rms_norm(src, w, residual=r, quantize="fp8")
    for n in range(4):
        src.copy_(x if n % 2 == 0 else r)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = want if n % 2 == 0 else cm.rms_norm(r, w, residual=r, quantize="fp8")
        assert all(torch.equal(a, b) for a, b in zip(out, ref)), n
    got = cm.rms_norm(x[:0], w, residual=r[:0], quantize="fp8")
    assert got.y.shape == (0, 4096) and got.codes.shape == (0, 4096) and got.scales.shape == (0,)
