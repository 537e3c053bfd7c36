"""4-bit integer groups where a rounding too many would show (int4_cases.py): exact
results under scales of whole mantissas and of both types, normal values within an
rms bound, values read back from fp16 scales, and the largest sums in LDS."""
import numpy as np
import pytest

import int4_cases
import int4_ref
from moe_case import to_f64
from test_gpu_int4 import bf16, exact_equal, integers, ints, some_ids

pytestmark = pytest.mark.gpu


def weights(rng, E, N, K, group, kind, zeros, ordinary=False):
    import torch

    q = rng.integers(0, 16, (E, N, K)).astype(np.uint8)
    s = int4_cases.whole_scales(rng, (E, N, K // group), kind, ordinary)
    z = rng.integers(0, 16, s.shape).astype(np.uint8) if zeros else None
    sd = torch.from_numpy(s).to(torch.float16 if kind == "f16" else torch.bfloat16).cuda()
    assert np.array_equal(to_f64(sd.float()), s)
    return q, s, z, (torch.from_numpy(int4_ref.pack(q)).cuda(), sd, None if z is None else torch.from_numpy(z).cuda())


@pytest.mark.parametrize("kind,zeros", [("bf16", True), ("f16", True), ("f16", False)])
@pytest.mark.parametrize("T,k,E,N,K,group", int4_cases.EXACT)
def test_scales_of_whole_mantissas(T, k, E, N, K, group, kind, zeros):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(T + N + K)
    q, s, z, w = weights(rng, E, N, K, group, kind, zeros)
    ids = some_ids(rng, T, k, E, "mixed")
    p = int4_cases.halves(rng, (T, k))
    i, pd = torch.from_numpy(ids).cuda(), torch.from_numpy(p).float().cuda()
    lin = cm.Int4Linear(*w)
    for x in (int4_cases.sparse(rng, (T, K)), int4_cases.sparse(rng, (T, k, K))):
        y, _ = int4_ref.assigned(x, ids, q, s, z)
        exact_equal(lin.forward(bf16(x), i, dtype=torch.float32), y)
        exact_equal(lin.forward(bf16(x), i), y)
        exact_equal(lin.forward(bf16(x), i, pd, dtype=torch.float32), (y * p[:, :, None]).sum(axis=1))
    if E == 1:
        x = int4_cases.sparse(rng, (T, K))
        dense = cm.Int4Linear(*(None if t is None else t[0] for t in w))
        exact_equal(dense.forward(bf16(x), dtype=torch.float32), x @ int4_ref.values(q[0], s[0], None if z is None else z[0]).T)
    q, s, z, w = weights(rng, E, N, K, group, kind, zeros, ordinary=True)
    if N % 2 == 0:
        x = int4_cases.sparse(rng, (T, K))
        y, _ = int4_ref.assigned(x, ids, q, s, z)
        want, tol = int4_ref.swiglu(y, np.zeros_like(y))
        got = to_f64(cm.Int4Linear(*w, swiglu=True).forward(bf16(x), i, dtype=torch.float32))
        assert (np.abs(got - want) <= tol + 1e-35).all()


@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("T,E,N,K,group", int4_cases.NORMAL)
def test_rms_error_of_normal_values(T, E, N, K, group, symmetric):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(K + T)
    w = cm.quantize_int4(bf16(rng.normal(0, K ** -0.5, (E, N, K))), group, symmetric=symmetric)
    x = bf16(rng.normal(0, 1, (T, K)))
    ids = rng.integers(0, E, (T, 1)).astype(np.int32)
    p = rng.random((T, 1))
    i, pd = torch.from_numpy(ids).cuda(), torch.from_numpy(p).float().cuda()
    lin = cm.Int4Linear(*w)
    y, _ = int4_ref.assigned(to_f64(x), ids, int4_ref.unpack(w[0].cpu().numpy()), to_f64(w[1].float()),
                             None if symmetric else w[2].cpu().numpy())
    for got, want in ((lin.forward(x, i, dtype=torch.float32), y),
                      (lin.forward(x, i, pd, dtype=torch.float32), y[:, 0] * to_f64(pd))):
        off = to_f64(got) - want
        assert np.sqrt((off ** 2).mean() / (want ** 2).mean()) < int4_cases.NORMAL_RMS


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("rows,cols,group", [(1, 32, 32), (37, 192, 64), (130, 1280, 128), (5, 1536, 768)])
def test_values_of_fp16_scales(rows, cols, group, zeros):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(rows + cols)
    q = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    bits = rng.integers(0, 0x7C00, (rows, cols // group)).astype(np.uint16)  # every finite one, subnormals among them
    bits.flat[:4] = np.array([0x0001, 0x7BFF, 0x0030, 0x03FF], np.uint16)[:bits.size]
    s = bits.view(np.float16).astype(np.float64)
    z = rng.integers(0, 16, s.shape).astype(np.uint8) if zeros else None
    exact = int4_ref.values(q, s, z)
    sd = torch.from_numpy(bits.view(np.float16)).cuda()
    args = torch.from_numpy(int4_ref.pack(q)).cuda(), sd, None if z is None else torch.from_numpy(z).cuda()
    assert np.array_equal(to_f64(cm.dequantize_int4(*args, dtype=torch.float32)), exact)
    assert np.array_equal(to_f64(cm.dequantize_int4(*args).float()), int4_ref.to_bf16(exact))


# 64 tokens' sums of 16 waves and one tile, or of 8 waves and two tiles, are 64 KiB of
# LDS beside the waves' x; one more token takes another form.
@pytest.mark.parametrize("T", [64, 65, 128])
@pytest.mark.parametrize("E,N,K,group", [(64, 40, 64, 32), (128, 34, 128, 128), (30, 50, 96, 32), (24, 66, 192, 64),
                                         (2, 8200, 64, 64), (64, 8210, 32, 32), (30, 8230, 64, 64)])
def test_weighted_sums_of_most_tokens(T, E, N, K, group):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(T + E + N)
    q, s, z, w = integers(rng, E, N, K, group)
    ids, p = some_ids(rng, T, 1, E, "mixed"), 2.0 ** rng.integers(-2, 2, (T, 1))
    x = ints(rng, (T, K))
    want = np.zeros((T, N))
    for t in range(T):
        e = ids[t, 0]
        if 0 <= e < E:
            want[t] = p[t, 0] * (int4_ref.values(q[e], s[e], z[e]) @ x[t])
    i, pd = torch.from_numpy(ids).cuda(), torch.from_numpy(p).float().cuda()
    lin = cm.Int4Linear(*w)
    exact_equal(lin.forward(bf16(x), i, pd, dtype=torch.float32), want)
    exact_equal(lin.forward(bf16(x), i, pd), want)
