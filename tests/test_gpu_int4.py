"""4-bit integer groups (quantize_int4, dequantize_int4, Int4Linear) against the
plain 64-bit reference of int4_ref.py.

* Codes, scales, zero points and values read back are exact.
* Products of small integers with power-of-two scales are exact in fp32, so every
  one must come out equal: all forms, sizes, row counts and group lengths.
* Products of normal values stay within the bound int4_ref derives, plus one
  rounding (bf16 2^-8, fp32 2^-24 of the result)."""
import numpy as np
import pytest

import int4_ref
from moe_case import to_f64

pytestmark = pytest.mark.gpu


# --- codec ---------------------------------------------------------------------------------------


def check_codec(t, group, symmetric, few_unsure=True):
    import torch

    import sparse_moe_gemm_amd as cm

    codes, scales, zeros = cm.quantize_int4(t, group, symmetric=symmetric)
    torch.cuda.synchronize()
    q, s, z, unsure = int4_ref.quantize(to_f64(t), group, symmetric)
    assert not few_unsure or unsure.mean() <= 1e-3
    sure = ~unsure.reshape(*s.shape, group).any(axis=-1)
    got_s, got_q = to_f64(scales.float()), int4_ref.unpack(codes.cpu().numpy())
    assert np.array_equal(np.isnan(got_s), np.isnan(s)) and np.array_equal(got_s[sure], s[sure], equal_nan=True)
    if symmetric:
        assert zeros is None
    else:
        assert np.array_equal(zeros.cpu().numpy()[sure], z[sure])
    wrong = (got_q != q) & ~unsure
    assert not wrong.any(), f"codes differ at {np.argwhere(wrong)[:3].tolist()}"
    assert (np.abs(got_q.astype(int) - q.astype(int))[unsure] <= 1).all()
    exact = int4_ref.values(got_q, got_s, None if symmetric else zeros.cpu().numpy())
    for dtype, fix in ((torch.float32, lambda v: v.astype(np.float32).astype(np.float64)), (None, int4_ref.to_bf16)):
        back = cm.dequantize_int4(codes, scales, zeros, dtype)
        ok = np.isfinite(exact)
        assert np.array_equal(to_f64(back.float())[ok], fix(exact[ok])) and back.float().isnan().cpu().numpy()[~ok].all()
    return codes, scales, zeros


@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,group", [(1, 32, 32), (3, 64, 64), (5, 96, 32), (7, 128, 128), (33, 2080, 32),
                                             (64, 1536, 64), (129, 1024, 128), (9, 1024, 256), (4, 768, 768),
                                             (2, 16384, 1024), (1025, 384, 128), (67, 1536, 512), (131, 512, 256), (3, 1920, 640)])
def test_codec(rows, cols, group, dtype, symmetric):
    import torch

    g = torch.Generator().manual_seed(rows + cols)
    w = torch.randn(rows, cols, generator=g) * torch.logspace(-6, 4, rows)[:, None]
    w[0, : cols // 2] = w[0, : cols // 2].abs()   # groups of one sign
    w[rows // 2, : group] = 0
    w = (w.bfloat16() if dtype == "bf16" else w).cuda()
    check_codec(w, group, symmetric, few_unsure=dtype == "bf16")
    wide = torch.zeros(rows, cols + 13, dtype=w.dtype, device="cuda")
    wide[:, 5:5 + cols] = w
    a, b = (__import__("sparse_moe_gemm_amd").quantize_int4(v, group, symmetric=symmetric)
            for v in (w, wide[:, 5:5 + cols]))
    assert all(x is y or torch.equal(x, y) for x, y in zip(a, b))


def test_codec_special_groups():
    import torch

    rows = np.zeros((16, 64))
    rows[0] = np.arange(64) - 20.0
    rows[1] = 2.0 ** -133  # least bf16 value: the scale rounds to 0
    rows[2, 5] = 3e38
    rows[3, 5], rows[3, 9] = 3e38, -3e38  # hi - lo is no fp32 value
    rows[4, 7] = np.inf
    rows[5, 40] = np.nan
    rows[6] = 1e-38 * np.linspace(-1, 1, 64)
    rows[7] = np.where(np.arange(64) % 2, 7.5, -7.5)
    rows[8] = -1.0
    rows[9] = 15.0
    rows[10] = np.arange(64) % 16 - 7.5  # ties in w / s
    rows[11] = np.arange(64) % 15 - 7.0
    t = torch.from_numpy(rows).float().bfloat16().cuda()
    for symmetric in (False, True):
        check_codec(t[[0, 1, 2, 4, 5, 6, 7, 8, 9, 10, 11, 12]], 32, symmetric, few_unsure=False)
        check_codec(t[[0, 2, 5, 7]], 64, symmetric, few_unsure=False)
    import sparse_moe_gemm_amd as cm

    codes, scales, zeros = cm.quantize_int4(t[3:4], 64)
    back = cm.dequantize_int4(codes, scales, zeros, torch.float32)
    assert abs(back[0, 5].item() - 3e38) <= 4e37 and abs(back[0, 9].item() + 3e38) <= 4e37 and back[0, 0].item() == 0


@pytest.mark.parametrize("symmetric", [False, True])
def test_codes_are_those_of_fp32_division(symmetric):
    """Values on the ties between codes and one float beside them, under scales of
    every exponent: rint of the IEEE quotient w / s, plus z."""
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(7)
    rows, group = 4096, 32
    s = ((1 + rng.integers(0, 128, rows) / 128) * 2.0 ** rng.integers(-124, 122, rows)).astype(np.float32)
    z = np.full(rows, 8) if symmetric else rng.integers(0, 16, rows)
    w = ((rng.integers(-z[:, None], 15 - z[:, None], (rows, group)) + 0.5) * s[:, None].astype(np.float64)).astype(np.float32)
    side = rng.integers(-1, 2, w.shape)
    w = np.where(side < 0, np.nextafter(w, np.float32(-np.inf)), np.where(side > 0, np.nextafter(w, np.float32(np.inf)), w))
    lo, hi = ((-7, 7) if symmetric else (-z, 15 - z))
    w = np.clip(w, (lo * s)[:, None], (hi * s)[:, None]).astype(np.float32)
    w[:, 0], w[:, 1] = lo * s, hi * s  # the group's scale is s, its zero point z
    codes, scales, zeros = cm.quantize_int4(torch.from_numpy(w).cuda(), group, symmetric=symmetric)
    torch.cuda.synchronize()
    assert np.array_equal(to_f64(scales.float())[:, 0], s.astype(np.float64))
    assert symmetric or np.array_equal(zeros.cpu().numpy()[:, 0], z)
    want = np.clip(np.rint(w / s[:, None]) + z[:, None], 0, 15)
    assert np.array_equal(int4_ref.unpack(codes.cpu().numpy()), want)


def test_codec_three_dimensions_empty_and_streams():
    import torch

    import sparse_moe_gemm_amd as cm

    w = torch.randn(5, 24, 256, device="cuda").bfloat16()
    got = cm.quantize_int4(w, 64)
    flat = cm.quantize_int4(w.view(120, 256), 64)
    assert all(torch.equal(a.view(b.shape), b) for a, b in zip(got, flat))
    assert got[0].shape == (5, 24, 128) and got[1].shape == (5, 24, 4)
    want = cm.dequantize_int4(*got)
    assert want.shape == w.shape
    assert cm.quantize_int4(w[0, :0], 64)[0].shape == (0, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = cm.quantize_int4(w, 64, stream=side)
    back = cm.dequantize_int4(*other, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, got)) and torch.equal(back, want)
    graph = torch.cuda.CUDAGraph()
    src = w.clone()
    with torch.cuda.graph(graph):
        out = cm.dequantize_int4(*cm.quantize_int4(src, 64))
    for r in range(3):
        src.copy_(torch.roll(w, r, 0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, torch.roll(want, r, 0)), r
        cm.quantize_int4(w, 64)


def test_codec_past_32_bits():
    """More than 2^32 values: the last rows as they are alone."""
    import torch

    import sparse_moe_gemm_amd as cm

    rows, cols = (1 << 20) + 3, 4096
    w = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    w.fill_(0.5)
    tail = torch.randn(3, cols, device="cuda").bfloat16()
    w[-3:] = tail
    codes, scales, zeros = cm.quantize_int4(w, 128)
    want = cm.quantize_int4(tail, 128)
    assert all(torch.equal(a[-3:], b) for a, b in zip((codes, scales, zeros), want))
    assert torch.equal(cm.dequantize_int4(codes, scales, zeros)[-3:], cm.dequantize_int4(*want))


# --- products ------------------------------------------------------------------------------------


def integers(rng, E, N, K, group, zeros=True, f16=False):
    """Weights whose products with small integers are exact in fp32."""
    import torch

    q = rng.integers(0, 16, (E, N, K)).astype(np.uint8)
    s = 2.0 ** rng.integers(-2, 2, (E, N, K // group))
    z = rng.integers(0, 16, (E, N, K // group)).astype(np.uint8) if zeros else None
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    return q, s, z, (dev(int4_ref.pack(q)), dev(s).to(torch.float16 if f16 else torch.bfloat16), dev(z))


def ints(rng, shape):
    return rng.integers(-3, 4, shape).astype(np.float64)


def bf16(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).float().bfloat16().cuda()


def exact_equal(y, want):
    """fp32 or bf16 results against exact ones."""
    import torch

    torch.cuda.synchronize()
    want = int4_ref.to_bf16(want) if y.dtype == torch.bfloat16 else want
    bad = np.argwhere(to_f64(y) != want)
    assert bad.size == 0, f"{len(bad)} differ, first {bad[0].tolist()}: {to_f64(y)[tuple(bad[0])]} for {want[tuple(bad[0])]}"


DENSE = [(1, 1, 32, 32), (1, 2, 64, 64), (1, 15, 128, 128), (2, 16, 96, 32), (3, 17, 160, 32), (5, 33, 192, 64),
         (16, 64, 256, 128), (17, 50, 288, 32), (31, 100, 512, 256), (33, 257, 2080, 32), (48, 31, 1024, 1024),
         (64, 2050, 384, 128), (65, 40, 640, 128), (127, 96, 320, 64), (128, 130, 1088, 64), (7, 1025, 4096, 128),
         (1, 48, 14336, 128), (9, 4096, 2048, 64)]


@pytest.mark.parametrize("zeros,f16", [(True, False), (False, True)])
@pytest.mark.parametrize("T,N,K,group", DENSE)
def test_dense(T, N, K, group, zeros, f16):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(T + N + K)
    q, s, z, w = integers(rng, 1, N, K, group, zeros, f16)
    x = ints(rng, (T, K))
    lin = cm.Int4Linear(*(None if t is None else t[0] for t in w))
    want = x @ int4_ref.values(q[0], s[0], None if z is None else z[0]).T
    exact_equal(lin.forward(bf16(x), dtype=torch.float32), want)
    exact_equal(lin.forward(bf16(x)), want)


def some_ids(rng, T, k, E, kind):
    if kind == "distinct":
        return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    if kind == "one":  # all on one expert, in every slot
        return np.full((T, k), E // 2, np.int32)
    if kind == "none":
        return rng.choice([-1, E, E + 7, -2 ** 31, 2 ** 31 - 1], (T, k)).astype(np.int32)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)  # repeats, and some of no expert
    ids[rng.random((T, k)) < 0.3] = rng.choice([-1, E, -2 ** 31, 2 ** 31 - 1])
    return ids


EXPERTS = [(1, 1, 1, 16, 32, 32), (1, 2, 8, 34, 256, 128), (7, 2, 8, 96, 384, 128), (16, 4, 128, 66, 256, 64),
           (16, 8, 24, 48, 160, 32), (5, 3, 6, 130, 1024, 256), (40, 3, 5, 50, 128, 64), (64, 2, 3, 64, 192, 32),
           (128, 1, 256, 32, 128, 128), (128, 1, 2, 62, 640, 128), (33, 3, 40, 36, 2080, 32), (2, 5, 7, 18, 4096, 128)]


@pytest.mark.parametrize("kind", ["distinct", "mixed", "one", "none"])
@pytest.mark.parametrize("T,k,E,N,K,group", EXPERTS)
def test_experts(T, k, E, N, K, group, kind):
    import torch

    import sparse_moe_gemm_amd as cm

    if kind == "distinct" and k > E:
        pytest.skip("fewer experts than slots")
    rng = np.random.default_rng(T * k + N + K)
    q, s, z, w = integers(rng, E, N, K, group, zeros=T % 2 == 1, f16=N % 4 == 0)
    ids = some_ids(rng, T, k, E, kind)
    weights = 2.0 ** rng.integers(-2, 2, (T, k))
    i = torch.from_numpy(ids).cuda()
    p = torch.from_numpy(weights).float().cuda()
    lin, glu = cm.Int4Linear(*w), cm.Int4Linear(*w, swiglu=True)
    for x in (ints(rng, (T, K)), ints(rng, (T, k, K))):
        y, _ = int4_ref.assigned(x, ids, q, s, z)
        exact_equal(lin.forward(bf16(x), i, dtype=torch.float32), y)
        exact_equal(lin.forward(bf16(x), i), y)
        exact_equal(lin.forward(bf16(x), i, p, dtype=torch.float32), (y * weights[:, :, None]).sum(axis=1))
        exact_equal(lin.forward(bf16(x), i, p), (y * weights[:, :, None]).sum(axis=1))
        want, tol = int4_ref.swiglu(y, np.zeros_like(y))
        got = to_f64(glu.forward(bf16(x), i, dtype=torch.float32))
        assert (np.abs(got - want) <= tol + 1e-35).all()


def test_dense_swiglu():
    import torch

    import sparse_moe_gemm_amd as cm

    for T, f, K, group in ((1, 1, 32, 32), (3, 15, 96, 32), (17, 33, 256, 128), (40, 100, 320, 64), (128, 16, 128, 128)):
        rng = np.random.default_rng(T + f)
        q, s, z, w = integers(rng, 1, 2 * f, K, group)
        x = ints(rng, (T, K))
        y, _ = int4_ref.product64(x, q[0], s[0], z[0])
        want, tol = int4_ref.swiglu(y, np.zeros_like(y))
        lin = cm.Int4Linear(*(t[0] for t in w), swiglu=True)
        got = to_f64(lin.forward(bf16(x), dtype=torch.float32))
        assert got.shape == (T, f) and (np.abs(got - want) <= tol + 1e-35).all()
        # one matrix through ids
        i = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
        assert np.array_equal(to_f64(lin.forward(bf16(x), i, dtype=torch.float32))[:, 0], got)


# More rows of weights: other divisions of the work among workgroups and waves, with
# last tiles that fill no group of them.
@pytest.mark.parametrize("T,N,K,group,swiglu", [
    (3, 9000, 96, 32, False), (7, 8233, 128, 128, False), (12, 9001, 192, 64, False), (2, 24650, 64, 64, False),
    (8, 24645, 128, 128, False), (9, 24650, 96, 32, False), (5, 8200, 8256, 64, False), (13, 8199, 8192, 128, False),
    (33, 5490, 160, 32, False), (128, 2130, 384, 128, False), (100, 2129, 320, 64, False),
    (4, 8800, 96, 32, True), (16, 24660, 64, 64, True), (6, 8260, 8224, 32, True), (128, 2200, 256, 128, True),
    (47, 7000, 96, 32, True)])
def test_dense_of_many_rows(T, N, K, group, swiglu):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(T + N + K)
    q, s, z, w = integers(rng, 1, N, K, group)
    x = ints(rng, (T, K))
    y = x @ int4_ref.values(q[0], s[0], z[0]).T
    got = cm.Int4Linear(*(t[0] for t in w), swiglu=swiglu).forward(bf16(x), dtype=torch.float32)
    if swiglu:
        want, tol = int4_ref.swiglu(y, np.zeros_like(y))
        assert (np.abs(to_f64(got) - want) <= tol + 1e-35).all()
    else:
        exact_equal(got, y)


@pytest.mark.parametrize("kind", ["distinct", "mixed", "one"])
@pytest.mark.parametrize("T,k,E,N,K,group", [(4, 2, 3, 8200, 64, 64), (10, 1, 3, 8202, 96, 32), (16, 2, 3, 8230, 128, 128),
                                             (100, 1, 30, 70, 256, 128), (100, 1, 100, 66, 128, 64), (90, 1, 3, 8200, 32, 32),
                                             (64, 2, 4, 4140, 64, 64), (16, 2, 40, 530, 128, 128), (33, 2, 3, 9010, 32, 32)])
def test_experts_of_many_rows(T, k, E, N, K, group, kind):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(T * k + N + K)
    q, s, z, w = integers(rng, E, N, K, group)
    ids = some_ids(rng, T, k, E, kind)
    x, weights = ints(rng, (T, K)), 2.0 ** rng.integers(-2, 2, (T, k))
    by_expert = [x @ int4_ref.values(q[e], s[e], z[e]).T for e in range(E)]
    y = np.array([[by_expert[e][t] if 0 <= e < E else np.zeros(N) for e in ids[t]] for t in range(T)])
    i, p = torch.from_numpy(ids).cuda(), torch.from_numpy(weights).float().cuda()
    lin = cm.Int4Linear(*w)
    exact_equal(lin.forward(bf16(x), i, dtype=torch.float32), y)
    exact_equal(lin.forward(bf16(x), i, p, dtype=torch.float32), (y * weights[:, :, None]).sum(axis=1))
    want, tol = int4_ref.swiglu(y, np.zeros_like(y))
    got = to_f64(cm.Int4Linear(*w, swiglu=True).forward(bf16(x), i, dtype=torch.float32))
    assert (np.abs(got - want) <= tol + 1e-35).all()


@pytest.mark.parametrize("T,k,E,N,K,group", [(1, 1, 1, 512, 4096, 128), (33, 1, 1, 130, 2080, 32), (7, 2, 8, 96, 14336, 128),
                                             (16, 4, 32, 256, 2048, 64), (64, 2, 4, 64, 1024, 256)])
def test_normal_values(T, k, E, N, K, group):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(K + T)
    wt = torch.from_numpy(rng.normal(0, K ** -0.5, (E, N, K))).float().bfloat16().cuda()
    ids = some_ids(rng, T, k, E, "mixed" if E > 1 else "one")
    weights = rng.random((T, k))
    i, p = torch.from_numpy(ids).cuda(), torch.from_numpy(weights).float().cuda()
    p64 = to_f64(p)
    for symmetric in (False, True):
        w = cm.quantize_int4(wt, group, symmetric=symmetric)
        q, s = int4_ref.unpack(w[0].cpu().numpy()), to_f64(w[1].float())
        z = None if symmetric else w[2].cpu().numpy()
        lin, glu = cm.Int4Linear(*w), cm.Int4Linear(*w, swiglu=True)
        x = bf16(rng.normal(0, 1, (T, K)))
        y, tol = int4_ref.assigned(to_f64(x), ids, q, s, z)
        ws = (y * p64[:, :, None]).sum(axis=1)
        wtol = ((tol + k * 2.0 ** -22 * np.abs(y)) * p64[:, :, None]).sum(axis=1)
        gl, gtol = int4_ref.swiglu(y, tol)
        for dtype, half in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
            for got, want, t in ((lin.forward(x, i, dtype=dtype), y, tol), (lin.forward(x, i, p, dtype=dtype), ws, wtol),
                                 (glu.forward(x, i, dtype=dtype), gl, gtol)):
                assert got.dtype == dtype
                assert (np.abs(to_f64(got) - want) <= t + half * (np.abs(want) + t) + 1e-35).all()


def test_gates_beyond_the_largest_float():
    """A gate of -infinity (its fp32 sum overflows) closes: its exact SiLU rounds to -0."""
    import torch

    import sparse_moe_gemm_amd as cm

    codes = torch.full((32, 64), 0x00, dtype=torch.uint8, device="cuda")
    codes[16:] = 0x99  # up: 1 each
    scales = torch.ones(32, 1, dtype=torch.bfloat16, device="cuda")
    scales[:8] = 2.0 ** 120
    lin = cm.Int4Linear(codes, scales, swiglu=True)
    for T in (1, 7, 40):
        y = lin.forward(bf16(np.ones((T, 128))), dtype=torch.float32)
        torch.cuda.synchronize()
        assert (y == 0).all() and y.shape == (T, 16)


def test_rows_do_not_reach_each_other():
    """The same rows in other batches give the same values (terms are added in an
    order that depends on the call: each result within its own bound), rows
    beside ones of NaN and infinities the same bits; scales of NaN reach their
    own outputs alone; the same call gives the same bits."""
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(4)
    E, N, K = 6, 80, 512
    w = cm.quantize_int4(bf16(rng.normal(0, 0.05, (E, N, K))), 128)
    lin = cm.Int4Linear(*w)
    x = bf16(rng.normal(0, 1, (40, K)))
    ids = torch.from_numpy(some_ids(rng, 40, 3, E, "distinct")).cuda()
    p = torch.rand(40, 3, device="cuda")
    whole, summed = lin.forward(x, ids, dtype=torch.float32), lin.forward(x, ids, p, dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(lin.forward(x, ids, dtype=torch.float32), whole)
        assert torch.equal(lin.forward(x, ids, p, dtype=torch.float32), summed)
    y, tol = int4_ref.assigned(to_f64(x), ids.cpu().numpy(), int4_ref.unpack(w[0].cpu().numpy()), to_f64(w[1].float()),
                               w[2].cpu().numpy())
    bound = ((tol + 3 * 2.0 ** -22 * np.abs(y)) * to_f64(p)[:, :, None]).sum(axis=1)
    for n in (1, 2, 15, 16, 17, 33):
        part = lin.forward(x[:n], ids[:n].contiguous(), dtype=torch.float32)
        assert (np.abs(to_f64(part) - to_f64(whole[:n])) <= 2 * tol[:n]).all(), n
        part = lin.forward(x[:n], ids[:n].contiguous(), p[:n].contiguous(), dtype=torch.float32)
        assert (np.abs(to_f64(part) - to_f64(summed[:n])) <= 2 * bound[:n]).all(), n
    bad = x.clone()
    bad[3, 7], bad[11, 0], bad[25, K - 1] = float("nan"), float("inf"), -float("inf")
    got, gots = lin.forward(bad, ids, dtype=torch.float32), lin.forward(bad, ids, p, dtype=torch.float32)
    rest = [t for t in range(40) if t not in (3, 11, 25)]
    assert torch.equal(got[rest], whole[rest]) and torch.equal(gots[rest], summed[rest])
    assert got[[3, 11, 25]].isnan().all() and gots[[3, 11, 25]].isnan().all()
    scales = w[1].clone()
    scales[2, 5, 1] = float("nan")
    got = cm.Int4Linear(w[0], scales, w[2]).forward(x, ids, dtype=torch.float32)
    hit = (ids == 2)[:, :, None] & (torch.arange(N, device="cuda") == 5)
    assert got[hit].isnan().all() and torch.equal(got[~hit], whole[~hit])


def test_memory_around_y_and_streams_and_graphs():
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(5)
    E, N, K, T, k = 9, 50, 416, 12, 2
    q, s, z, w = integers(rng, E, N, K, 32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    lin = cm.Int4Linear(*w, stream=side)
    torch.cuda.synchronize()
    x, ids = ints(rng, (T, K)), some_ids(rng, T, k, E, "mixed")
    want, _ = int4_ref.assigned(x, ids, q, s, z)
    xd, i, p = bf16(x), torch.from_numpy(ids).cuda(), torch.full((T, k), 0.5, device="cuda")
    flat = torch.full((T * k * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = flat[32:32 + T * k * N].view(T, k, N)
    assert lin.forward(xd, i, y=y) is y
    exact_equal(y, want)
    assert (flat[:32] == 7).all() and (flat[-32:] == 7).all()
    got = lin.forward(xd, i, stream=side)
    exact_equal(got, want)
    # two streams at once on the same weights
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [lin.forward(xd, i, p, dtype=torch.float32, stream=st) for _ in range(10) for st in (side, other)]
    for o in outs:
        exact_equal(o, 0.5 * want.sum(axis=1))
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    src = xd.clone()
    with torch.cuda.graph(graph):
        out = lin.forward(src, i, p)
    with torch.cuda.graph(second):
        out2 = lin.forward(src, i)
    for r in range(4):
        src.copy_(xd if r % 2 == 0 else -xd)
        torch.cuda.synchronize()
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        sign = 1 if r % 2 == 0 else -1
        exact_equal(out, sign * 0.5 * want.sum(axis=1))
        exact_equal(out2, sign * want)
        lin.forward(xd, i)
    assert lin.forward(xd[:0], i[:0]).shape == (0, k, N)
    assert lin.forward(xd[:0], i[:0], p[:0]).shape == (0, N)
    with pytest.raises(cm.ColibriError):
        lin.forward(bf16(np.zeros((65, K))), torch.zeros(65, 2, dtype=torch.int32, device="cuda"))


def test_weights_past_32_bits():
    """Codes of more than 4 GiB: rows at both ends."""
    import torch

    import sparse_moe_gemm_amd as cm

    N, K = (1 << 20) + 5, 12288
    codes = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    pick = [0, 1, 77, N // 2, N - 2, N - 1]
    rng = np.random.default_rng(8)
    q = rng.integers(0, 16, (len(pick), K)).astype(np.uint8)
    codes[torch.tensor(pick, device="cuda")] = torch.from_numpy(int4_ref.pack(q)).cuda()
    scales = torch.full((N, K // 128), 0.5, dtype=torch.bfloat16, device="cuda")
    lin = cm.Int4Linear(codes, scales)
    x = ints(rng, (2, K))
    y = lin.forward(bf16(x), dtype=torch.float32)
    exact_equal(y[:, pick], x @ ((q.astype(np.float64) - 8) * 0.5).T)
    y[:, pick] = 0
    assert (y == 0).all()
