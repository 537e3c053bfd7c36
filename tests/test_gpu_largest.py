"""The largest calls of the operators around the layer: outputs of more than 2^31 values,
against the same rows in small calls, at both ends and beside every power of two that an
index of 32 bits would wrap at."""
import numpy as np
import pytest

import int4_ref
from test_gpu_int4 import bf16, exact_equal, ints

pytestmark = pytest.mark.gpu


def slices(rows, *borders):
    for b in (0, *borders, rows):
        a, e = max(0, b - 40), min(rows, b + 40)
        if a < e:
            yield slice(a, e)


def test_route_of_more_tokens_than_one_launch_takes():
    import torch

    import sparse_moe_gemm_amd as cm

    T, E, k = (1 << 28) + 21, 8, 8
    logits = torch.randn(T, E, device="cuda", dtype=torch.bfloat16)
    rule = cm.RoutingRule("sigmoid", groups=4, top_groups=4, scale=2.0)
    ids, w = cm.route(logits, k, rule)
    assert ids.numel() > 1 << 31
    for s in slices(T, 1 << 27, 1 << 28, (1 << 27) + (1 << 26)):
        i, v = cm.route(logits[s], k, rule)
        assert torch.equal(ids[s], i) and torch.equal(w[s], v), s


def test_rms_norm_of_more_values_than_32_bits_count():
    import torch

    import sparse_moe_gemm_amd as cm

    rows, d = (1 << 20) + 3, 4104  # above 2^32 values
    x = torch.randn(1 << 16, d, device="cuda").bfloat16().repeat(17, 1)[:rows]
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    got = cm.rms_norm(x, w, residual=x, quantize="fp8")
    for s in slices(rows, (1 << 31) // d, (1 << 32) // d, (1 << 30) // d):
        want = cm.rms_norm(x[s], w, residual=x[s], quantize="fp8")
        assert all(torch.equal(a[s], b) for a, b in zip(got, want)), s


@pytest.mark.parametrize("T", [128, 1])
def test_products_of_most_weight_rows(T):
    """2^24 rows of weights, all zero but a few: T * 2^24 results."""
    import torch

    import sparse_moe_gemm_amd as cm

    N, K = 1 << 24, 32
    codes = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    pick = [0, 1, 15, 16, 4097, N // 2 - 1, N // 2, N - 17, N - 1]
    rng = np.random.default_rng(9)
    q = rng.integers(0, 16, (len(pick), K)).astype(np.uint8)
    codes[torch.tensor(pick, device="cuda")] = torch.from_numpy(int4_ref.pack(q)).cuda()
    scales = torch.full((N, 1), 0.5, dtype=torch.bfloat16, device="cuda")
    x = ints(rng, (T, K))
    y = cm.Int4Linear(codes, scales).forward(bf16(x))
    assert y.numel() == T << 24
    exact_equal(y[:, pick], x @ ((q.astype(np.float64) - 8) * 0.5).T)
    y[:, pick] = 0
    assert all(not row.any().item() for row in y)
