"""Zero points whose bytes hold more than four bits: the low four count, for the
values read back and for the products alike."""
import numpy as np
import pytest

import int4_ref
from moe_case import to_f64
from test_gpu_int4 import bf16, exact_equal, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,group", [(3, 32, 32), (50, 384, 128), (17, 192, 64)])
def test_low_four_bits_count(rows, cols, group):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(rows + cols)
    q = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    s = 2.0 ** rng.integers(-2, 2, (rows, cols // group))
    z = rng.integers(0, 256, s.shape).astype(np.uint8)
    z.flat[:3] = [0x1F, 0xF0, 0x80]
    want = int4_ref.values(q, s, z & 15)
    args = torch.from_numpy(int4_ref.pack(q)).cuda(), torch.from_numpy(s).bfloat16().cuda(), torch.from_numpy(z).cuda()
    assert np.array_equal(to_f64(cm.dequantize_int4(*args, dtype=torch.float32)), want)
    assert np.array_equal(to_f64(cm.dequantize_int4(*args).float()), want)
    x = ints(rng, (4, cols))
    exact_equal(cm.Int4Linear(*args).forward(bf16(x), dtype=torch.float32), x @ want.T)
