"""An Int4Linear that goes out of use while its product waits on another stream than the
one it was made on: its memory is not handed out before."""
import numpy as np
import pytest

import int4_ref
from test_gpu_int4 import bf16, exact_equal, integers, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_packed_outlives_its_object(captured):
    import torch

    import sparse_moe_gemm_amd as cm

    rng = np.random.default_rng(11)
    T, N, K = 5, 640, 1024
    q, s, z, w = integers(rng, 1, N, K, 128)
    x = ints(rng, (T, K))
    xd, want = bf16(x), x @ int4_ref.values(q[0], s[0], z[0]).T
    busy = torch.randn(2048, 2048, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(3):
        lin = cm.Int4Linear(*(t[0] for t in w))
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = lin.forward(xd)
            for _ in range(3):
                graph.replay()
                lin.forward(xd)
                exact_equal(y, want)
            del lin
            exact_equal(y, want)
            continue
        size = lin.packed.numel()
        with torch.cuda.stream(side):
            for _ in range(20):  # keeps the stream busy
                busy @ busy
            y = lin.forward(xd, dtype=torch.float32)
        del lin
        junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        exact_equal(y, want)
        del junk
