"""Cases and references of the sharp layer checks (tight_ref.py), shared by the
GPU tests and by the CPU test that plants mistakes in a model of the kernels."""
from __future__ import annotations

import torch

import oracle
import synth
import tight_ref
from test_gpu_few import CASES as FEW, MODES, NARROW as FEW_NARROW
from test_gpu_mxfp4 import CASES as LAYERS

C = synth.LayerConfig
# Long rows of W_down: the few-token down kernel takes several trips through its
# two register sets (all modes), with a last partial one. Long token rows: three
# chunks of the token fragments that the gate/up kernel keeps.
FEW_DEEP = [C("deep-3", 3, 256, 8, 4, 8448, "bf16"), C("deep-16", 16, 256, 8, 4, 8448, "bf16"),
            C("deep-9", 9, 384, 4, 2, 4352, "bf16"), C("chunks-6", 6, 8448, 3, 2, 256, "bf16"),
            C("chunks-16", 16, 8576, 3, 1, 384, "bf16")]
# Down GEMMs of the 4-bit layers in two and four K splits, from even and odd K
# units, for one m-tile of every height and for many.
LAYERS_DEEP = [
    C("split-1", 1, 256, 4, 2, 4352, "bf16"),
    C("split-20", 20, 384, 4, 2, 4224, "bf16"),
    C("split-20-odd", 20, 256, 4, 2, 2176, "bf16"),
    C("split-70", 70, 384, 4, 2, 4352, "bf16"),
    C("split-300", 300, 256, 2, 2, 4352, "bf16"),
    # more than 384 rows per expert on average: n-tiles in groups, 17 and 34 of
    # them in the gate/up GEMM (groups of 16)
    C("n-groups-1000", 1000, 1152, 2, 1, 2176, "bf16"),
    C("n-groups-900", 900, 256, 4, 2, 4352, "bf16", {1: 0.5}),
]


def tokens_and_weights(inp, mode, device="cpu"):
    """(x, x of the experts, float64 weights) as a layer of that mode holds them."""
    fp8 = mode.startswith("fp8")
    src = oracle.quantized_expert_weights(inp) if fp8 else inp
    val = tight_ref.mx_round if mode.startswith("mxfp4") else (lambda v: v)
    x = xf = tight_ref.f64(inp["x"], device)
    if mode == "fp8-rows":
        xf = tight_ref.f64(oracle.dequantize_fp8(*oracle.quantize_fp8(inp["x"])), device)
    if mode == "mxfp4-rows":
        xf = tight_ref.mx_round(x)
    w = dict(router=tight_ref.f64(inp["w_router"], device),
             bias=torch.from_numpy(inp["b_router"]).to(device).double())
    for n in ("gate", "up", "down"):
        w[n] = val(tight_ref.f64(src[f"w_{n}"], device))
    return x, xf, w


def route(x, w, k):
    """ids and fp32 weights (as float64) of the k largest logits."""
    logits = x @ w["router"] + w["bias"]
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    return ids[:, :k], torch.softmax(top[:, :k], dim=1).float().double()
