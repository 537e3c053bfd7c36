"""4-bit microscaled rows and weights, what needs no GPU: the test reference
against hand-worked blocks, and the refusals of the entry points and flags
(checked before anything reaches the device)."""
import numpy as np
import pytest

import mx_ref
import sparse_moe_gemm_amd as cm

FAKE = 0x100000  # never dereferenced


def test_reference_on_hand_worked_blocks():
    v = np.zeros(32)
    v[:8] = [6.0, -6.0, 0.25, 0.75, 1.75, 2.5, 3.5, 5.0]  # every tie but one, scale 1
    c, s = mx_ref.quantize(v[None])
    assert s.tolist() == [[127]]
    assert c[0, :8].tolist() == [7, 15, 0, 2, 4, 4, 6, 6]
    v[0] = 6.5  # no longer fits under 6: the next power of two
    c, s = mx_ref.quantize(v[None])
    assert s.tolist() == [[128]] and c[0, 0] == 5  # 3.25 -> 3
    c, s = mx_ref.quantize(np.zeros((1, 32)))
    assert s.tolist() == [[127]] and not c.any()
    assert mx_ref.quantize(-np.zeros((1, 32)))[0].tolist() == [[8] * 32]
    assert mx_ref.scale_bytes([2.0 ** -130, 2.0 ** 127 * 1.99, np.inf, np.nan]).tolist() == [0, 253, 255, 255]
    big = np.full((1, 64), 3.0)
    big[0, 40] = np.nan
    c, s = mx_ref.quantize(big)
    val = mx_ref.values(c, s)
    assert s.tolist() == [[126, 255]] and np.all(val[0, :32] == 3.0) and np.isnan(val[0, 32:]).all()


def test_reference_values_are_nearest_and_requantize_to_themselves():
    rng = np.random.default_rng(5)
    v = rng.standard_normal((20, 96)) * np.exp(rng.uniform(-30, 30, (20, 1)))
    q = mx_ref.rounded(v)
    blk = np.abs(v).reshape(20, 3, 32).max(axis=-1)
    # half of the widest step, 2 under a maximum above 3 (of 6)
    assert np.all(np.abs(q - v).reshape(20, 3, 32).max(axis=-1) <= blk / 3 * 1.0000001)
    assert np.array_equal(mx_ref.rounded(q), q)
    c = rng.integers(0, 16, (7, 64)).astype(np.uint8)
    assert np.array_equal(mx_ref.unpack(mx_ref.pack(c)), c)


@pytest.mark.parametrize("args,status", [
    ((None, cm.BF16, 4, 64, 64, FAKE, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, cm.BF16, 4, 64, 64, None, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, cm.BF16, 4, 64, 64, FAKE, None), cm.ERR_INVALID_ARG),
    ((FAKE, 7, 4, 64, 64, FAKE, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, cm.BF16, 0, 64, 64, FAKE, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, cm.BF16, -1, 64, 64, FAKE, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, cm.BF16, 4, 0, 64, FAKE, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, cm.BF16, 4, 48, 64, FAKE, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, cm.BF16, 4, 64, 63, FAKE, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, cm.BF16, 1 << 36, 64, 64, FAKE, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, cm.BF16, 1 << 20, 64, 1 << 40, FAKE, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE + 1, cm.BF16, 4, 64, 64, FAKE, FAKE), cm.ERR_ALIGNMENT),
    ((FAKE + 2, cm.F32, 4, 64, 64, FAKE, FAKE), cm.ERR_ALIGNMENT),
    ((FAKE, cm.F32, 4, 64, 64, FAKE + 2, FAKE), cm.ERR_ALIGNMENT),
])
def test_quantize_mxfp4_rejects_bad_arguments(args, status):
    assert cm.colibri_moe_quantize_mxfp4(*args) == status


@pytest.mark.parametrize("args,status", [
    ((None, FAKE, 4, 64, cm.BF16, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, None, 4, 64, cm.BF16, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, FAKE, 4, 64, cm.BF16, None), cm.ERR_INVALID_ARG),
    ((FAKE, FAKE, 4, 64, 2, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, FAKE, 0, 64, cm.BF16, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, FAKE, 4, 40, cm.BF16, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE, FAKE, 1 << 36, 64, cm.BF16, FAKE), cm.ERR_INVALID_ARG),
    ((FAKE + 2, FAKE, 4, 64, cm.BF16, FAKE), cm.ERR_ALIGNMENT),
    ((FAKE, FAKE, 4, 64, cm.F32, FAKE + 8), cm.ERR_ALIGNMENT),
])
def test_dequantize_mxfp4_rejects_bad_arguments(args, status):
    assert cm.colibri_moe_dequantize_mxfp4(*args) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=cm.F32, flags=cm.FLAG_MXFP4_WEIGHTS), cm.ERR_UNSUPPORTED),
    (dict(flags=cm.FLAG_MXFP4_WEIGHTS | cm.FLAG_FP8_WEIGHTS), cm.ERR_UNSUPPORTED),
    (dict(flags=cm.FLAG_MXFP4_ACTIVATIONS), cm.ERR_UNSUPPORTED),
    (dict(flags=cm.FLAG_FP8_WEIGHTS | cm.FLAG_MXFP4_ACTIVATIONS), cm.ERR_UNSUPPORTED),
    (dict(flags=cm.FLAG_MXFP4_WEIGHTS | cm.FLAG_FP8_ACTIVATIONS), cm.ERR_UNSUPPORTED),
    (dict(d_model=192, flags=cm.FLAG_MXFP4_WEIGHTS), cm.ERR_UNSUPPORTED),
    (dict(d_ff=64, flags=cm.FLAG_MXFP4_WEIGHTS), cm.ERR_UNSUPPORTED),
])
def test_init_rejects_bad_4_bit_configs(kw, status):
    base = dict(d_model=256, d_ff=128, n_experts=8, top_k=2, max_tokens=64, dtype=cm.BF16, flags=0)
    base.update(kw)
    st, h = cm.colibri_moe_init(cm.Config(**base), cm.Weights(FAKE, None, FAKE, FAKE, FAKE))
    assert st == status and not h


def test_forward_few_rejects_unknown_handles():
    assert cm.colibri_moe_forward_few(None, FAKE, 4, FAKE) == cm.ERR_INVALID_ARG
    assert cm.colibri_moe_forward_few(FAKE, FAKE, 4, FAKE) == cm.ERR_INVALID_ARG


def test_few_token_limit_matches_the_header():
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "colibri_moe.h")).read()
    assert int(re.search(r"#define COLIBRI_MOE_FEW_TOKENS (\d+)", text).group(1)) == cm.FEW_TOKENS


def test_python_wrappers_reject_wrong_tensors():
    import torch

    with pytest.raises(TypeError):
        cm.quantize_mxfp4(torch.zeros(2, 32, dtype=torch.bfloat16))  # not on a GPU
    with pytest.raises(TypeError):
        cm.dequantize_mxfp4(torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8))
    with pytest.raises(TypeError):
        cm.dequantize_mxfp4(None, None, dtype=torch.float16)
