"""The sharp layer checks (tight_ref.py) on the CPU: a model of the kernels in
fp32 passes them, and the same model with a mistake planted in it does not, in
every case that the GPU tests use them for."""
import numpy as np
import pytest
import torch

import mx_ref
import synth
import tight_cases as tc
import tight_ref


def model(x, w, ids, wt, h_parts, mistake=None):
    """y of a kernel-like computation: fp32 products and sums, h in one or two
    bf16 parts, y rounded to bf16."""
    y = torch.zeros(x.shape)
    for e in torch.unique(ids).tolist():
        t, j = torch.where(ids == e)
        rows = x[t].float()
        if mistake == "k":  # 32 of the k of gate and up lost
            rows[:, -32:] = 0
        Wd = w["down"][e].float()
        if mistake == "scale":  # one scale block of 32 down rows doubled
            Wd = Wd.clone()
            Wd[32:64, -32:] *= 2
        g, u = rows @ w["gate"][e].float().T, rows @ w["up"][e].float().T
        h = g / (1 + torch.exp(-g)) * u
        hi = h.bfloat16().float()
        lo = (h - hi).bfloat16().float()
        if mistake == "f":  # 32 of the columns of h lost
            hi[:, -32:] = lo[:, -32:] = 0
        if mistake == "no low part":
            lo = torch.zeros_like(lo)
        if mistake == "low part moved":
            lo = torch.roll(lo, 8, dims=1)
        y.index_add_(0, t, wt[t, j][:, None].float() * ((hi if h_parts == 1 else hi + lo) @ Wd.T))
    return y.bfloat16().double()


def cases():
    for c in tc.FEW + tc.FEW_NARROW + tc.FEW_DEEP:
        for mode in tc.MODES:
            if mode == "fp8-rows" and min(c.d, c.f) < 256:
                continue
            if c in tc.FEW_DEEP and mode in ("fp8", "mxfp4"):
                continue  # as with quantized rows, for the time this takes
            yield pytest.param(c, mode, 2, id=f"few-{c.name}-{mode}")
    for c in tc.LAYERS + tc.LAYERS_DEEP:
        for mode in ("mxfp4", "mxfp4-rows"):
            yield pytest.param(c, mode, 1, id=f"layer-{c.name}-{mode}")


@pytest.mark.parametrize("cfg,mode,h_parts", cases())
def test_planted_mistakes_are_found(cfg, mode, h_parts):
    x, xf, w = tc.tokens_and_weights(synth.make_inputs(cfg), mode)
    x, xf = x[:64], xf[:64]
    ids, wt = tc.route(x, w, cfg.k)
    ref = tight_ref.layer(xf, w, ids, wt, h_parts)
    r = tight_ref.check(model(xf, w, ids, wt, h_parts), ref, cfg.name)
    found = {}
    for mistake in ["k", "f", "scale"] + (["no low part", "low part moved"] if h_parts == 2 else []):
        y = model(xf, w, ids, wt, h_parts, mistake)
        with pytest.raises(AssertionError):
            tight_ref.check(y, ref, cfg.name)
        found[mistake] = float((tight_ref.excess(y, ref[0]) / (2 * ref[1])).max())
    print(r, found)


def test_roundings_agree_with_the_plain_models():
    rng = np.random.default_rng(3)
    v = rng.standard_normal((50, 96)) * np.exp(rng.uniform(-40, 40, (50, 1)))
    v[0, :40] = 0
    v[1, :4] = [6.0, 0.25, 2.5, -5.0]
    assert np.array_equal(tight_ref.mx_round(torch.from_numpy(v)).numpy(), mx_ref.rounded(v))
    f = torch.from_numpy(v.astype(np.float32))
    assert torch.equal(tight_ref.rn(f.double()), f.bfloat16().double())
    want = torch.tensor([1.0, 1 + 2.0 ** -6, 1 + 2.0 ** -7, -0.0, 0.0], dtype=torch.float64)
    assert torch.equal(tight_ref.rn(torch.tensor([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -40,
                                                  -2.0 ** -134, 2.0 ** -135], dtype=torch.float64)), want)
