"""Cases that measure three kinds of calls of the MoE layer library, beside their plain forms in elementary torch
operations:

* ``quant``: bf16 or fp32 rows to 4-bit microscaled codes (E2M1, one power-of-two scale per 32 values) and back to the
  values the codes stand for (``quantize_mxfp4``, ``dequantize_mxfp4``);
* ``layer``: a forward of a layer whose expert weights are 4-bit microscaled (``FLAG_MXFP4_WEIGHTS``), with bf16 token
  rows or with 4-bit ones for the gate/up product (``FLAG_MXFP4_ACTIVATIONS``), from a few tokens to a long prompt;
* ``few``: the whole layer for at most 16 tokens in two launches (``MoELayer.forward_few``), for bf16, 8-bit and 4-bit
  expert weights.
"""
import math

import torch

own = False  # True: the library's calls instead of the plain forms


def listed():
    mixtral = dict(d=4096, E=8, k=2, f=14336, bias=0.0)  # few large experts
    fine = dict(d=2048, E=128, k=4, f=768, bias=0.0)  # many small experts
    skew = dict(d=4096, E=64, k=2, f=1408, bias=4.0)  # two experts take most tokens
    return [
        # the token rows of one small decode batch
        dict(name="quant-decode-rows", op="quant", rows=5, cols=2048, pad=0, dtype="bf16"),
        # one projection of one large expert, as a converter quantises a checkpoint
        dict(name="quant-expert-matrix", op="quant", rows=14336, cols=4096, pad=0, dtype="bf16"),
        # fp32 master weights that are a slice of a wider buffer, odd row count
        dict(name="quant-fp32-slice", op="quant", rows=1003, cols=2080, pad=36, dtype="f32"),
        # one decode step of 32 sequences, large experts: weights are read once
        dict(name="layer-decode-32", op="layer", T=32, act4=False, **mixtral),
        # a decode step of many sequences over many small experts, 4-bit token rows
        dict(name="layer-decode-333", op="layer", T=333, act4=True, **fine),
        # a prompt on large experts, 4-bit token rows: bound by the matrix units
        dict(name="layer-prompt-4096", op="layer", T=4096, act4=True, **mixtral),
        # an odd-sized prompt on many small experts, weights alone in 4 bits
        dict(name="layer-prompt-2047", op="layer", T=2047, act4=False, **fine),
        # skewed routing: two experts with hundreds of rows, many with a few or none
        dict(name="layer-skewed-1000", op="layer", T=1000, act4=False, **skew),
        # one sequence generating, large experts, bf16 weights
        dict(name="few-1-bf16", op="few", T=1, mode="bf16", **mixtral),
        # a full call of 16 tokens over many small experts
        dict(name="few-16-bf16", op="few", T=16, mode="bf16", **fine),
        # a short speculative run on 4-bit weights
        dict(name="few-7-mxfp4", op="few", T=7, mode="mxfp4", **mixtral),
        # three tokens on 8-bit weights with skewed routing
        dict(name="few-3-fp8", op="few", T=3, mode="fp8", **skew),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "layer", "few"])
    if op == "quant":
        cols = 32 * _log_int(rng, 1, 512)
        rows = _log_int(rng, 1, 14336)
        rows = min(rows, 14336 * 4096 // cols)
        return dict(op=op, rows=rows, cols=cols, pad=4 * rng.choice([0, 0, 1, 9, 32]), dtype=rng.choice(["bf16", "f32"]))
    while True:
        d, f = 128 * _log_int(rng, 1, 32), 128 * _log_int(rng, 1, 112)
        E = _log_int(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        T = rng.randint(1, 16) if op == "few" else _log_int(rng, 1, 4096)
        if E * d * f <= 8 * 4096 * 14336 and T * k * d * f <= 4096 * 2 * 4096 * 14336:
            break
    c = dict(op=op, T=T, d=d, E=E, k=k, f=f, bias=rng.choice([0.0, 0.0, 4.0]))
    if op == "few":
        return dict(c, mode=rng.choice(["bf16", "fp8", "mxfp4"]))
    return dict(c, act4=rng.random() < 0.5)


# --- inputs -------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _quant_input(case, seed):
    g = _gen(seed)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    wide = _normal(g, (case["rows"], case["cols"] + case["pad"]), 0.02, dtype)
    return wide[:, : case["cols"]]


def _layer_inputs(case, seed):
    """Token rows with a few large channels, weights of standard deviation fan_in^-1/2 and a router whose bias favours
    two experts where the case says so. Tokens whose logits nearly tie among the first k + 1 are drawn again: there the
    order of the sums decides which experts a token goes to."""
    g = _gen(seed)
    T, d, E, k, f = (case[n] for n in ("T", "d", "E", "k", "f"))
    w = dict(router=_normal(g, (d, E), d**-0.5), bias=torch.zeros(E, device="cuda"),
             gate=_normal(g, (E, f, d), d**-0.5), up=_normal(g, (E, f, d), d**-0.5), down=_normal(g, (E, d, f), f**-0.5))
    w["bias"][:2] = case["bias"]
    channels = torch.ones(d, device="cuda")
    channels[torch.randperm(d, generator=g, device="cuda")[: max(1, d // 256)]] = 6.0
    x = (torch.randn((T, d), generator=g, device="cuda") * channels).bfloat16()
    for _ in range(8):
        top = torch.topk(x.double() @ w["router"].double() + w["bias"].double(), min(k + 1, E), dim=1).values
        near = ((top[:, :-1] - top[:, 1:]) < 1e-4).any(dim=1)
        if not bool(near.any()):
            break
        again = (torch.randn((T, d), generator=g, device="cuda") * channels).bfloat16()
        x = torch.where(near[:, None], again, x)
    return x, w


def prepare(case, seed):
    if case["op"] == "quant":
        return dict(case=case, x=_quant_input(case, seed))
    x, w = _layer_inputs(case, seed)
    state = dict(case=case, x=x)
    mode = case["mode"] if case["op"] == "few" else "mxfp4"
    if own:
        import sparse_moe_gemm_amd as cm

        flags = cm.FLAG_ASYNC
        if mode == "fp8":
            flags |= cm.FLAG_FP8_WEIGHTS
        if mode == "mxfp4":
            flags |= cm.FLAG_MXFP4_WEIGHTS
        if case.get("act4"):
            flags |= cm.FLAG_MXFP4_ACTIVATIONS
        state["layer"] = cm.MoELayer(w["router"], w["bias"], w["gate"], w["up"], w["down"], case["k"],
                                     max_tokens=case["T"], flags=flags)
        return state
    state.update(router=w["router"], bias=w["bias"])
    for name in ("gate", "up", "down"):
        if mode == "mxfp4":  # E2M1 values are E4M3 values too: one byte each, beside their scales
            state[name] = _mx_weights(w[name])
        elif mode == "fp8":
            state[name] = _fp8_rows(w[name])
        else:
            state[name] = (w[name], None)
    return state


# --- plain forms --------------------------------------------------------------------------------


def _mx_split(x):
    """E2M1 values and block scales of x [..., cols] in 32-bit arithmetic: the smallest power of two 2^e with the block's
    largest magnitude at most 6 * 2^e, values over 2^e rounded to nearest, ties to the even code."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(dim=-1, keepdim=True)
    m, p = torch.frexp(amax)
    e = torch.where(m <= 0.75, p - 3, p - 2)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp_(min=-127)
    u = torch.ldexp(b, -e)
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.round(u / step) * step
    return q, torch.ldexp(torch.ones_like(amax), e)


def _mx_weights(w):
    parts = [_mx_split(v) for v in w]
    return (torch.stack([q.flatten(-2).to(torch.float8_e4m3fn) for q, _ in parts]), torch.stack([s for _, s in parts]))


def _fp8_rows(w):
    """E4M3 codes of the rows and their scales: the smallest power of two 2^e with the row's largest magnitude at most
    448 * 2^e."""
    amax = w.float().abs().amax(dim=-1, keepdim=True)
    m, p = torch.frexp(amax)
    e = torch.where(m <= 0.875, p - 9, p - 8)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp_(min=-126)
    return torch.ldexp(w.float(), -e).to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(amax), e)


def _gathered(w, experts):
    """fp32 weights of the given experts [n]."""
    codes, scales = w
    if scales is None:
        return codes[experts].float()
    v = codes.view(torch.uint8)[experts].view(torch.float8_e4m3fn).float()
    s = scales[experts]
    return (v.unflatten(-1, (-1, 32)) * s).flatten(-2) if s.dim() == 4 else v * s


def _plain_layer(state):
    """The layer in 32 bits: assignments sorted by expert and cut into chunks of c rows of one expert, so that all
    chunks go through one batched product each for gate, up and down."""
    case, x = state["case"], state["x"].float()
    T, d, E, k = (case[n] for n in ("T", "d", "E", "k"))
    logits = x @ state["router"].float() + state["bias"]
    top, ids = torch.topk(logits, k, dim=1)
    weight = torch.exp(top - top[:, :1])
    weight = weight / weight.sum(dim=1, keepdim=True)
    A = T * k
    c = max(1, min(256, 1 << int(math.log2(max(1, A // E)))))
    chunks = min(E, A) + (A - min(E, A)) // c
    expert, order = torch.sort(ids.reshape(-1), stable=True)
    counts = (expert[:, None] == torch.arange(E, device=x.device)).sum(dim=0)
    per = (counts + c - 1) // c
    first = torch.cumsum(per, 0) - per  # chunk at which an expert's chunks begin
    rank = torch.arange(A, device=x.device) - (torch.cumsum(counts, 0) - counts)[expert]
    slot = first[expert] * c + rank
    owner = torch.searchsorted(torch.cumsum(per, 0), torch.arange(chunks, device=x.device), right=True).clamp_(max=E - 1)
    rows = x
    if case.get("act4"):
        q, s = _mx_split(x)
        rows = (q * s).flatten(-2)
    xc = torch.zeros(chunks * c, d, device=x.device)
    xc[slot] = rows[order // k]
    xc = xc.view(chunks, c, d)
    g = torch.bmm(xc, _gathered(state["gate"], owner).transpose(1, 2))
    u = torch.bmm(xc, _gathered(state["up"], owner).transpose(1, 2))
    h = g / (1 + torch.exp(-g)) * u
    y = torch.bmm(h, _gathered(state["down"], owner).transpose(1, 2)).view(chunks * c, d)[slot]
    by_token = torch.empty(A, d, device=x.device)
    by_token[order] = y
    return (by_token.view(T, k, d) * weight[:, :, None]).sum(dim=1).bfloat16()


def run(state):
    case, x = state["case"], state["x"]
    if own:
        if case["op"] == "quant":
            import sparse_moe_gemm_amd as cm

            codes, scales = cm.quantize_mxfp4(x)
            return cm.dequantize_mxfp4(codes, scales, x.dtype)
        return state["layer"].forward_few(x) if case["op"] == "few" else state["layer"].forward(x)
    if case["op"] == "quant":
        q, s = _mx_split(x)
        return (q * s).flatten(-2).to(x.dtype)
    return _plain_layer(state)


def work(case):
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        size = 2 if case["dtype"] == "bf16" else 4
        # the values read, codes and scales written and read back, the values they stand for written
        return {"bytes": 2 * n * size + 2 * (n // 2 + n // 32), "flops": 2 * n}
    T, d, E, k, f = (case[n] for n in ("T", "d", "E", "k", "f"))
    # experts that some token goes to, on average: with a bias of 4 on two experts they take about 93% of the
    # assignments (k = 2), the others share the rest
    if case["bias"]:
        share = (max(0, k - 2) + 0.13) / max(1, E - 2)
        active = min(2, k) + (E - 2) * (1 - (1 - min(1.0, share)) ** T)
    else:
        active = E * (1 - (1 - k / E) ** T)
    mode = case.get("mode", "mxfp4")
    per = {"bf16": 2.0, "fp8": 1.0, "mxfp4": 0.5 + 1 / 32}[mode]
    return {"bytes": active * 3 * d * f * per + d * E * 2 + 2 * T * d * 2, "flops": 2 * T * d * E + 6 * T * k * d * f}


# --- the same in 64 bits, from the definitions ----------------------------------------------------


def _mx_exact(v):
    """Values of the 4-bit codes of v [..., cols] in 64 bits: thresholds between neighbouring codes, the even code's
    side taking the tie."""
    b = v.double().reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(amax / 6.0)).clamp(min=-127))
    scale = torch.where(scale / 2 * 6 >= amax, scale / 2, scale)  # log2 may round up to the next integer ...
    scale = torch.where(scale * 6 < amax, scale * 2, scale)  # ... or down
    scale = torch.where(amax == 0, torch.ones_like(scale), scale.clamp(min=2.0**-127))
    u = b / scale
    a = u.abs()
    at = lambda t, eq: (a >= t if eq else a > t).double()  # noqa: E731
    value = 0.5 * (at(0.25, False) + at(0.75, True) + at(1.25, False) + at(1.75, True))
    value = value + at(2.5, False) + at(3.5, True) + 2 * at(5.0, False)
    return (torch.sign(u) * value * scale).reshape(v.shape)


def _fp8_exact(v):
    w = v.double()
    amax = w.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
    scale = torch.where(scale / 2 * 448 >= amax, scale / 2, scale)
    scale = torch.where(scale * 448 < amax, scale * 2, scale)
    u = w / scale
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0**-6))) - 3)
    return torch.round(u / step) * step * scale


def exact(case, seed):
    if case["op"] == "quant":
        return _mx_exact(_quant_input(case, seed))
    x, w = _layer_inputs(case, seed)
    mode = case["mode"] if case["op"] == "few" else "mxfp4"
    values = {"bf16": lambda v: v.double(), "fp8": _fp8_exact, "mxfp4": _mx_exact}[mode]
    x64 = x.double()
    logits = x64 @ w["router"].double() + w["bias"].double()
    top, ids = logits.sort(dim=1, descending=True, stable=True)
    top, ids = top[:, : case["k"]], ids[:, : case["k"]]
    share = torch.softmax(top, dim=1)
    xe = _mx_exact(x) if case.get("act4") else x64
    y = torch.zeros_like(x64)
    for e in torch.unique(ids).tolist():
        token, slot = torch.where(ids == e)
        rows = xe[token]
        g = rows @ values(w["gate"][e]).t()
        h = g * torch.sigmoid(g) * (rows @ values(w["up"][e]).t())
        y[token] += share[token, slot][:, None] * (h @ values(w["down"][e]).t())
    return y
