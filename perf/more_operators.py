"""Cases that measure the operators around the MoE layer when a decoder block is served, beside their plain forms in
elementary torch operations:

* ``norm``: residual addition, root-mean-square norm and E4M3 rows with a power-of-two scale each (``rms_norm``);
* ``route``: router logits to expert ids and weights by softmax or sigmoid scores, a selection bias, groups of experts
  and renormalisation (``route``);
* ``int4``: products of 1 to 128 rows with 4-bit weights that have a scale and a zero point per group, dense or through
  expert ids, with SiLU(gate) * up or the weighted sum over a token's experts at the end (``Int4Linear``);
* ``codec``: bf16 weights to such 4-bit groups and back (``quantize_int4``, ``dequantize_int4``).
"""
import math

import torch

own = False  # True: the library's calls instead of the plain forms

EPS = 1e-6


def listed():
    plain = dict(bias=False, groups=1, top_groups=1, pair=False, normalize=True, scale=1.0, masked=0)
    return [
        # one sequence generating: the row before the layer, residual stream added
        dict(name="norm-1", op="norm", rows=1, cols=4096, pad=0, dtype="bf16", residual=True, fp8=False, y=True),
        # a long prompt: rows for the router (bf16) and for 8-bit expert products (codes)
        dict(name="norm-prompt-16384-fp8", op="norm", rows=16384, cols=4096, pad=0, dtype="bf16", residual=True, fp8=True,
             y=True),
        # fp32 rows that are slices of wider ones, odd row count, codes alone
        dict(name="norm-fp32-slice", op="norm", rows=1003, cols=2080, pad=36, dtype="f32", residual=False, fp8=True, y=False),
        # a decode batch over few experts: softmax of the two winners
        dict(name="route-32x8", op="route", T=32, E=8, k=2, pad=0, dtype="f32", score="softmax", **plain),
        # a long prompt over many experts in groups: sigmoid scores, balance bias, two best of each group, half the groups
        dict(name="route-16384x256-groups", op="route", T=16384, E=256, k=8, pad=0, dtype="f32", score="sigmoid", bias=True,
             groups=8, top_groups=4, pair=True, normalize=True, scale=2.5, masked=0),
        # bf16 logits (equal ones occur), odd token count, some experts masked, weights not renormalised
        dict(name="route-2047x128-bf16", op="route", T=2047, E=128, k=4, pad=0, dtype="bf16", score="softmax",
             **{**plain, "normalize": False, "scale": 1.5, "masked": 20}),
        # one token through a square projection
        dict(name="int4-dense-1", op="int4", form="dense", T=1, k=1, E=1, N=4096, K=4096, group=128, zeros=True, half=True),
        # 33 rows, ragged sizes: rows and columns that fill no tile, small groups, no zero points
        dict(name="int4-dense-33", op="int4", form="dense", T=33, k=1, E=1, N=2050, K=2080, group=32, zeros=False, half=False),
        # gate and up of 16 tokens over many small experts, SiLU product at the end
        dict(name="int4-swiglu-16", op="int4", form="swiglu", T=16, k=4, E=128, N=1536, K=2048, group=64, zeros=True,
             half=False),
        # down projections of 7 tokens on few large experts, summed with the routing weights
        dict(name="int4-down-7", op="int4", form="down", T=7, k=2, E=8, N=4096, K=14336, group=128, zeros=True, half=False),
        # one projection of one large expert, as a converter reads and writes a checkpoint
        dict(name="codec-expert-matrix", op="codec", rows=14336, cols=4096, group=128, symmetric=False),
        # a small matrix of odd height, small groups, symmetric
        dict(name="codec-small", op="codec", rows=333, cols=2080, group=32, symmetric=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "int4", "codec"])
    if op == "norm":
        cols = _log_int(rng, 8, 16384)
        rows = min(_log_int(rng, 1, 16384), 16384 * 4096 // cols // 2)
        fp8 = rng.random() < 0.5
        return dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 1, 8, 36]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.7, fp8=fp8, y=not fp8 or rng.random() < 0.5)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log_int(rng, 4, 256 // groups)
        E = groups * size
        top_groups = rng.randint(1, groups)
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, min(8, top_groups * size)),
                    pad=rng.choice([0, 0, 1, 4]), dtype=rng.choice(["f32", "f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                    pair=rng.random() < 0.5, normalize=rng.random() < 0.7, scale=rng.choice([1.0, 1.0, 2.5]),
                    masked=rng.choice([0, 0, E // 8]))
    if op == "codec":
        group = rng.choice([32, 64, 128])
        cols = group * _log_int(rng, 1, 16384 // group)
        return dict(op=op, rows=min(_log_int(rng, 1, 14336), 14336 * 4096 // cols), cols=cols, group=group,
                    symmetric=rng.random() < 0.5)
    form = rng.choice(["dense", "swiglu", "down"])
    group = rng.choice([32, 64, 128, 128])
    while True:
        K, N = group * _log_int(rng, max(1, 128 // group), 14336 // group), 2 * _log_int(rng, 16, 14336)
        E = 1 if form == "dense" else _log_int(rng, 2, 128)
        k = 1 if form == "dense" else rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 128 // k)
        if min(E, T * k) * N * K <= 8 * 4096 * 14336 and E * N * K <= 16 * 4096 * 14336:
            break
    return dict(op=op, form=form, T=T, k=k, E=E, N=N, K=K, group=group, zeros=rng.random() < 0.6, half=rng.random() < 0.4)


# --- inputs -------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _norm_inputs(case, seed):
    """Rows with a few large channels, a residual stream of larger values, weights around 1. Rows whose largest normed
    value lies next to a border between two scales are shifted away from it: there the order of the sums decides."""
    g = _gen(seed)
    rows, cols, pad = case["rows"], case["cols"], case["pad"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    channels = torch.ones(cols, device="cuda")
    channels[torch.randperm(cols, generator=g, device="cuda")[: max(1, cols // 256)]] = 6.0
    wide = torch.zeros((rows, cols + pad), dtype=dtype, device="cuda")
    x = wide[:, :cols]
    x.copy_(torch.randn((rows, cols), generator=g, device="cuda").mul_(channels))
    r = _normal(g, (rows, cols), 3.0, dtype) if case["residual"] else None
    w = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dtype)
    if case["fp8"]:
        for _ in range(4):
            v = x.float() if r is None else x.float() + r.float()
            amax = (v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * w.float()).abs().amax(1)
            m = torch.frexp(amax).mantissa
            near = (m - 0.875).abs() < 1e-5
            x.copy_(torch.where(near[:, None], torch.roll(x, 1, 1), x))
    return x, r, w


def _route_inputs(case, seed):
    """Logits of deviation 1.5, a bias of a few hundredths as balancing leaves it, masked experts at -inf. Tokens with
    scores so near each other that rounding decides between them are drawn again; equal scores stay."""
    g = _gen(seed)
    T, E, k = case["T"], case["E"], case["k"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    bias = 0.05 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
    masked = torch.randperm(E, generator=g, device="cuda")[: case["masked"]]
    wide = torch.zeros((T, E + case["pad"]), dtype=dtype, device="cuda")
    logits = wide[:, :E]
    fresh = torch.ones(T, dtype=torch.bool, device="cuda")
    for _ in range(12):
        new = torch.randn((T, E), generator=g, device="cuda").mul_(1.5).to(dtype)
        new[:, masked] = -math.inf
        logits.copy_(torch.where(fresh[:, None], new, logits))
        _, choice, group, kept = _scores64(logits, bias, case)
        fresh = _near(group, case["top_groups"]) if case["groups"] > 1 else torch.zeros_like(fresh)
        fresh |= _near(kept, k)
    return logits, bias


def _near(values, n):
    """Rows whose n + 1 largest values hold two that differ by less than 1e-5 of their size, but are not equal."""
    top = values.sort(dim=1, descending=True).values[:, : n + 1]
    a, b = top[:, :-1], top[:, 1:]
    gap = torch.where(torch.isinf(b), torch.ones_like(a), a - b)
    return ((gap > 0) & (gap < 1e-5 * a.abs().clamp(max=1.0))).any(dim=1)


def _int4_inputs(case, seed):
    """Weights of deviation fan_in^-1/2 with a few wide groups, as 4-bit groups; token rows of deviation 1 with a few
    large channels; distinct experts per token and their weights."""
    g = _gen(seed)
    E, N, K, T, k, group = (case[n] for n in ("E", "N", "K", "T", "k", "group"))
    dtype = torch.float16 if case["half"] else torch.bfloat16
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, N, K // group), dtype=dtype, device="cuda")
    zeros = torch.empty((E, N, K // group), dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = torch.randn((N, K), generator=g, device="cuda").mul_(K**-0.5)
        w = w.view(N, -1, group)
        w *= 1.0 + 2.0 * (torch.rand((N, K // group, 1), generator=g, device="cuda") < 0.02)
        q, s, z = _int4_split(w.view(N, K), group, not case["zeros"], dtype)
        codes[e], scales[e], zeros[e] = _pack(q.view(N, K)), s, z
    channels = torch.ones(K, device="cuda")
    channels[torch.randperm(K, generator=g, device="cuda")[: max(1, K // 256)]] = 6.0
    shape = (T, k, K) if case["form"] == "down" else (T, K)
    x = (torch.randn(shape, generator=g, device="cuda") * channels).bfloat16()
    ids = weights = None
    if case["form"] != "dense":
        ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.int()
    else:
        codes, scales, zeros = codes[0], scales[0], zeros[0]
    if case["form"] == "down":
        weights = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
    return codes, scales, zeros if case["zeros"] else None, x, ids, weights


def _codec_inputs(case, seed):
    g = _gen(seed)
    w = _normal(g, (case["rows"], case["cols"]), case["cols"] ** -0.5)
    w[: case["rows"] // 16, : case["group"]] = 0  # a group of zeros here and there
    return w


def _pack(q):
    """Two codes a byte, the even column in the low half."""
    q = q.to(torch.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4)


def prepare(case, seed):
    op = case["op"]
    if op == "norm":
        return dict(case=case, args=_norm_inputs(case, seed))
    if op == "route":
        state = dict(case=case, args=_route_inputs(case, seed))
        if own:
            import sparse_moe_gemm_amd as cm

            state["rule"] = cm.RoutingRule(scoring=case["score"], groups=case["groups"], top_groups=case["top_groups"],
                                           group_score="top2" if case["pair"] else "max", normalize=case["normalize"],
                                           scale=case["scale"])
        return state
    if op == "codec":
        return dict(case=case, args=(_codec_inputs(case, seed),))
    codes, scales, zeros, x, ids, weights = _int4_inputs(case, seed)
    if own:
        import sparse_moe_gemm_amd as cm

        return dict(case=case, linear=cm.Int4Linear(codes, scales, zeros, swiglu=case["form"] == "swiglu"),
                    args=(x, ids, weights))
    return dict(case=case, args=(codes, scales, zeros, x, ids, weights))


# --- plain forms --------------------------------------------------------------------------------


def _plain_norm(case, x, r, w):
    v = x.float() if r is None else x.float() + r.float()
    y = v * (1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)) * w.float()
    out = dict(y=y.to(x.dtype) if case["y"] else None, residual=None if r is None else v.to(x.dtype))
    if case["fp8"]:
        amax = y.abs().amax(dim=1, keepdim=True)
        m, p = torch.frexp(amax)
        e = torch.where(m <= 0.875, p - 9, p - 8)
        e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp_(min=-126)
        out["codes"] = torch.ldexp(y, -e).to(torch.float8_e4m3fn)
        out["scales"] = torch.ldexp(torch.ones_like(amax), e)[:, 0]
    return out


def _plain_route(case, logits, bias):
    l = logits.float()
    T, E = l.shape
    out = torch.isinf(l) & (l < 0)
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(dim=1, keepdim=True))
        s = p / p.sum(dim=1, keepdim=True)
    choice = s if bias is None else s + bias
    choice = torch.where(out, torch.full_like(choice, -math.inf), choice)
    if case["groups"] > 1:
        by = choice.view(T, case["groups"], -1)
        n = 2 if case["pair"] and by.shape[2] > 1 else 1
        best = by.sort(dim=2, descending=True).values[:, :, :n]
        rest = torch.where(torch.isinf(best), torch.zeros_like(best), best)[:, :, 1:].sum(dim=2)
        order = (best[:, :, 0] + rest).sort(dim=1, descending=True, stable=True).indices[:, : case["top_groups"]]
        keep = torch.zeros(T, case["groups"], dtype=torch.bool, device=l.device).scatter_(1, order, True)
        by = torch.where(keep[:, :, None], by.clamp(min=torch.finfo(torch.float32).min), torch.full_like(by, -math.inf))
        choice = by.view(T, E)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, : case["k"]]
    w = torch.where(out, torch.zeros_like(s), s).gather(1, ids)
    if case["normalize"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return dict(ids=ids.int(), weights=w * case["scale"])


def _int4_split(w, group, symmetric, dtype):
    """Codes 0..15 by group [..][groups][group], scales and zero points [..][groups] of w in 32-bit arithmetic."""
    b = w.float().unflatten(-1, (-1, group))
    if symmetric:
        s = (b.abs().amax(dim=-1) / 7).to(dtype)
    else:
        lo, hi = b.amin(dim=-1).clamp(max=0), b.amax(dim=-1).clamp(min=0)
        s = ((hi - lo) / 15).to(dtype)
    empty = s == 0
    s = torch.where(empty, torch.ones_like(s), s)
    wide = s.float()
    z = torch.full_like(wide, 8.0) if symmetric else torch.round(-lo / wide).clamp_(0, 15)
    q = (torch.round(b / wide[..., None]) + z[..., None]).clamp_(0, 15)
    q = torch.where(empty[..., None], z[..., None], q)
    return q, s, z.to(torch.uint8)


def _unpack(codes):
    return torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)


def _int4_values(codes, scales, zeros):
    """fp32 values of packed codes."""
    q = _unpack(codes).float().unflatten(-1, (scales.shape[-1], -1))
    z = 8.0 if zeros is None else zeros.float()[..., None]
    return ((q - z) * scales.float()[..., None]).flatten(-2)


def _plain_int4(case, codes, scales, zeros, x, ids, weights):
    x = x.float()
    if case["form"] == "dense":
        return (x @ _int4_values(codes, scales, zeros).t()).bfloat16()
    T, k, E = case["T"], case["k"], case["E"]
    flat = ids.reshape(-1).long()
    if E <= T * k:  # every expert with every row, then each assignment's
        rows = x.reshape(-1, case["K"])
        w = _int4_values(codes, scales, zeros).flatten(0, 1)
        every = (rows @ w.t()).view(-1, E, case["N"])
        at = torch.arange(T * k, device=x.device)
        y = every[at if case["form"] == "down" else at // k, flat]
    else:
        w = _int4_values(codes[flat], scales[flat], None if zeros is None else zeros[flat])
        rows = x.reshape(T * k, case["K"]) if case["form"] == "down" else x.repeat_interleave(k, dim=0)
        y = (w @ rows[:, :, None])[:, :, 0]
    y = y.view(T, k, case["N"])
    if case["form"] == "down":
        return (y * weights[:, :, None]).sum(dim=1).bfloat16()
    g, u = y.chunk(2, dim=2)
    return (g / (1.0 + torch.exp(-g)) * u).bfloat16()


def _plain_codec(case, w):
    q, s, z = _int4_split(w, case["group"], case["symmetric"], torch.bfloat16)
    values = (q - z.float()[..., None]) * s.float()[..., None]
    return dict(values=values.flatten(-2).bfloat16(), scales=s)


def run(state):
    case, args = state["case"], state["args"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "route": _plain_route, "int4": _plain_int4, "codec": _plain_codec}[op](case, *args)
    import sparse_moe_gemm_amd as cm

    if op == "norm":
        x, r, w = args
        got = cm.rms_norm(x, w, EPS, residual=r, quantize="fp8" if case["fp8"] else None, with_y=case["y"])
        out = dict(y=got.y, residual=got.residual)
        if case["fp8"]:
            out.update(codes=got.codes.view(torch.float8_e4m3fn), scales=got.scales)
        return out
    if op == "route":
        logits, bias = args
        ids, weights = cm.route(logits, case["k"], state["rule"], bias=bias)
        return dict(ids=ids, weights=weights)
    if op == "int4":
        x, ids, weights = args
        return state["linear"].forward(x, ids, weights)
    codes, scales, zeros = cm.quantize_int4(args[0], case["group"], symmetric=case["symmetric"])
    return dict(values=cm.dequantize_int4(codes, scales, zeros), scales=scales)


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        size = 2 if case["dtype"] == "bf16" else 4
        per = size * (1 + 2 * case["residual"] + case["y"]) + case["fp8"]
        return {"bytes": n * per + case["cols"] * size + 4 * case["rows"] * case["fp8"], "flops": 5 * n}
    if case["op"] == "route":
        n = case["T"] * case["E"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 8 * case["T"] * case["k"] + 4 * case["E"] * case["bias"],
                "flops": 10 * n}
    if case["op"] == "codec":
        n = case["rows"] * case["cols"]
        groups = n // case["group"]
        # values read, codes, scales and zero points written and read back, values written
        return {"bytes": 4 * n + 2 * (n // 2 + groups * (2 if case["symmetric"] else 3)), "flops": 6 * n}
    E, N, K, T, k = (case[n] for n in ("E", "N", "K", "T", "k"))
    active = E * (1 - (1 - k / E) ** T)  # experts that some token goes to, on average
    per = N * K // 2 + N * K // case["group"] * (3 if case["zeros"] else 2)
    rows = T * k if case["form"] == "down" else T
    out = T * N if case["form"] != "swiglu" else T * k * N // 2
    return {"bytes": active * per + 2 * rows * K + 2 * out + (8 * T * k if E > 1 else 0), "flops": 2 * T * k * N * K}


# --- the same in 64 bits, from the definitions ----------------------------------------------------


def _exact_norm(case, x, r, w):
    v = x.double() + (0 if r is None else r.double())
    y = v / (v.pow(2).mean(-1) + EPS).sqrt()[:, None] * w.double()
    out = dict(y=y if case["y"] else None, residual=None if r is None else v)
    if case["fp8"]:
        amax = y.abs().amax(-1)
        scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
        scale = torch.where(scale / 2 * 448 >= amax, scale / 2, scale)  # log2 may round up to the next integer ...
        scale = torch.where(scale * 448 < amax, scale * 2, scale)  # ... or down
        u = y / scale[:, None]
        step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0**-6))) - 3)
        out.update(codes=torch.round(u / step) * step, scales=scale)
    return out


def _scores64(logits, bias, case):
    """Scores, choices, group scores and the choices of the kept groups in 64 bits."""
    l = logits.double()
    T, E = l.shape
    gone = torch.isneginf(l)
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
    choice = (s if bias is None else s + bias.double()).masked_fill(gone, -math.inf)
    by = choice.reshape(T, case["groups"], E // case["groups"])
    first, at = by.max(dim=2, keepdim=True)
    group = first.squeeze(2)
    if case["pair"] and by.shape[2] > 1:
        second = by.scatter(2, at, -math.inf).amax(dim=2)
        group = group + second.masked_fill(torch.isneginf(second), 0.0)
    # a group stays where fewer than top_groups others come before it (larger, or equal with a lower index)
    index = torch.arange(case["groups"], device=l.device)
    ahead = (group[:, None, :] > group[:, :, None]) | (
        (group[:, None, :] == group[:, :, None]) & (index[None, None, :] < index[None, :, None]))
    keep = ahead.sum(dim=2) < case["top_groups"]
    lowest = torch.finfo(torch.float64).min  # a masked expert of a kept group comes before one of another group
    kept = by.clamp(min=lowest).masked_fill(~keep[:, :, None], -math.inf).reshape(T, E)
    return s.masked_fill(gone, 0.0), choice, group, kept


def _exact_route(case, logits, bias):
    s, _, _, kept = _scores64(logits, bias, case)
    ids = torch.argsort(-kept, dim=1, stable=True)[:, : case["k"]]
    w = torch.gather(s, 1, ids)
    if case["normalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return dict(ids=ids.int(), weights=w * case["scale"])


def _exact_matrix(codes, scales, zeros):
    """64-bit values of one matrix of packed codes."""
    q = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device=codes.device)
    q[:, 0::2] = (codes % 16).double()
    q[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    per = q.shape[1] // scales.shape[1]
    q -= 8 if zeros is None else zeros.double().repeat_interleave(per, dim=1)
    return q * scales.double().repeat_interleave(per, dim=1)


def _exact_int4(case, codes, scales, zeros, x, ids, weights):
    x = x.double()
    if case["form"] == "dense":
        return x @ _exact_matrix(codes, scales, zeros).t()
    y = torch.zeros((case["T"], case["k"], case["N"]), dtype=torch.float64, device=x.device)
    for e in torch.unique(ids).tolist():
        t, j = torch.where(ids == e)
        m = _exact_matrix(codes[e], scales[e], None if zeros is None else zeros[e])
        y[t, j] = (x[t, j] if case["form"] == "down" else x[t]) @ m.t()
    if case["form"] == "down":
        return (y * weights.double()[:, :, None]).sum(1)
    f = case["N"] // 2
    return y[..., :f] * torch.sigmoid(y[..., :f]) * y[..., f:]


def _exact_codec(case, w):
    b = w.double().reshape(case["rows"], -1, case["group"])
    if case["symmetric"]:
        s = b.abs().amax(-1) / 7
    else:
        lo = torch.minimum(b.amin(-1), torch.zeros((), dtype=torch.float64, device=b.device))
        s = (torch.maximum(b.amax(-1), torch.zeros_like(lo)) - lo) / 15
    # to bf16: eight significant bits, ties to even
    m, p = torch.frexp(s)
    s = torch.ldexp(torch.round(m * 256) / 256, p)
    s = torch.where(s == 0, torch.ones_like(s), s)
    z = torch.full_like(s, 8.0) if case["symmetric"] else torch.round(-lo / s).clamp(0, 15)
    steps = (torch.round(b / s[..., None])).clamp(min=-z[..., None], max=15 - z[..., None])
    return dict(values=(steps * s[..., None]).reshape(w.shape), scales=s)


def exact(case, seed):
    if case["op"] == "norm":
        return _exact_norm(case, *_norm_inputs(case, seed))
    if case["op"] == "route":
        return _exact_route(case, *_route_inputs(case, seed))
    if case["op"] == "codec":
        return _exact_codec(case, _codec_inputs(case, seed))
    return _exact_int4(case, *_int4_inputs(case, seed))
