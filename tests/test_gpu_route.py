"""route and layers with a RoutingRule against the plain 64-bit definition of
route_ref.py: ids equal on every token that fp32 cannot decide otherwise,
weights within the bound derived there. A layer's routing is what route gives
for its logits, bit for bit, in every forward."""
import itertools

import numpy as np
import pytest

import oracle
import route_ref
import synth
from moe_case import TOL_Y, to_dev, to_f64

pytestmark = pytest.mark.gpu


def run(logits, k, bias=None, **rule):
    """route's outputs for float32 logits (or a device tensor)."""
    import torch

    import sparse_moe_gemm_amd as cm

    t = logits if torch.is_tensor(logits) else torch.from_numpy(np.asarray(logits, np.float32)).cuda()
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    ids, w = cm.route(t, k, cm.RoutingRule(**rule), bias=b)
    torch.cuda.synchronize()
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    return ids.cpu().numpy(), to_f64(w)


def check(logits, k, bias=None, few_near=True, **rule):
    ids, w = run(logits, k, bias, **rule)
    ref = {("group_score_" if n == "group_score" else n): v for n, v in rule.items()}
    l64 = to_f64(logits) if not isinstance(logits, np.ndarray) else logits.astype(np.float64)
    rid, rw, tol, near = route_ref.route(l64, k, bias=bias, **ref)
    assert not few_near or near.mean() <= 0.05
    T, E = l64.shape
    assert all(len(set(r)) == k and min(r) >= 0 and max(r) < E for r in ids.tolist())
    bad = np.where(~near & (ids != rid).any(axis=1))[0]
    assert bad.size == 0, f"token {bad[0]}: {ids[bad[0]]} for {rid[bad[0]]}"
    off = np.abs(w - rw) - tol[:, None] * np.abs(rw) - 2.0 ** -140
    off[near] = 0
    assert (off <= 0).all(), f"weights off at {np.argwhere(off > 0)[:3].tolist()}"
    return ids, w


def logits_of(T, E, seed):
    return np.random.default_rng(seed).normal(0, 1.5, (T, E)).astype(np.float32)


RULES = [dict(), dict(normalize=False), dict(scoring="sigmoid", scale=2.5),
         dict(scoring="sigmoid", normalize=False, scale=0.5)]


@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 2), (9, 8), (60, 4), (64, 8), (65, 1), (128, 4), (129, 3), (200, 8),
                                 (256, 8)])
def test_plain_rules(E, k, rule):
    for bias in (None, np.random.default_rng(E).normal(0, 0.05, E).astype(np.float32)):
        check(logits_of(77, E, 10 * E + k), k, bias, **rule)


@pytest.mark.parametrize("score", ["max", "top2"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (256, 8, 1, 8), (16, 16, 3, 3), (160, 8, 3, 6), (60, 4, 2, 4),
                                            (64, 64, 8, 8), (128, 64, 5, 8), (255, 5, 2, 7), (12, 3, 1, 4), (192, 2, 1, 8),
                                            (64, 4, 2, 6), (256, 2, 1, 8), (128, 2, 1, 5), (128, 4, 3, 8), (24, 3, 2, 3),
                                            (40, 5, 3, 8), (256, 4, 1, 8), (250, 10, 7, 8)])
def test_groups(E, groups, top, k, scoring, score):
    for bias in (None, np.random.default_rng(E).normal(0, 0.05, E).astype(np.float32)):
        check(logits_of(70, E, E + top), k, bias, scoring=scoring, groups=groups, top_groups=top, group_score=score)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 1000, 33000])
def test_token_counts(T):
    l = logits_of(T, 24, T)
    ids, w = run(l, 4, scoring="sigmoid", groups=4, top_groups=2, group_score="top2")
    part = np.unique(np.linspace(0, T - 1, 200).astype(int))
    rid, rw, tol, near = route_ref.route(l[part], 4, "sigmoid", 4, 2, "top2")
    assert (near | (ids[part] == rid).all(axis=1)).all()
    assert (np.abs(w[part] - rw) <= tol[:, None] * rw)[~near].all()


def test_ties_go_to_the_lower_index():
    """Few distinct logits: equal experts and equal groups everywhere."""
    l = np.random.default_rng(5).integers(-2, 3, (300, 96)).astype(np.float32)
    for scoring, score in itertools.product(("softmax", "sigmoid"), ("max", "top2")):
        check(l, 8, scoring=scoring)
        check(l, 8, scoring=scoring, groups=12, top_groups=5, group_score=score)
    ids, w = run(np.zeros((2, 256)), 8, groups=8, top_groups=3)
    assert (ids == np.arange(8)).all() and (w == 0.125).all()
    ids, _ = run(np.array([[0.0, -0.0, 0.0, -0.0]]), 4)
    assert (ids == np.arange(4)).all()


def test_masked_experts():
    """-inf and NaN logits are out: chosen last, with weight 0; a row of them
    leaves no weight."""
    rng = np.random.default_rng(6)
    for E, k, groups, top in ((32, 4, 1, 1), (256, 8, 8, 4), (48, 6, 6, 2)):
        l = logits_of(200, E, E)
        l[rng.random(l.shape) < 0.7] = -np.inf
        l[rng.random(l.shape) < 0.1] = np.nan
        l[0], l[1], l[2] = -np.inf, np.nan, -np.inf
        l[2, 5] = 0.25
        for scoring, score, bias in itertools.product(("softmax", "sigmoid"), ("max", "top2"),
                                                      (None, rng.normal(0, 0.05, E).astype(np.float32))):
            ids, w = check(l, k, bias, few_near=False, scoring=scoring, groups=groups, top_groups=top, group_score=score)
            assert (w[:2] == 0).all() and ids[2, 0] == 5 and w[2, 0] == 1 and (w[2, 1:] == 0).all()
            out = ~(l > -np.inf)
            chosen_out = np.take_along_axis(out, ids, axis=1)
            assert (w[chosen_out] == 0).all() and np.isfinite(w).all()


def test_largest_and_infinite_logits():
    low = np.finfo(np.float32).min
    l = np.full((3, 8), low, np.float32)
    l[1, 3], l[2, 6] = 0.0, -low
    ids, w = run(l, 2)
    assert ids.tolist() == [[0, 1], [3, 0], [6, 0]] and w.tolist() == [[0.5, 0.5], [1, 0], [1, 0]]
    ids, w = run(l, 2, scoring="sigmoid")
    assert ids.tolist() == [[0, 1], [3, 0], [6, 0]] and w.tolist() == [[0, 0], [1, 0], [1, 0]]
    l = np.zeros((1, 8), np.float32)
    l[0, 2] = l[0, 5] = np.inf
    for scoring in ("softmax", "sigmoid"):
        ids, w = run(l, 2, scoring=scoring)
        assert ids.tolist() == [[2, 5]] and w.tolist() == [[0.5, 0.5]]
    # a bias that rules an expert out, or in
    b = np.zeros(8, np.float32)
    b[0], b[7] = -np.inf, np.nan
    ids, w = run(np.zeros((1, 8)), 8, bias=b, normalize=False)
    assert ids.tolist() == [[1, 2, 3, 4, 5, 6, 0, 7]] and w.tolist() == [[0.125] * 6 + [0, 0]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (7, 3), (32, 1)])
def test_strided_rows(dtype, pad, offset):
    import torch

    wide = torch.randn(65, 90 + pad + offset, generator=torch.Generator().manual_seed(pad)) * 1.5
    wide = (wide.bfloat16() if dtype == "bf16" else wide).cuda()
    check(wide[:, offset:offset + 90], 5, scoring="sigmoid", groups=9, top_groups=4, few_near=False)
    check(wide[:1, offset:offset + 90], 5)
    check(wide[:, offset:offset + 90][::2], 5)


def test_rows_past_32_bits():
    import torch

    stride = (1 << 31) + 24
    flat = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.as_strided(flat, (3, 64), (stride, 1))
    rows.copy_(torch.from_numpy(logits_of(3, 64, 1)))
    check(rows, 8, scoring="sigmoid")


def test_default_rule_is_the_layers_softmax():
    l = logits_of(500, 40, 3)
    ids, w = run(l, 4)
    rid, rw, _ = oracle.topk(l, 4)
    near = oracle.near_tie_tokens(l, 4)
    assert (near | (ids == rid).all(axis=1)).all()
    assert np.abs(w - rw)[~near].max() <= 2.0 ** -20


def test_streams_graphs_and_empty_calls():
    import torch

    import sparse_moe_gemm_amd as cm

    rule = cm.RoutingRule("sigmoid", groups=8, top_groups=3, group_score="top2")
    l = torch.randn(300, 64, device="cuda")
    b = 0.1 * torch.randn(64, device="cuda")
    want = cm.route(l, 6, rule, bias=b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = cm.route(l, 6, rule, bias=b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    src = l.clone()
    with torch.cuda.graph(graph):
        out = cm.route(src, 6, rule, bias=b)
    for r in range(4):
        src.copy_(torch.roll(l, r, 0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], torch.roll(want[0], r, 0)) and torch.equal(out[1], torch.roll(want[1], r, 0)), r
        cm.route(l, 6, rule)
    ids, w = cm.route(l[:0], 6, rule)
    assert ids.shape == (0, 6) and w.shape == (0, 6)


# --- layers -------------------------------------------------------------------------------------

C = synth.LayerConfig
LAYERS = [
    (C("rule-groups", 45, 256, 32, 4, 128, "bf16"), dict(scoring="sigmoid", groups=8, top_groups=3, group_score="top2",
                                                         scale=2.5), True),
    (C("rule-softmax", 300, 256, 40, 3, 128, "bf16"), dict(normalize=False), False),
    (C("rule-256", 70, 128, 256, 8, 128, "bf16"), dict(scoring="sigmoid", groups=8, top_groups=4, group_score="top2"), True),
    (C("rule-f32", 33, 128, 12, 2, 128, "f32"), dict(scoring="sigmoid", groups=3, top_groups=2), True),
    (C("rule-long", 4100, 128, 64, 2, 128, "bf16"), dict(scoring="sigmoid", normalize=False), True),
]


def ffn64(inp, x, ids, w):
    """Sum of the given experts' outputs in 64 bits."""
    wide = lambda a: to_f64(to_dev(a))  # noqa: E731
    g, u, dn = (wide(inp[n]) for n in ("w_gate", "w_up", "w_down"))
    xs = wide(x)
    y = np.zeros_like(xs)
    for e in np.unique(ids):
        t, j = np.where(ids == e)
        a = xs[t] @ g[e].T
        h = a / (1 + np.exp(-a)) * (xs[t] @ u[e].T)
        np.add.at(y, t, w[t, j][:, None] * (h @ dn[e].T))
    return y


@pytest.mark.parametrize("cfg,rule,biased", LAYERS, ids=[c[0].name for c in LAYERS])
def test_layers_with_a_rule(cfg, rule, biased):
    import torch

    import sparse_moe_gemm_amd as cm

    inp = synth.make_inputs(cfg)
    bias = torch.from_numpy(np.random.default_rng(9).normal(0, 0.05, cfg.E).astype(np.float32)).cuda() if biased else None
    r = cm.RoutingRule(**rule)
    layer = cm.MoELayer(*(to_dev(inp[n]) for n in ("w_router", "b_router", "w_gate", "w_up", "w_down")), cfg.k,
                        max_tokens=cfg.T, rule=r, select_bias=bias)
    kept = None if bias is None else bias.clone()
    if bias is not None:
        bias.fill_(float("nan"))  # the layer has its own copy
    x = to_dev(inp["x"])
    seen = []
    for call, n in (("forward", cfg.T), ("static", min(cfg.T, 16)), ("few", min(cfg.T, 16))):
        if call == "few" and cfg.dtype == "f32":
            continue
        xs, rt = x[:n].contiguous(), layer.routing_buffers(n)
        if call == "few":
            y = layer.forward_few(xs, routing=rt)
        else:
            y = layer.forward(xs, routing=rt, static_scratch=call == "static")
        ids, w = cm.route(rt["logits"], cfg.k, r, bias=kept)
        torch.cuda.synchronize()
        assert torch.equal(rt["topk_ids"], ids) and torch.equal(rt["topk_w"], w), call
        d = oracle.dispatch(ids.cpu().numpy(), cfg.E)
        for key, name in (("counts", "expert_counts"), ("offsets", "expert_offsets"), ("perm", "perm"), ("inv", "inv")):
            assert np.array_equal(rt[name].cpu().numpy(), d[key]), (call, name)
        ref = ffn64(inp, inp["x"][:n], ids.cpu().numpy(), to_f64(w))
        err = np.abs(to_f64(y) - ref).max(axis=1) / np.abs(ref).max(axis=1)
        assert err.max() <= TOL_Y[cfg.dtype], (call, err.max())
        seen.append({k: v[:min(n, 16) * (cfg.k if v.dim() == 1 else 1)].cpu() for k, v in rt.items()
                     if k in ("logits", "topk_ids", "topk_w")})
    for other in seen[1:]:
        assert all(torch.equal(seen[0][k], other[k]) for k in other)
    layer.close()
