"""forward_few (the layer for at most 16 tokens in two kernels) against the
plain 64-bit reference of mx_ref.py, for bf16, 8-bit and 4-bit weights with and
without quantized token rows, and against forward: every routing output bit for
bit. y within the bound mx_ref derives, with h kept as a pair of bf16
(relative 2^-16)."""
import numpy as np
import pytest

import mx_ref
import oracle
import synth
from moe_case import make_layer, run_gpu, to_dev, to_f64

pytestmark = pytest.mark.gpu

C = synth.LayerConfig
H_EPS = 2.0 ** -16

MODES = ["bf16", "fp8", "fp8-rows", "mxfp4", "mxfp4-rows"]


def flags_of(mode):
    import sparse_moe_gemm_amd as cm

    return {"bf16": 0, "fp8": cm.FLAG_FP8_WEIGHTS, "fp8-rows": cm.FLAG_FP8_WEIGHTS | cm.FLAG_FP8_ACTIVATIONS,
            "mxfp4": cm.FLAG_MXFP4_WEIGHTS, "mxfp4-rows": cm.FLAG_MXFP4_WEIGHTS | cm.FLAG_MXFP4_ACTIVATIONS}[mode]


def reference(inp, k, mode):
    x = mx_ref.widen(inp["x"])
    xf = x
    if mode == "bf16":
        w = mx_ref.layer_weights(inp)
    elif mode.startswith("fp8"):
        w = mx_ref.layer_weights(oracle.quantized_expert_weights(inp))
        if mode == "fp8-rows":
            xf = mx_ref.widen(oracle.dequantize_fp8(*oracle.quantize_fp8(inp["x"])))
    else:
        w = mx_ref.layer_weights(inp, mx_ref.rounded)
        if mode == "mxfp4-rows":
            xf = mx_ref.rounded(x)
    return mx_ref.layer64(x, xf, w, k, H_EPS)


def run_few(layer, x, full=True):
    import torch

    rt = layer.routing_buffers(x.shape[0]) if full else None
    y = layer.forward_few(to_dev(x), routing=rt)
    torch.cuda.synchronize()
    out = {n: v.cpu().numpy() for n, v in (rt or {}).items()}
    out["y"] = to_f64(y)
    return out


CASES = [
    C("sixteen", 16, 512, 8, 2, 1024, "bf16"),
    C("one", 1, 256, 8, 2, 256, "bf16"),
    C("three-k3", 3, 384, 16, 3, 384, "bf16"),
    C("many-experts", 16, 256, 128, 4, 256, "bf16"),
    C("odd-experts", 7, 640, 37, 5, 384, "bf16"),
    C("one-expert", 9, 256, 1, 1, 256, "bf16"),
    C("router-apart", 16, 256, 256, 8, 256, "bf16"),
    C("router-apart-130", 2, 384, 130, 8, 256, "bf16"),
    C("wide-tokens", 5, 4608, 3, 2, 256, "bf16"),
    C("d4096", 13, 4096, 4, 2, 256, "bf16"),
    C("d2176", 2, 2176, 4, 1, 640, "bf16"),
    C("skewed", 16, 256, 64, 2, 256, "bf16", {0: 4.0, 3: 4.0, **{e: -1.0e4 for e in range(44, 64)}}),
]
NARROW = [C("narrow-1", 1, 128, 8, 2, 128, "bf16"), C("narrow-16", 16, 128, 40, 8, 128, "bf16")]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("cfg", CASES, ids=[c.name for c in CASES])
def test_few_matches_reference_and_routes_as_forward(cfg, mode):
    print(f"few case {cfg} mode {mode}", flush=True)
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=flags_of(mode))
    got = run_few(layer, inp["x"])
    plain = run_few(layer, inp["x"], full=False)
    ref = run_gpu(layer, inp["x"])
    layer.close()
    for key in ref:
        if key != "y":
            assert np.array_equal(got[key], ref[key]), key
    assert np.array_equal(plain["y"], got["y"])
    print(mx_ref.check_layer(got, reference(inp, cfg.k, mode), cfg.name), flush=True)


@pytest.mark.parametrize("mode", ["bf16", "fp8", "mxfp4", "mxfp4-rows"])
@pytest.mark.parametrize("cfg", NARROW, ids=[c.name for c in NARROW])
def test_few_narrow_layers(cfg, mode):
    test_few_matches_reference_and_routes_as_forward(cfg, mode)


@pytest.mark.parametrize("mode", MODES)
def test_few_every_token_count(mode):
    """Calls of 1 to 16 tokens on one handle, each token within its bound."""
    cfg = C("counts", 16, 512, 12, 3, 384, "bf16")
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=flags_of(mode))
    ref = reference(inp, cfg.k, mode)
    for T in range(1, 17):
        got = run_few(layer, inp["x"][:T])
        mx_ref.check_layer(got, tuple(v[:T] for v in ref), f"T={T}")
    layer.close()


def test_few_refusals():
    import torch

    import sparse_moe_gemm_amd as cm

    cfg = C("refuse", 40, 256, 8, 2, 256, "bf16")
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp)
    x = to_dev(inp["x"])
    y = torch.full_like(x, 7.0)
    assert cm.colibri_moe_forward_few(layer.handle, x.data_ptr(), 17, y.data_ptr()) == cm.ERR_TOO_LARGE
    assert cm.colibri_moe_forward_few(layer.handle, x.data_ptr(), 41, y.data_ptr()) == cm.ERR_INVALID_ARG
    assert cm.colibri_moe_forward_few(layer.handle, x.data_ptr(), -1, y.data_ptr()) == cm.ERR_INVALID_ARG
    assert cm.colibri_moe_forward_few(layer.handle, x.data_ptr(), 0, y.data_ptr()) == cm.OK
    assert cm.colibri_moe_forward_few(layer.handle, 0, 4, y.data_ptr()) == cm.ERR_INVALID_ARG
    assert cm.colibri_moe_forward_few(layer.handle, x.data_ptr() + 2, 4, y.data_ptr()) == cm.ERR_ALIGNMENT
    with pytest.raises(TypeError):
        layer.forward_few(x[:4].float())
    torch.cuda.synchronize()
    assert bool(torch.all(y == 7.0)), "a refused call wrote y"
    # rows behind the call's tokens stay as they were
    assert cm.colibri_moe_forward_few(layer.handle, x.data_ptr(), 5, y.data_ptr()) == cm.OK
    torch.cuda.synchronize()
    assert bool(torch.all(y[5:] == 7.0)) and bool(torch.all(y[:5] != 7.0))
    layer.close()
    cfg = synth.CONFIGS["tiny-f32"]
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp)
    with pytest.raises(cm.ColibriError) as ei:
        layer.forward_few(to_dev(inp["x"][:4]))
    assert ei.value.status == cm.ERR_UNSUPPORTED
    layer.close()


@pytest.mark.parametrize("mode", MODES)
def test_few_non_finite_values_stay_where_they_belong(mode):
    """A token's NaN or infinity reaches no other token, and the NaN weights of
    an expert reach only the tokens that chose it."""
    cfg = C("non-finite", 16, 256, 8, 2, 256, "bf16")
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=flags_of(mode))
    clean = run_few(layer, inp["x"])
    x = inp["x"].copy()
    x[3, 7], x[9, 100] = 0x7FC0, 0x7F80
    got = run_few(layer, x)
    layer.close()
    others = [t for t in range(16) if t not in (3, 9)]
    assert np.array_equal(got["y"][others], clean["y"][others])
    assert np.isnan(got["y"][3]).any()
    if mode.startswith("fp8"):
        return  # a row scale of an infinite row is not defined
    bad = int(clean["topk_ids"][0, 0])
    for name in ("w_gate", "w_down"):
        broken = dict(inp)
        broken[name] = inp[name].copy()
        broken[name][bad, 5, 40] = 0x7FC0
        broken[name][bad, 6, 41] = 0x7F80
        layer = make_layer(cfg, broken, flags=flags_of(mode))
        got = run_few(layer, inp["x"])
        layer.close()
        chose = (clean["topk_ids"] == bad).any(axis=1)
        assert chose.any() and not chose.all()
        assert np.array_equal(got["y"][~chose], clean["y"][~chose]), name
        assert np.isnan(got["y"][chose]).any(axis=1).all(), name


@pytest.mark.parametrize("mode", ["bf16", "mxfp4-rows"])
def test_few_graph_replay_matches_eager(mode):
    import torch

    import sparse_moe_gemm_amd as cm

    cfg = C("graph", 16, 512, 8, 2, 512, "bf16")
    inp = synth.make_inputs(cfg)
    s = torch.cuda.Stream()
    layer = cm.MoELayer(to_dev(inp["w_router"]), to_dev(inp["b_router"]), to_dev(inp["w_gate"]), to_dev(inp["w_up"]),
                        to_dev(inp["w_down"]), cfg.k, max_tokens=64, flags=cm.FLAG_ASYNC | flags_of(mode), stream=s)
    x = to_dev(inp["x"])
    flip = torch.flip(x, dims=[0]).contiguous()
    torch.cuda.synchronize()
    y, other = torch.empty_like(x), torch.empty_like(x)
    layer.forward_few(x, y)
    torch.cuda.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer.forward_few(x, y)
    for r in range(4):
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {r}"
        layer.forward_few(flip, other)  # eager work on the same handle between the replays
        layer.forward(flip, other)
        torch.cuda.synchronize()
    x.copy_(flip)  # new contents under the captured pointers
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(torch.flip(y, dims=[0]), want)
    del graph
    layer.close()


def test_few_on_two_streams_and_beside_forward():
    """Two handles queued on two streams before either finishes, few-token calls
    and general ones in turn, give each handle's results alone."""
    import torch

    import sparse_moe_gemm_amd as cm

    hs = []
    for i, mode in enumerate(("bf16", "mxfp4")):
        cfg = C(f"streams-{i}", 16, 512, 16, 4, 512, "bf16", seed=i)
        inp = synth.make_inputs(cfg)
        s = torch.cuda.Stream()
        layer = cm.MoELayer(to_dev(inp["w_router"]), to_dev(inp["b_router"]), to_dev(inp["w_gate"]),
                            to_dev(inp["w_up"]), to_dev(inp["w_down"]), cfg.k, max_tokens=16,
                            flags=cm.FLAG_ASYNC | flags_of(mode), stream=s)
        x = to_dev(inp["x"])
        torch.cuda.synchronize()
        few, gen = torch.empty_like(x), torch.empty_like(x)
        layer.forward_few(x, few)
        layer.forward(x, gen)
        torch.cuda.synchronize()
        hs.append((layer, x, few, gen))
    outs = []
    for r in range(6):
        for layer, x, few, gen in hs:
            y = torch.empty_like(x)
            (layer.forward_few if r % 3 else layer.forward)(x, y)
            outs.append((y, few if r % 3 else gen))
    torch.cuda.synchronize()
    for i, (y, want) in enumerate(outs):
        assert torch.equal(y, want), i
    for h in hs:
        h[0].close()


@pytest.mark.parametrize("E", [24, 200])
def test_few_writes_only_the_routing_outputs_asked_for(E):
    """Each routing output alone, and each left out, as in a call that asks for
    all of them."""
    import torch

    cfg = C("partial", 9, 256, E, 3, 256, "bf16")
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp)
    x = to_dev(inp["x"])
    full = layer.routing_buffers(9)
    want = layer.forward_few(x, routing=full)
    for name in full:
        for keys in ([name], [n for n in full if n != name]):
            rt = {n: torch.full_like(full[n], -5) for n in keys}
            y = layer.forward_few(x, routing=rt)
            torch.cuda.synchronize()
            assert torch.equal(y, want), keys
            for n in keys:
                assert torch.equal(rt[n], full[n]), (n, keys)
    layer.close()


def test_few_stage_times():
    import sparse_moe_gemm_amd as cm

    cfg = C("timed", 4, 256, 200, 2, 256, "bf16")
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=cm.FLAG_STAGE_TIMING)
    layer.forward_few(to_dev(inp["x"]))
    t = layer.stage_times()
    layer.close()
    assert set(t) == set(cm.STAGES) and t["gate_up_gemm"] > 0 and t["down_gemm"] > 0 and t["router"] > 0
