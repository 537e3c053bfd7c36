"""A layer with a rule in every weight and token precision, without routing buffers, with
stage timing and captured. With one expert per token and weights divided by their sum,
a sigmoid rule chooses the expert of the largest logit with weight 1, as the layer without
a rule does: outputs must be equal, bit for bit, in every forward."""
import pytest

pytestmark = pytest.mark.gpu


def make(cm, rule, flags, E, d=256, f=256, max_tokens=600, k=1):
    import torch

    g = torch.Generator().manual_seed(E)
    r = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).bfloat16().cuda()  # noqa: E731
    return cm.MoELayer(r(d, E), None, r(E, f, d), r(E, f, d), r(E, d, f), k, max_tokens, flags=flags, rule=rule)


@pytest.mark.parametrize("E", [8, 130])
@pytest.mark.parametrize("mode", ["bf16", "w8", "w8a8", "w4", "w4a4"])
def test_one_expert_is_the_same_with_and_without_a_rule(mode, E):
    import torch

    import sparse_moe_gemm_amd as cm

    flags = {"bf16": 0, "w8": cm.FLAG_FP8_WEIGHTS, "w8a8": cm.FLAG_FP8_WEIGHTS | cm.FLAG_FP8_ACTIVATIONS,
             "w4": cm.FLAG_MXFP4_WEIGHTS, "w4a4": cm.FLAG_MXFP4_WEIGHTS | cm.FLAG_MXFP4_ACTIVATIONS}[mode]
    plain, ruled = make(cm, None, flags, E), make(cm, cm.RoutingRule("sigmoid"), flags, E)
    timed = make(cm, cm.RoutingRule("sigmoid"), flags | cm.FLAG_STAGE_TIMING, E)
    x = torch.randn(600, 256, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    for T in (1, 7, 16, 60, 600):
        want = plain.forward(x[:T])
        calls = [ruled.forward, timed.forward, lambda v: ruled.forward(v, static_scratch=True)]
        if T <= cm.FEW_TOKENS:
            few = plain.forward_few(x[:T])
            torch.cuda.synchronize()
            for layer in (ruled, timed):
                assert torch.equal(layer.forward_few(x[:T]), few), T
        for call in calls:
            assert torch.equal(call(x[:T]), want), T
    assert timed.stage_times()["router"] > 0
    for layer in (plain, ruled, timed):
        layer.close()


def test_captured_layers_with_a_rule():
    import torch

    import sparse_moe_gemm_amd as cm

    rule = cm.RoutingRule("sigmoid", groups=4, top_groups=2, group_score="top2", scale=2.5)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer = make(cm, rule, cm.FLAG_ASYNC, 32, k=3)
        base = torch.randn(40, 256, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
        src = base.clone()
        for T, call in ((40, layer.forward), (9, layer.forward_few)):
            call(src[:T])
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = call(src[:T])
            for n in range(4):
                src.copy_(torch.roll(base, n, 0))
                graph.replay()
                torch.cuda.synchronize()
                got = out.clone()
                assert torch.equal(got, call(src[:T])), (T, n)
                torch.cuda.synchronize()
        layer.close()
