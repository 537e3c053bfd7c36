"""Calls on another stream than the current one while the current stream still
has work queued on memory that is already free for it to hand out: that work's
results and the calls' are both right."""
import pytest

pytestmark = pytest.mark.gpu


class Queued:
    """Work queued on the current stream: blocks of the given tensors' sizes are
    filled, read again after other work, and given back to the allocator before
    any of it has run."""

    def __init__(self, like):
        import torch

        a = torch.randn(2048, 2048, device="cuda")
        b = torch.empty_like(a)
        torch.cuda.synchronize()
        blocks = [torch.full(t.shape, 3, dtype=t.dtype, device="cuda") for t in like]
        for _ in range(20):
            torch.mul(a, 1.5, out=b)
        self.sums = [t.double().sum() for t in blocks]
        self.sizes = [t.numel() for t in blocks]

    def check(self, what):
        assert [float(v) for v in self.sums] == [3.0 * n for n in self.sizes], what


def test_mxfp4_quantizers_on_a_given_stream():
    import torch

    import sparse_moe_gemm_amd as cm

    w = torch.randn(512, 4096, device="cuda").bfloat16()
    want_c, want_s = cm.quantize_mxfp4(w)
    want_v = cm.dequantize_mxfp4(want_c, want_s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for r in range(4):
        queued = Queued((want_c, want_s, want_v))
        codes, scales = cm.quantize_mxfp4(w, stream=side)
        values = cm.dequantize_mxfp4(codes, scales, stream=side)
        torch.cuda.synchronize()
        queued.check(r)
        assert torch.equal(codes, want_c) and torch.equal(scales, want_s) and torch.equal(values, want_v), r


def test_fp8_quantizer_on_a_given_stream():
    import torch

    import sparse_moe_gemm_amd as cm

    w = torch.randn(512, 4096, device="cuda").bfloat16()
    want_c, want_s = cm.quantize_fp8(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for r in range(4):
        queued = Queued((want_c, want_s))
        codes, scales = cm.quantize_fp8(w, stream=side)
        torch.cuda.synchronize()
        queued.check(r)
        assert torch.equal(codes, want_c) and torch.equal(scales, want_s), r


@pytest.mark.parametrize("entry", ["forward", "forward_few"])
def test_layer_of_another_stream(entry):
    import torch

    import sparse_moe_gemm_amd as cm
    import synth
    from moe_case import to_dev

    cfg = synth.LayerConfig("other-stream", 16, 512, 8, 2, 512, "bf16")
    inp = synth.make_inputs(cfg)
    layer = cm.MoELayer(to_dev(inp["w_router"]), to_dev(inp["b_router"]), to_dev(inp["w_gate"]), to_dev(inp["w_up"]),
                        to_dev(inp["w_down"]), cfg.k, max_tokens=16, flags=cm.FLAG_ASYNC, stream=torch.cuda.Stream())
    x = to_dev(inp["x"])
    torch.cuda.synchronize()
    want = getattr(layer, entry)(x, torch.empty_like(x))
    torch.cuda.synchronize()
    for r in range(4):
        queued = Queued((x,))
        y = getattr(layer, entry)(x)
        torch.cuda.synchronize()
        queued.check(r)
        assert torch.equal(y, want), r
    layer.close()
