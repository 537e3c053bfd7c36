"""4-bit microscaled rows (quantize_mxfp4, dequantize_mxfp4) and layers on 4-bit
expert weights against the plain 64-bit reference of mx_ref.py.

* Codes, scales and read-back values are exact: every tie, every scale step,
  zeros, subnormals, infinities and NaN, all bf16 bit patterns, random fp32 bit
  patterns, strided and oddly aligned rows.
* Layers: routing as the reference decides it, y within the bound mx_ref
  derives (h rounded to bf16), on both GEMM paths and for both kinds of token
  rows. 4-bit token rows are an exact function of x, so the reference quantizes
  x itself.
"""
import numpy as np
import pytest

import mx_ref
import synth
from moe_case import make_layer, run_gpu, to_dev, to_f64

pytestmark = pytest.mark.gpu

C = synth.LayerConfig


def dev_f32(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def in_range(v):
    """Products of 2^128 and more, which no fp32 (or bf16) holds, as infinities."""
    with np.errstate(over="ignore"):
        return v.astype(np.float32).astype(np.float64)


def check_quantize(t, ref64):
    import torch

    import sparse_moe_gemm_amd as cm

    codes, scales = cm.quantize_mxfp4(t)
    back = cm.dequantize_mxfp4(codes, scales, t.dtype)
    torch.cuda.synchronize()
    rc, rs = mx_ref.quantize(ref64)
    got = mx_ref.unpack(codes.cpu().numpy())
    bad = np.argwhere(scales.cpu().numpy() != rs)
    assert bad.size == 0, f"scales differ at {bad[:4].tolist()}"
    bad = np.argwhere(got != rc)
    assert bad.size == 0, f"codes differ at {bad[:4].tolist()}: {got[tuple(bad[0])]} for {ref64[tuple(bad[0])]}"
    same = np.array_equal(back.double().cpu().numpy(), in_range(mx_ref.values(rc, rs)), equal_nan=True)
    assert same, "values read back differ"


def special_rows():
    """Blocks with a probe value and a maximum that fixes the scale: all
    values of the grid and all midpoints, both signs, at several scales; then
    maxima around every scale step, zeros and tiny blocks."""
    probes = sorted({(a + b) / 2 for a, b in zip(mx_ref.E2M1, mx_ref.E2M1[1:])} | set(mx_ref.E2M1) | {2.0 ** -20})
    rows = []
    for e in (-100, -3, 0, 40, 120):
        for p in probes:
            for near in (0.0, 2.0 ** -7, -2.0 ** -7):  # a tie, and one bf16 step to either side of it
                r = np.zeros(32)
                r[5], r[6], r[30] = p * (1 + near), -p * (1 + near), 6.0
                rows.append(r * 2.0 ** e)
    for amax in (6.0, 6.03125, 5.96875, 3.0, 3.015625, 1.0, 1.5, 1.5078125, 7.96875, 8.0, 2.0 ** -126, 2.0 ** -128,
                 2.0 ** -133, 1.5 * 2.0 ** 126, 3.3e38):
        rows.append(np.linspace(-amax, amax, 32))
    rows += [np.zeros(32), -np.zeros(32)]
    bits = np.stack(rows).astype(np.float32).view(np.uint32) & np.uint32(0xFFFF0000)  # as bf16 has them
    return bits


def test_special_blocks():
    import torch

    bits = special_rows()
    v = bits.view(np.float32)
    check_quantize(to_dev((bits >> 16).astype(np.uint16)), v.astype(np.float64))
    check_quantize(dev_f32(v), v.astype(np.float64))
    # the same values with the fp32 neighbours of each tie
    up = np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(-np.inf))
    for w in up:
        w = np.where(np.abs(w) < 2.0 ** -120, v, w).astype(np.float32)
        check_quantize(dev_f32(w), w.astype(np.float64))
    torch.cuda.synchronize()


def test_all_bf16_patterns_and_random_fp32_patterns():
    rng = np.random.default_rng(11)
    allp = rng.permutation(np.arange(65536, dtype=np.uint32)).astype(np.uint16).reshape(-1, 64)
    check_quantize(to_dev(allp), mx_ref.widen(allp))
    fin = np.sort(np.arange(65536, dtype=np.uint32)[(np.arange(65536) & 0x7F80) != 0x7F80]).astype(np.uint16)
    fin = fin[: fin.size // 64 * 64].reshape(-1, 64)  # neighbours share a block: every magnitude near its scale
    check_quantize(to_dev(fin), mx_ref.widen(fin))
    bits = rng.integers(0, 1 << 32, (500, 96), dtype=np.uint64).astype(np.uint32)
    bits[:400] = (bits[:400] & 0x80FFFFFF) | 0x3F000000  # values of like magnitude
    with np.errstate(invalid="ignore"):
        check_quantize(dev_f32(bits.view(np.float32)), bits.view(np.float32).astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,ld,off", [
    (1, 32, 32, 0), (1, 32, 32, 1), (3, 64, 67, 0), (5, 2048, 2048, 0), (17, 96, 104, 8), (1003, 288, 300, 4),
    (1, 14336, 14336, 0), (257, 4096, 4096, 0), (2, 32, 1000003, 3),
])
def test_quantize_shapes_and_strides(rows, cols, ld, off, dtype):
    import torch

    g = torch.Generator(device="cpu").manual_seed(rows * 31 + cols)
    base = torch.randn(off + rows * ld, generator=g) * 0.3
    base = base.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    t = torch.as_strided(base, (rows, cols), (ld, 1), off)
    check_quantize(t, t.double().cpu().numpy())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dequantize_every_code_and_scale(dtype):
    import torch

    import sparse_moe_gemm_amd as cm

    c = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    s = np.arange(256, dtype=np.uint8)[:, None]
    out = cm.dequantize_mxfp4(torch.from_numpy(mx_ref.pack(c)).cuda(), torch.from_numpy(s).cuda(),
                              torch.bfloat16 if dtype == "bf16" else torch.float32)
    same = np.array_equal(out.double().cpu().numpy(), in_range(mx_ref.values(c, s)), equal_nan=True)
    assert same


def test_empty_tensors_and_refused_tensors():
    import torch

    import sparse_moe_gemm_amd as cm

    z = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    codes, scales = cm.quantize_mxfp4(z)
    assert codes.shape == (0, 32) and scales.shape == (0, 2)
    assert cm.dequantize_mxfp4(codes, scales).shape == (0, 64)
    w = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (w[:, ::2], w.t(), w[:, :40], w[:1].expand(4, 64)):
        with pytest.raises(ValueError):
            cm.quantize_mxfp4(bad)
    with pytest.raises(TypeError):
        cm.quantize_mxfp4(w.half())
    with pytest.raises(ValueError):
        cm.dequantize_mxfp4(*[torch.zeros(4, n, dtype=torch.uint8, device="cuda") for n in (32, 3)])


def test_quantize_on_another_stream_and_in_a_graph():
    import torch

    import sparse_moe_gemm_amd as cm

    w = torch.randn(64, 512, device="cuda").bfloat16()
    want = cm.dequantize_mxfp4(*cm.quantize_mxfp4(w)).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = cm.dequantize_mxfp4(*cm.quantize_mxfp4(w))
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        codes, scales = cm.quantize_mxfp4(w)
        out = cm.dequantize_mxfp4(codes, scales)
    for i in range(3):
        w.copy_(torch.randn(64, 512, device="cuda"))
        want = cm.dequantize_mxfp4(*cm.quantize_mxfp4(w))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"


# --- layers --------------------------------------------------------------------


CASES = [
    C("decode-small", 32, 512, 8, 2, 1024, "bf16"),
    C("one-token", 1, 128, 8, 2, 128, "bf16"),
    C("ragged-17", 17, 384, 16, 3, 384, "bf16"),
    C("single-expert", 130, 128, 1, 1, 128, "bf16"),
    C("mixtral-small", 1500, 256, 8, 2, 512, "bf16"),
    C("long-k", 300, 1152, 2, 1, 896, "bf16"),
    C("fine-grained-small", 1000, 256, 128, 4, 256, "bf16"),
    C("k8-E256", 64, 128, 256, 8, 128, "bf16"),
    C("skewed-masked-small", 2000, 256, 64, 2, 128, "bf16",
      {0: 4.0, 3: 4.0, **{e: -1.0e4 for e in range(44, 64)}}),
]


def mx_flags(act4):
    import sparse_moe_gemm_amd as cm

    return cm.FLAG_MXFP4_WEIGHTS | (cm.FLAG_MXFP4_ACTIVATIONS if act4 else 0)


_refs = {}


def reference(cfg, inp, act4):
    if (cfg.name, act4) not in _refs:
        x = mx_ref.widen(inp["x"])
        _refs[cfg.name, act4] = mx_ref.layer64(x, mx_ref.rounded(x) if act4 else x,
                                          mx_ref.layer_weights(inp, mx_ref.rounded), cfg.k, 2.0 ** -8)
    return _refs[cfg.name, act4]


@pytest.mark.parametrize("act4", [False, True], ids=["w4a16", "w4a4"])
@pytest.mark.parametrize("cfg", CASES, ids=[c.name for c in CASES])
def test_mxfp4_layer(cfg, act4):
    print(f"mxfp4 case {cfg} act4 {act4}", flush=True)
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=mx_flags(act4))
    g = run_gpu(layer, inp["x"])
    layer.close()
    print(mx_ref.check_layer(g, reference(cfg, inp, act4), cfg.name), flush=True)
    if cfg.name == "skewed-masked-small":
        assert np.all(g["expert_counts"][44:] == 0)


def test_mxfp4_layer_from_values_read_back():
    """A checkpoint's codes, read back to bf16 and given to init, make the same
    layer as the weights they came from."""
    import torch

    import sparse_moe_gemm_amd as cm

    cfg = C("from-codes", 40, 256, 8, 2, 256, "bf16")
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=mx_flags(False))
    want = run_gpu(layer, inp["x"])["y"]
    layer.close()
    w = {}
    for n in ("w_gate", "w_up", "w_down"):
        t = to_dev(inp[n])
        w[n] = cm.dequantize_mxfp4(*cm.quantize_mxfp4(t.view(-1, t.shape[-1]))).view(t.shape)
        assert not torch.equal(w[n], t)
    layer = cm.MoELayer(to_dev(inp["w_router"]), to_dev(inp["b_router"]), w["w_gate"], w["w_up"], w["w_down"], cfg.k,
                        max_tokens=cfg.T, flags=mx_flags(False))
    got = run_gpu(layer, inp["x"])["y"]
    layer.close()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("act4", [False, True], ids=["w4a16", "w4a4"])
def test_mxfp4_static_scratch_and_every_token_count(act4):
    """colibri_moe_forward_static gives forward's y bit for bit, for calls of
    one token to all of them on one handle (every tile height of the rules),
    and leaves the rows of y behind a call's tokens as they were."""
    import torch

    import sparse_moe_gemm_amd as cm

    cfg = C("counts", 900, 256, 8, 2, 384, "bf16")
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=mx_flags(act4))
    x = to_dev(inp["x"])
    ref = reference(cfg, inp, act4)
    for T in (1, 2, 31, 33, 80, 81, 161, 400, 401, 900):
        y = torch.full_like(x, 7.0)
        rt = layer.routing_buffers(T)
        assert cm.colibri_moe_forward(layer.handle, x.data_ptr(), T, y.data_ptr()) == cm.OK
        ys = layer.forward(x[:T], routing=rt, static_scratch=True)
        torch.cuda.synchronize()
        assert torch.equal(ys, y[:T]) and bool(torch.all(y[T:] == 7.0)), T
        g = dict(y=to_f64(ys), **{n: rt[n].cpu().numpy() for n in ("topk_ids", "topk_w")})
        mx_ref.check_layer(g, tuple(v[:T] for v in ref), f"T={T}")
    layer.close()


@pytest.mark.parametrize("act4", [False, True], ids=["w4a16", "w4a4"])
def test_from_a_quantized_checkpoint_to_single_tokens(act4):
    """The operators as they are used together: expert weights arrive as codes
    and scales, are read back and given to init; a prompt goes through forward,
    and each next token (made from the last y) through forward_few, on the same
    handle and without waiting. Every step is held against the 64-bit layer on
    the codes' values and, for the same tokens, forward_few against forward."""
    import torch

    import sparse_moe_gemm_amd as cm

    cfg = C("together", 75, 384, 16, 3, 256, "bf16")
    inp = synth.make_inputs(cfg)
    w64 = mx_ref.layer_weights(inp, mx_ref.rounded)
    packed = {n: cm.quantize_mxfp4(to_dev(inp[n]).view(-1, inp[n].shape[-1])) for n in ("w_gate", "w_up", "w_down")}
    wts = [cm.dequantize_mxfp4(*packed[n]).view(inp[n].shape) for n in packed]
    for n, t in zip(("gate", "up", "down"), wts):
        assert np.array_equal(to_f64(t), w64[n])  # exact in bf16
    layer = cm.MoELayer(to_dev(inp["w_router"]), to_dev(inp["b_router"]), *wts, cfg.k, max_tokens=cfg.T,
                        flags=cm.FLAG_ASYNC | mx_flags(act4))
    del wts

    def check(x, y, rt, h_eps, what):
        x = to_f64(x)
        ref = mx_ref.layer64(x, mx_ref.rounded(x) if act4 else x, w64, cfg.k, h_eps)
        g = dict(y=to_f64(y), **{n: rt[n].cpu().numpy() for n in ("topk_ids", "topk_w")})
        mx_ref.check_layer(g, ref, what)
        return ref[1]

    x = to_dev(inp["x"])
    steps = []
    rt = layer.routing_buffers(cfg.T)
    y = layer.forward(x, routing=rt)
    check(x, y, rt, 2.0 ** -8, "prompt")
    for i, T in enumerate((1, 4, 1, 16, 1)):
        xi = (x[-T:] * 0.5 + y[-T:]).contiguous()
        rt, rt2 = layer.routing_buffers(T), layer.routing_buffers(T)
        yi = layer.forward_few(xi, routing=rt)
        y2 = layer.forward(xi, routing=rt2)
        steps.append((xi, yi, rt, y2, rt2))
        y = torch.cat([y, yi])
    torch.cuda.synchronize()
    for i, (xi, yi, rt, y2, rt2) in enumerate(steps):
        assert torch.equal(rt["topk_ids"], rt2["topk_ids"]) and torch.equal(rt["topk_w"], rt2["topk_w"])
        a = check(xi, yi, rt, 2.0 ** -16, f"step {i} few")
        b = check(xi, y2, rt2, 2.0 ** -8, f"step {i} forward")
        assert np.all(np.linalg.norm(to_f64(yi) - to_f64(y2), axis=1) <= a + b)
    layer.close()


@pytest.mark.parametrize("act4", [False, True], ids=["w4a16", "w4a4"])
@pytest.mark.parametrize("T", [20, 900])
def test_mxfp4_graph_replay_matches_eager(T, act4):
    import torch

    import sparse_moe_gemm_amd as cm

    cfg = C("graph", T, 256, 8, 2, 256, "bf16")
    inp = synth.make_inputs(cfg)
    s = torch.cuda.Stream()
    layer = cm.MoELayer(to_dev(inp["w_router"]), to_dev(inp["b_router"]), to_dev(inp["w_gate"]), to_dev(inp["w_up"]),
                        to_dev(inp["w_down"]), cfg.k, max_tokens=T, flags=cm.FLAG_ASYNC | mx_flags(act4), stream=s)
    x = to_dev(inp["x"])
    flip = torch.flip(x, dims=[0]).contiguous()
    torch.cuda.synchronize()
    y = torch.empty_like(x)
    layer.forward(x, y)
    torch.cuda.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer.forward(x, y)
    for r in range(3):
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {r}"
        other = torch.empty_like(x)
        layer.forward(flip, other)
        torch.cuda.synchronize()
        assert torch.equal(torch.flip(other, dims=[0]), want)
    del graph
    layer.close()


@pytest.mark.parametrize("act4", [False, True], ids=["w4a16", "w4a4"])
def test_mxfp4_non_finite_rows_stay_in_their_token(act4):
    """A NaN or an infinity in one token's row reaches no other token."""
    cfg = C("non-finite", 70, 256, 8, 2, 256, "bf16")
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=mx_flags(act4))
    clean = run_gpu(layer, inp["x"])
    x = inp["x"].copy()
    x[11, 3], x[40, 200] = 0x7FC0, 0x7F80
    got = run_gpu(layer, x)
    layer.close()
    others = [t for t in range(cfg.T) if t not in (11, 40)]
    assert np.array_equal(got["y"][others], clean["y"][others])
    assert np.isnan(got["y"][11]).any()
