"""Layers on 4-bit weights and the few-token forward under the sharp checks of
tight_ref.py, in the cases of the other GPU tests and in longer ones: every K
split and tile order of the 4-bit GEMMs, several trips through the few-token
down kernel's register sets, and full-size layers. Every call is made twice and
must repeat itself bit for bit."""
import pytest
import torch

import synth
import tight_cases as tc
import tight_ref
from moe_case import make_layer, to_dev
from test_gpu_few import flags_of

pytestmark = pytest.mark.gpu


def call(layer, x, entry):
    rt = layer.routing_buffers(x.shape[0])
    y = getattr(layer, entry)(x, routing=rt)
    again = getattr(layer, entry)(x)
    torch.cuda.synchronize()
    assert torch.equal(y, again), "a second call differs"
    return y, rt


def check(y, rt, x, xf, w, h_parts, what, expert=None):
    """y and the routing against float64; returns tight_ref's report."""
    ids, wt = rt["topk_ids"].long(), rt["topk_w"].double()
    logits = x @ w["router"] + w["bias"]
    kth = torch.topk(logits, ids.shape[1], dim=1).values
    mine = torch.gather(logits, 1, ids)
    assert bool((mine >= kth - 1e-5 * kth.abs().clamp(min=1)).all()), what
    assert float((wt - torch.softmax(mine, dim=1)).abs().max()) <= 1e-5, what
    r = tight_ref.check(y.double(), tight_ref.layer(xf, w, ids, wt, h_parts, expert), what)
    print(what, r, flush=True)
    return r


def compute_units():
    return torch.cuda.get_device_properties(0).multi_processor_count


def run_case(cfg, mode, entry, max_tokens=None):
    print(f"{entry} case {cfg} mode {mode}", flush=True)
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=flags_of(mode), max_tokens=max_tokens)
    y, rt = call(layer, to_dev(inp["x"]), entry)
    layer.close()
    x, xf, w = tc.tokens_and_weights(inp, mode, "cuda")
    check(y, rt, x, xf, w, 2 if entry == "forward_few" else 1, f"{cfg.name} {mode}")
    return rt


def down_trips(cfg, mode, active):
    """Trips of the few-token down kernel's loop, each through its two register
    sets."""
    columns = 64 if mode.startswith("mxfp4") else 32
    units = {"b": 32, "f": 64, "m": 128}[mode[0]]
    split = max(1, min(8, compute_units() // (cfg.d // columns)))
    per_set = {"b": 4 if cfg.T <= 8 else 3, "f": 2 if cfg.T <= 8 else 1, "m": 1}[mode[0]]
    return -(-active * (cfg.f // units) // (16 * split * 2 * per_set))


@pytest.mark.parametrize("mode", tc.MODES)
@pytest.mark.parametrize("cfg", tc.FEW + tc.FEW_NARROW + tc.FEW_DEEP, ids=lambda c: c.name)
def test_few(cfg, mode):
    if mode == "fp8-rows" and min(cfg.d, cfg.f) < 256:
        pytest.skip("8-bit token rows need d and f of at least 256")
    rt = run_case(cfg, mode, "forward_few")
    if cfg in tc.FEW_DEEP[:2]:
        assert down_trips(cfg, mode, int((rt["expert_counts"] > 0).sum())) >= 2


def down_split(T, cfg):
    """K splits of the 4-bit down GEMM."""
    A = T * cfg.k
    mean = -(-A // cfg.E)
    rows = 32 if mean <= 20 else 64 if mean <= 50 else 128
    tiles = max(-(-A // rows), min(A, cfg.E)) * -(-cfg.d // 256)
    s = 1
    while s < 4 and tiles * s < 3 * compute_units() and cfg.f // (2 * s) >= 1024:
        s *= 2
    return s


SPLITS = {"split-1": 4, "split-20": 4, "split-20-odd": 2, "split-70": 4, "split-300": 4, "n-groups-1000": 2,
          "n-groups-900": 4}


@pytest.mark.parametrize("mode", ["mxfp4", "mxfp4-rows"])
@pytest.mark.parametrize("cfg", tc.LAYERS + tc.LAYERS_DEEP, ids=lambda c: c.name)
def test_4_bit_layers(cfg, mode):
    assert down_split(cfg.T, cfg) == SPLITS.get(cfg.name, 1)
    if cfg.name.startswith("n-groups"):
        assert cfg.T * cfg.k > 384 * cfg.E and 2 * cfg.f > 16 * 256
    run_case(cfg, mode, "forward")


@pytest.mark.parametrize("mode", ["mxfp4", "mxfp4-rows"])
def test_4_bit_layer_of_many_tokens_called_with_few(mode):
    """Calls of every K split on one handle made for more tokens, with forward's
    and the static scratch's working memory."""
    cfg = tc.C("many-then-few", 7000, 2048, 4, 2, 4352, "bf16")
    inp = synth.make_inputs(cfg)
    layer = make_layer(cfg, inp, flags=flags_of(mode))
    x, xf, w = tc.tokens_and_weights(inp, mode, "cuda")
    xd = to_dev(inp["x"])
    splits = set()
    for T in (7000, 1, 33, 4000, 300, 41, 7000):
        y, rt = call(layer, xd[:T], "forward")
        check(y, rt, x[:T], xf[:T], w, 1, f"T={T} {mode}")
        if T <= 300:
            assert torch.equal(layer.forward(xd[:T], static_scratch=True), y)
        splits.add(down_split(T, cfg))
    layer.close()
    assert splits == {1, 2, 4}


# --- full size ------------------------------------------------------------------


def normal(g, *shape, std=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in out.view(shape[0], -1):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * std)
    return out


class Full:
    """A layer of the given sizes on standard normal inputs made on the GPU."""

    def __init__(self, d, E, k, f, mode, max_tokens, seed=5):
        import sparse_moe_gemm_amd as cm

        g = torch.Generator(device="cuda").manual_seed(seed)
        self.mode, self.gen, self.d = mode, g, d
        self.router, self.bias = normal(g, d, E, std=d ** -0.5), torch.zeros(E, device="cuda")
        self.wt = (normal(g, E, f, d, std=d ** -0.5), normal(g, E, f, d, std=d ** -0.5),
                   normal(g, E, d, f, std=f ** -0.5))
        self.layer = cm.MoELayer(self.router, self.bias, *self.wt, k, max_tokens=max_tokens, flags=flags_of(mode))

    def rounded(self, v):
        import sparse_moe_gemm_amd as cm

        if self.mode.startswith("mxfp4"):
            return tight_ref.mx_round(v.double())
        if self.mode.startswith("fp8"):
            codes, scales = cm.quantize_fp8(v)
            return codes.view(torch.float8_e4m3fn).double() * scales.double()[:, None]
        return v.double()

    def check(self, T, entry):
        x = normal(self.gen, T, self.d)
        print(f"{entry} {T} tokens, mode {self.mode}", flush=True)
        y, rt = call(self.layer, x, entry)
        xf = self.rounded(x) if self.mode.endswith("rows") else x.double()
        check(y, rt, x.double(), xf, dict(router=self.router.double(), bias=self.bias.double()),
              2 if entry == "forward_few" else 1, f"{T} tokens {self.mode} {entry}",
              lambda e: tuple(self.rounded(v[e]) for v in self.wt))


@pytest.mark.parametrize("mode", ["mxfp4", "mxfp4-rows"])
def test_full_size_4_bit_layers(mode):
    full = Full(4096, 8, 2, 14336, mode, 4096)
    for T in (4096, 333, 32):
        full.check(T, "forward")
    full.layer.close()
    full = Full(2048, 128, 4, 768, mode, 2047)
    for T in (2047, 333):
        full.check(T, "forward")
    full.layer.close()


@pytest.mark.parametrize("mode", tc.MODES)
def test_full_size_few(mode):
    full = Full(4096, 8, 2, 14336, mode, 16)
    for T in (1, 7, 16):
        full.check(T, "forward_few")
    full.layer.close()
    full = Full(2048, 128, 4, 768, mode, 16)
    for T in (3, 16):
        full.check(T, "forward_few")
    full.layer.close()
