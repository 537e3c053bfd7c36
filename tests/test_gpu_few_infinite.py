"""forward_few on down weights that are infinite (in bf16, or as 8-bit and 4-bit
values that round up to 2^128): y is infinite or NaN exactly where forward's is,
with the same signs. A finite h times an infinite weight is infinite, whatever
the parts are that h is kept in."""
import numpy as np
import pytest

import synth
from moe_case import make_layer, run_gpu
from test_gpu_few import MODES, flags_of, run_few

pytestmark = pytest.mark.gpu

MAX, INF = 0x7F7F, 0x7F80


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T", [1, 7, 8, 9, 16])
def test_infinite_down_weights_give_what_forward_gives(T, mode):
    print(f"infinite down weights, T {T} mode {mode}", flush=True)
    cfg = synth.LayerConfig("infinite", T, 256, 4, 2, 384, "bf16")
    inp = synth.make_inputs(cfg)
    w = inp["w_down"].copy()
    big = INF if mode == "bf16" else MAX
    for e in range(cfg.E):  # one in a row, of either sign, in every k step and 16-row group
        for o in range(3, cfg.d, 7):
            w[e, o, (37 * o + 11 * e) % cfg.f] = big | (0x8000 if o % 2 else 0)
    w[1, 10, :] = big  # a whole row: both infinities meet
    inp = dict(inp, w_down=w)
    layer = make_layer(cfg, inp, flags=flags_of(mode))
    got, ref = run_few(layer, inp["x"]), run_gpu(layer, inp["x"])
    layer.close()
    assert np.array_equal(got["topk_ids"], ref["topk_ids"])
    y, want = got["y"], ref["y"]
    assert np.isinf(want).any() and np.isfinite(want).any()
    assert np.array_equal(np.isnan(y), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(y), inf) and np.array_equal(y[inf], want[inf])
