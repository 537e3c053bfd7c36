"""The operators around the layer together, as a block's decode step runs them:
residual addition and norm, router logits, routing by a rule, gate/up and down
products of the chosen experts' 4-bit weights, the sum back into the residual
stream; eagerly and captured into one graph. Checked against 64 bits step by
step, and against a layer built from the weights read back."""
import numpy as np
import pytest

import int4_ref
import route_ref
from moe_case import TOL_Y, to_f64

pytestmark = pytest.mark.gpu

RULE = dict(scoring="sigmoid", groups=4, top_groups=2, group_score="top2", scale=1.5)


class Block:
    def __init__(self, T, d, f, E, k, group, seed):
        import torch

        import sparse_moe_gemm_amd as cm

        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.k, self.x, self.r = k, rand(T, d).bfloat16().cuda(), (3 * rand(T, d)).bfloat16().cuda()
        self.norm = (1 + 0.1 * rand(d)).bfloat16().cuda()
        self.router = (rand(d, E) * d ** -0.5).bfloat16().cuda()
        self.bias = (0.05 * rand(E)).cuda()
        self.gu = cm.quantize_int4((rand(E, 2 * f, d) * d ** -0.5).bfloat16().cuda(), group)
        self.dn = cm.quantize_int4((rand(E, d, f) * f ** -0.5).bfloat16().cuda(), group)
        self.up, self.down = cm.Int4Linear(*self.gu, swiglu=True), cm.Int4Linear(*self.dn)
        self.rule = cm.RoutingRule(**RULE)

    def step(self, x, r):
        import sparse_moe_gemm_amd as cm

        n = cm.rms_norm(x, self.norm, residual=r)
        ids, w = cm.route((n.y @ self.router).float(), self.k, self.rule, bias=self.bias)
        h = self.up.forward(n.y, ids)
        return n, ids, w, h, self.down.forward(h, ids, w)


@pytest.mark.parametrize("T,d,f,E,k,group", [(1, 256, 128, 8, 2, 128), (5, 512, 256, 16, 3, 64), (16, 2048, 768, 64, 4, 128),
                                             (32, 384, 96, 12, 4, 32)])
def test_decode_step(T, d, f, E, k, group):
    import torch

    import sparse_moe_gemm_amd as cm

    b = Block(T, d, f, E, k, group, T + d)
    n, ids, w, h, y = b.step(b.x, b.r)
    torch.cuda.synchronize()
    # each step on the outputs of the one before
    logits = to_f64((n.y @ b.router).float())
    rid, rw, tol, near = route_ref.route(logits, k, "sigmoid", 4, 2, "top2", True, 1.5, to_f64(b.bias))
    got_ids = ids.cpu().numpy()
    assert (near | (got_ids == rid).all(axis=1)).all() and (np.abs(to_f64(w) - rw) <= tol[:, None] * rw)[~near].all()

    def parts(q):
        return int4_ref.unpack(q[0].cpu().numpy()), to_f64(q[1].float()), q[2].cpu().numpy()

    hy, ht = int4_ref.swiglu(*int4_ref.assigned(to_f64(n.y), got_ids, *parts(b.gu)))
    assert (np.abs(to_f64(h) - hy) <= ht + 2.0 ** -8 * (np.abs(hy) + ht)).all()
    yy, yt = int4_ref.assigned(to_f64(h), got_ids, *parts(b.dn))
    p = to_f64(w)[:, :, None]
    want, wt = (yy * p).sum(axis=1), ((yt + k * 2.0 ** -22 * np.abs(yy)) * p).sum(axis=1)
    assert (np.abs(to_f64(y) - want) <= wt + 2.0 ** -8 * (np.abs(want) + wt)).all()
    # the same step as one graph, replayed on other rows
    src_x, src_r = b.x.clone(), b.r.clone()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.step(src_x, src_r)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = b.step(src_x, src_r)
    for i in range(4):
        src_x.copy_(torch.roll(b.x, i, 1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = b.step(src_x, src_r)
        for a, c in zip((out[0].y, out[0].residual, *out[1:]), (eager[0].y, eager[0].residual, *eager[1:])):
            assert torch.equal(a, c), i
    # a layer of the values the weights stand for, with the same rule
    if d % 128 == 0 and f % 128 == 0:
        gate, up = (v.contiguous() for v in cm.dequantize_int4(*b.gu).chunk(2, dim=1))
        layer = cm.MoELayer(b.router, None, gate, up, cm.dequantize_int4(*b.dn), k, max_tokens=T, rule=b.rule,
                            select_bias=b.bias)
        rt = layer.routing_buffers(T)
        for call in (layer.forward, layer.forward_few) if T <= cm.FEW_TOKENS else (layer.forward,):
            ly = call(n.y, routing=rt)
            same = (rt["topk_ids"] == ids).all(dim=1).cpu().numpy()
            assert same.sum() >= same.size - 1  # logits rounded to bf16 above may decide a near tie otherwise
            off = np.abs(to_f64(ly) - to_f64(y)).max(axis=1) / np.abs(to_f64(y)).max(axis=1)
            # two results of bf16 weights, rows and sums each off by the layer's own tolerance at most
            assert off[same].max() <= 2 * TOL_Y["bf16"]
        layer.close()
