"""Sharp checks of a bf16 layer's y, in float64 torch on any device: a lost K
step, a lost or misplaced low part of h, a missing K split fail them by a wide
margin. Test code only; it shares nothing with the library.

The final rounding is taken out exactly. Where a kernel's fp32 result is z =
y64 + e, it returns RN(z), RN the rounding to bf16. RN(z) is the bf16 number
nearest to z, so |RN(z) - z| <= |RN(y64) - z| and

    |RN(z) - y64| <= |RN(y64) - y64| + 2 |e|.

The excess max(0, |y - y64| - |RN(y64) - y64|) of every output is thus at most
2 |e|, and its 2-norm over a token's outputs is held against 2 ||e||, where ||e||
is four times the root mean square of the parts below (each an error per output
or per h; errors of different h are independent, and their signs independent of
the weights').

* A sum of n products p_i in fp32. A matrix instruction adds 16 products or more
  to the running sum, which, with products of independent signs, stays below
  ||p||_2 in the mean square. If every addition truncates, half of 2^-23 of that
  sum is lost each time, n / 16 times with one sign; if every single product
  is added with a rounding, in any order, the errors, each at most 2^-24 of the
  sum, make a random walk of n steps:

    s(n, p) = 2^-24 (n / 16 + sqrt(n)) ||p||_2.

* h = SiLU(g) u from g and u off by s: |dh| <= 1.1 dg |u| + (|SiLU(g)| + 1.1 dg)
  du + 2^-20 |h|, the last for the exponential and the reciprocal, a few fp32
  steps; |SiLU'| <= 1.1.
* h kept as a pair of bf16 (h_parts = 2): the remainder, at most 2^-8 |h| and on
  average at most half of that, is rounded by at most half a bf16 step, 2^-8 of
  itself: 2^-17 |h| more.
* h rounded to bf16 (h_parts = 1): the reference rounds its own h. The kernel's
  differs where a rounding border lies between the two, by one bf16 step of h:
  with the chance dh / step, so sqrt(dh step) in the mean square.
* Down: sqrt(sum W^2 dh^2 + s(f, W h)^2) per output.
* The kernel's own routing weights are taken as given (they are checked apart);
  the products with them and the sum over the k slots round k + 1 times.
"""
from __future__ import annotations

import torch

HALF = 2.0 ** -24  # half an fp32 step


def f64(bits, device="cpu"):
    """bf16 bit patterns (uint16 numpy) as float64."""
    return torch.from_numpy(bits.view("int16")).to(device).view(torch.bfloat16).double()


def pow2(e):
    """2^e of integers -1022 <= e <= 1023, made from its bits: torch.ldexp goes
    through a 32-bit power function, which on a GPU is off by a step for some e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def rn(v):
    """float64 rounded to bf16, ties to even, without passing through fp32
    (a double rounding)."""
    m, e = torch.frexp(v)  # v = m * 2^e, |m| in [0.5, 1)
    step = pow2((e - 8).clamp(min=-133))
    return torch.round(v / step) * step


def mx_round(v):
    """Values of the 4-bit microscaled codes of v [..., cols] float64."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, torch.where(m <= 0.75, e - 3, e - 2).clamp(min=-127), torch.zeros_like(e))
    scale = pow2(e)
    u = b / scale
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0).double())
    return (torch.round(u / step) * step * scale).flatten(-2)


def _sum_error(n, norm2):
    return HALF * (n / 16 + n ** 0.5) * norm2


def layer(x, w, ids, wt, h_parts, expert=None):
    """(y64, ||e|| [T]) of tokens x [T][d] (as the experts see them) with the given
    routing ids, wt [T][k]; w: float64 gate, up [E][f][d], down [E][d][f], or
    with expert(e) -> (gate, up, down) one expert's at a time."""
    d = x.shape[1]
    k = ids.shape[1]
    expert = expert or (lambda e: (w["gate"][e], w["up"][e], w["down"][e]))
    y = torch.zeros_like(x)
    e2 = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        t, j = torch.where(ids == e)
        rows = x[t]
        Wg, Wu, Wd = expert(e)
        f = Wg.shape[0]
        g, u = rows @ Wg.T, rows @ Wu.T
        r2 = rows * rows
        dg, du = (_sum_error(d, (r2 @ (v * v).T).sqrt()) for v in (Wg, Wu))
        sg = g * torch.sigmoid(g)
        h = sg * u
        dh = 1.1 * dg * u.abs() + (sg.abs() + 1.1 * dg) * du + 2.0 ** -20 * h.abs()
        if h_parts == 2:
            dh2 = (dh + 2.0 ** -17 * h.abs()) ** 2
        else:
            h = rn(h)
            step = pow2(torch.frexp(h)[1] - 8)
            dh2 = torch.maximum(dh * step, dh * dh)
        W2 = Wd * Wd
        ye = h @ Wd.T
        we = wt[t, j][:, None]
        y.index_add_(0, t, we * ye)
        e2.index_add_(0, t, we * we * (dh2 @ W2.T + _sum_error(f, (h * h @ W2.T).sqrt()) ** 2
                                       + ((k + 1) * HALF * ye) ** 2))
    return y, 4 * e2.sum(dim=1).sqrt()


def excess(y, y64):
    """2-norm per token of what y is off beyond the rounding of y64 to bf16."""
    own = (rn(y64) - y64).abs()
    return torch.linalg.vector_norm(((y - y64).abs() - own).clamp(min=0), dim=1)


def check(y, ref, what=""):
    """Assert y [T][d] float64 against layer's answer; returns the largest share
    of the allowance taken and the largest allowance relative to ||y||."""
    y64, e = ref
    got = excess(y, y64)
    ok = got <= 2 * e
    if not bool(ok.all()):
        t = int(torch.where(~ok)[0][0])
        raise AssertionError(f"{what}: token {t} off by {float(got[t]):.3e} beyond rounding, allowed {float(2 * e[t]):.3e}")
    norm = torch.linalg.vector_norm(y64, dim=1).clamp(min=1e-300)
    return dict(share=float((got / (2 * e).clamp(min=1e-300)).max()), allowed=float((2 * e / norm).max()))
