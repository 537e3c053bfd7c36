"""Plain 64-bit reference of the 4-bit microscaled format and of a layer on
given weight values, with the error a bf16/fp32 kernel may have (derived
below). Test code only; it shares nothing with the library.

Error bound of layer64, per token, in the 2-norm over the d outputs:
  * every fp32 sum of n products p_i is off by at most n * 2^-23 * sum |p_i| (the
    standard bound n * 2^-24 with a factor 2, since the order and the rounding
    inside a matrix instruction are not specified);
  * h = SiLU(g) u from off g and u: |dh| <= |dSiLU| |u| + |SiLU(g)| |du|
    + 2^-20 |h| for the exponential and the reciprocal (a few fp32 steps), with
    |SiLU'| <= 1.1;
  * h rounded with relative error h_eps (2^-8 for bf16, half a step of
    2^-7; 2^-16 for a bf16 pair);
  * down: a change dh of h moves y by at most ||W_down||_2 ||dh||_2, and the fp32
    sum is off as above;
  * the routing weights: logits off by dl change each weight by at most
    2 dl relatively, plus 2^-20 for the exponentials;
  * y rounded to bf16: at most 2^-8 ||y||.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_bytes(amax: np.ndarray) -> np.ndarray:
    """E8M0 byte of blocks with the given largest magnitudes, by search over
    all exponents."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.arange(-127, 127)
    fits = amax[..., None] <= 6.0 * np.ldexp(1.0, e)
    b = np.argmax(fits, axis=-1)  # the first that fits; byte = e + 127
    b = np.where(amax == 0, 127, b)
    return np.where(np.isfinite(amax), b, 255).astype(np.uint8)


def quantize(v: np.ndarray):
    """(codes uint8 [..., cols], one per value, scale bytes [..., cols / 32])."""
    v = np.asarray(v, dtype=np.float64)
    blocks = v.reshape(*v.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore"):
        amax = np.where(np.isfinite(blocks).all(axis=-1), np.abs(blocks).max(axis=-1), np.inf)
    sb = scale_bytes(amax)
    bad = sb == 255
    u = np.where(bad[..., None], 0.0, blocks) / np.ldexp(1.0, sb.astype(np.int64) - 127)[..., None]
    dist = np.abs(np.abs(u)[..., None] - E2M1)
    near = dist == dist.min(axis=-1, keepdims=True)
    even = near[..., ::2]
    code = np.where(even.any(axis=-1), 2 * np.argmax(even, axis=-1), np.argmax(near, axis=-1))
    code = code | (np.signbit(np.where(bad[..., None], 0.0, blocks)).astype(np.int64) << 3)
    return code.astype(np.uint8).reshape(v.shape), sb


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((*packed.shape[:-1], packed.shape[-1] * 2), dtype=np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def values(codes: np.ndarray, sb: np.ndarray) -> np.ndarray:
    """64-bit values of codes (one per value) under their scale bytes."""
    mag = E2M1[codes & 7]
    v = np.where(codes & 8, -mag, mag).reshape(*codes.shape[:-1], -1, 32)
    scale = np.where(sb == 255, np.nan, np.ldexp(1.0, sb.astype(np.int64) - 127))
    return (v * scale[..., None]).reshape(codes.shape)


def rounded(v: np.ndarray) -> np.ndarray:
    """v as the 4-bit format holds it."""
    return values(*quantize(v))


def widen(bits: np.ndarray) -> np.ndarray:
    """bf16 bit patterns to float64."""
    with np.errstate(invalid="ignore"):
        return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def layer64(x, x_ffn, w: dict, k: int, h_eps: float):
    """(y, tol, ids, weights, near) of tokens x [T][d] float64: the router reads
    x, the experts x_ffn; w holds float64 router [d][E], bias [E], gate/up
    [E][f][d], down [E][d][f]. tol [T] bounds a kernel's 2-norm error of y[t]
    (module docstring); near [T] marks tokens whose first k+1 logits nearly tie
    (relative gap 1e-5), where the choice of experts is the kernel's."""
    T, d = x.shape
    E, f = w["gate"].shape[:2]
    u = 2.0 ** -23
    logits = x @ w["router"] + w["bias"]
    order = np.argsort(-logits, axis=1, kind="stable")
    ids = order[:, :k]
    terms = np.abs(x) @ np.abs(w["router"]) + np.abs(w["bias"])
    dl = (d + 1) * u * np.take_along_axis(terms, ids, axis=1).max(axis=1)
    top = np.take_along_axis(logits, order[:, : min(k + 1, E)], axis=1)
    gap = top[:, :-1] - top[:, 1:]
    scale = np.maximum(np.abs(top[:, :-1]), np.abs(top[:, 1:]))
    near = (gap < 1e-5 * np.maximum(scale, 1e-30)).any(axis=1) if top.shape[1] > 1 else np.zeros(T, bool)
    ex = np.exp(top[:, :k] - top[:, :1])
    wt = ex / ex.sum(axis=1, keepdims=True)
    y = np.zeros((T, d))
    tol = np.zeros(T)
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        rows, a = x_ffn[t], np.abs(x_ffn[t])
        Wg, Wu, Wd = w["gate"][e], w["up"][e], w["down"][e]
        g, up = rows @ Wg.T, rows @ Wu.T
        sg = g / (1.0 + np.exp(-g))
        h = sg * up
        dg, du = d * u * (a @ np.abs(Wg).T), d * u * (a @ np.abs(Wu).T)
        dh = 1.1 * dg * np.abs(up) + (np.abs(sg) + 1.1 * dg) * du + 2.0 ** -20 * np.abs(h)
        dh = dh + h_eps * (np.abs(h) + dh)
        ye = h @ Wd.T
        norm2 = np.linalg.norm(Wd, 2)
        err = norm2 * np.linalg.norm(dh, axis=1) + f * u * np.linalg.norm(np.abs(h) @ np.abs(Wd).T, axis=1)
        we = wt[t, j]
        y[t] += we[:, None] * ye
        tol[t] += we * (err + (2 * dl[t] + 2.0 ** -20) * np.linalg.norm(ye, axis=1))
    tol = tol + 2.0 ** -8 * (np.linalg.norm(y, axis=1) + tol)
    return y, tol, ids, wt, near


def layer_weights(inp: dict, expert=lambda v: v) -> dict:
    """float64 weights of synthetic inputs, the experts' passed through expert."""
    return dict(router=widen(inp["w_router"]), bias=inp["b_router"].astype(np.float64),
                gate=expert(widen(inp["w_gate"])), up=expert(widen(inp["w_up"])), down=expert(widen(inp["w_down"])))


def check_layer(g: dict, ref, what: str = "") -> dict:
    """Assert a GPU run's ids, weights and y against layer64's answer."""
    y, tol, ids, wt, near = ref
    ok = ~near
    assert np.array_equal(g["topk_ids"][ok], ids[ok]), f"{what}: ids differ"
    assert np.abs(g["topk_w"][ok] - wt[ok]).max(initial=0.0) <= 1e-5, f"{what}: weights differ"
    err = np.linalg.norm(g["y"] - y, axis=1)
    bad = np.nonzero(ok & ~(err <= tol))[0]
    assert bad.size == 0, f"{what}: token {bad[0]} off by {err[bad[0]]:.3e}, allowed {tol[bad[0]]:.3e}"
    norm = np.linalg.norm(y, axis=1)
    rel = err[ok] / np.where(norm[ok] > 0, norm[ok], 1.0)
    return dict(max_rel=float(rel.max(initial=0.0)), allowed=float((tol / np.where(norm > 0, norm, 1)).max(initial=0.0)),
                near=int(near.sum()))
