"""Plain 64-bit reference of 4-bit integer groups and of products with them, from
the definitions in include/colibri_moe.h; it shares nothing with the library.

Error bound of a product (product64): a group of g values is summed in fp32 as
sum (16 + q) x and sum x, each off by at most g * 2^-23 times the sum of its
terms' magnitudes (the standard bound g * 2^-24 with a factor 2, as the order and
the rounding inside a matrix instruction are not specified; at most 128 terms at
a time); s * (first - (16 + z) * second) adds 4 steps of 2^-24 of those
magnitudes, and the sum over the n groups and 16 waves (n + 16) * 2^-23 of the
groups' magnitudes, which are at most the same ones. In all
  (min(g, 128) + 4 + n + 16) * 2^-23 * sum |s| ((16 + q) + (16 + z)) |x|."""
from __future__ import annotations

import numpy as np


def to_bf16(v):
    """Nearest bf16 value, ties to even, of float64 (finite, in range)."""
    m, e = np.frexp(np.asarray(v, np.float64))
    e2 = np.maximum(e, -125)  # below: multiples of 2^-133
    return np.ldexp(np.rint(np.ldexp(np.asarray(v, np.float64), 8 - e2)), e2 - 8)


def quantize(w, group, symmetric):
    """(codes [..][K] one per value, scales float64, zeros, unsure): unsure
    marks codes whose quotient, or whose group's scale or zero point, lies so
    near a tie that fp32 may round it the other way."""
    w = np.asarray(w, np.float64)
    b = w.reshape(*w.shape[:-1], -1, group)
    bad = ~np.isfinite(b).all(axis=-1)
    with np.errstate(all="ignore"):
        clean = np.where(bad[..., None], 0.0, b)
        lo, hi = np.minimum(clean.min(axis=-1), 0), np.maximum(clean.max(axis=-1), 0)
        raw = np.maximum(hi, -lo) / 7 if symmetric else (hi - lo) / 15
        s = to_bf16(raw)
        unsure = to_bf16(raw * (1 + 2.0 ** -22)) != to_bf16(raw * (1 - 2.0 ** -22))
        empty = s == 0
        s = np.where(empty, 1.0, s)
        zq = -lo / s
        z = np.full_like(s, 8.0) if symmetric else np.clip(np.rint(zq), 0, 15)
        if not symmetric:
            unsure |= (np.abs(zq - np.floor(zq) - 0.5) < 1e-6) & (zq != np.floor(zq) + 0.5)
        u = clean / s[..., None]
        near = np.abs(u - np.floor(u) - 0.5)
        q = np.clip(np.rint(u) + z[..., None], 0, 15)
        q = np.where((bad | empty)[..., None], (8.0 if symmetric else 0.0), q)
        z = np.where(bad, 8.0 if symmetric else 0.0, z)
    unsure = (unsure & ~bad)[..., None] | ((near > 0) & (near < 1e-5))
    return (q.astype(np.uint8).reshape(w.shape), np.where(bad, np.nan, s), z.astype(np.uint8),
            np.broadcast_to(unsure, b.shape).reshape(w.shape))


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty((*packed.shape[:-1], packed.shape[-1] * 2), np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def values(codes, scales, zeros):
    """64-bit values of codes (one per value)."""
    g = codes.shape[-1] // scales.shape[-1]
    q = codes.astype(np.float64).reshape(*scales.shape, g)
    z = 8.0 if zeros is None else zeros.astype(np.float64)[..., None]
    return ((q - z) * scales[..., None]).reshape(codes.shape)


def product64(x, codes, scales, zeros):
    """(y, tol) of y = W x for x [T][K] and one matrix's codes [N][K]."""
    g = codes.shape[-1] // scales.shape[-1]
    n = scales.shape[-1]
    z = 8.0 if zeros is None else zeros.astype(np.float64)
    big = np.abs(scales) * (32 + z)
    mag = np.repeat(big, g, axis=-1) + codes * np.abs(np.repeat(scales, g, axis=-1))
    tol = (min(g, 128) + 4 + n + 16) * 2.0 ** -23 * (np.abs(x) @ mag.T)
    return x @ values(codes, scales, zeros).T, tol


def assigned(x, ids, codes, scales, zeros):
    """(y [T][k][N], tol) for x [T][K] or [T][k][K]; ids outside 0..E-1 give 0."""
    T, k = ids.shape
    E, N = codes.shape[:2]
    y, tol = np.zeros((T, k, N)), np.zeros((T, k, N))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < E:
                row = x[t, j] if x.ndim == 3 else x[t]
                a, b = product64(row[None], codes[e], scales[e], None if zeros is None else zeros[e])
                y[t, j], tol[t, j] = a[0], b[0]
    return y, tol


def swiglu(y, tol):
    """SiLU(g) * u of the two halves and its bound: |SiLU'| <= 1.1, 2^-20 of the
    result for the exponential, the division and the product."""
    f = y.shape[-1] // 2
    g, u = y[..., :f], y[..., f:]
    e = np.exp(-np.abs(g))
    s = np.where(g < 0, g * e, g) / (1 + e)
    dg, du = 1.1 * tol[..., :f], tol[..., f:]
    return s * u, dg * np.abs(u) + np.abs(s) * du + dg * du + 2.0 ** -20 * np.abs(s * u)
