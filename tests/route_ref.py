"""Plain 64-bit routing by a rule, token by token, sharing nothing with the
library: the definition in include/colibri_moe.h (colibri_moe_rule_t) written
out. Also which tokens the library's fp32 may decide differently.

Error of a kernel's score (in steps of 2^-24, relative): the exponential of a
correctly rounded difference d is off by |d| + 2, 1 + exp and its reciprocal
by 2, a softmax's sum over at most 256 terms (4 levels of additions in a lane,
4 across its row, each term off as above), its reciprocal and the product by
8 + 4 + |d_max|; a weight adds its own sum of at most 8 terms, a division and
the scale: 10.
Scores are therefore within (2 |d|max + 32) * 2^-24, weights within twice that."""
from __future__ import annotations

import numpy as np

STEP = 2.0 ** -24


def scores(l, scoring):
    """Scores of one token's logits [E] and whether each expert is out."""
    out = ~(l > -np.inf)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-np.where(out, 0.0, l)))
        return np.where(out, 0.0, s), out
    if out.all():
        return np.zeros_like(l), out
    m = l[~out].max()
    p = np.array([0.0 if o else 1.0 if v == m else np.exp(v - m) for v, o in zip(l, out)])
    return p / p.sum(), out


def group_score(c, pair):
    c = np.sort(c[np.isfinite(c) | (c > 0)])[::-1]
    if c.size == 0:
        return -np.inf
    return c[0] + c[1] if pair and c.size > 1 else c[0]


def best(values, n, among):
    """The n largest of values[among], ties to the lower index; and the smallest
    relative gap that decided, but for equal values."""
    order = sorted(among, key=lambda i: (-values[i], i))
    gap = np.inf
    for a, b in zip(order[:n], order[1:n + 1]):
        va, vb = values[a], values[b]
        if va != vb and np.isfinite(vb):
            gap = min(gap, (va - vb) / max(abs(va), abs(vb)))
    return order[:n], gap


def route(logits, k, scoring="softmax", groups=1, top_groups=None, group_score_="max", normalize=True, scale=1.0,
          bias=None):
    """(ids [T][k], weights [T][k], tol [T], near [T]) in float64: tol bounds a
    kernel's relative error of the weights; near marks tokens whose choice
    fp32 may make otherwise."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    top_groups = groups if top_groups is None else top_groups
    size = E // groups
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    ids, w = np.empty((T, k), np.int64), np.empty((T, k))
    tol, near = np.empty(T), np.zeros(T, bool)
    for t in range(T):
        l = logits[t]
        s, out = scores(l, scoring)
        with np.errstate(invalid="ignore"):
            c = np.where(out, -np.inf, s + b)
        bad = ~(c > -np.inf)
        c, s = np.where(bad, -np.inf, c), np.where(bad, 0.0, s)
        fin = l[np.isfinite(l)]
        span = np.ptp(fin) if fin.size and scoring == "softmax" else np.abs(fin).max() if fin.size else 0.0
        err = (2 * span + 32) * STEP
        kept = range(groups)
        if top_groups < groups:
            g = np.array([group_score(c[i * size:(i + 1) * size], group_score_ == "top2") for i in range(groups)])
            kept, gap = best(g, top_groups, range(groups))
            near[t] |= gap < 4 * err
        among = [e for e in range(E) if e // size in set(kept)]
        chosen, gap = best(c, k, among)
        near[t] |= gap < 4 * err
        ids[t] = chosen
        v = s[ids[t]]
        if normalize:
            v = v / v.sum() if v.sum() > 0 else np.zeros(k)
        w[t] = v * scale
        tol[t] = 2 * err
    return ids, w, tol, near
