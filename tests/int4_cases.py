"""Products of 4-bit integer groups whose scales use their type's whole mantissa and
whose fp32 results are exact all the same, so that a weight, a scale or a group's
sum rounded on its way to them shows.

Row n's scales are odd integers m times one power of two u: subnormals, large ones
and ordinary ones in turn (m < 2^7 for bf16 subnormals, 2^8 for other bf16, 2^10 for
fp16 subnormals, 2^11 for other fp16). A row of x holds at most four integers of
magnitude at most 3, so every partial sum of a group is an integer below 2^8, and every
sum of groups at most 4 * 3 * 15 * 2047 < 2^19 multiples of u. Weights of a token's
slots, 1/2 or 1, and their sum over at most 8 slots stay below 2^23 halves: all of it
is exact in fp32, in any order of the sums."""
from __future__ import annotations

import numpy as np

SUBNORMAL = {"bf16": (7, -133), "f16": (10, -24)}  # bits, exponent of u
LARGE = {"bf16": (8, 90), "f16": (11, 5)}
ORDINARY = {"bf16": (8, -9), "f16": (11, -12)}


def whole_scales(rng, shape, kind, ordinary=False):
    """float64 [E][N][groups] of a type; ordinary: every row of the third sort."""
    E, N, G = shape
    s = np.empty(shape)
    for n in range(N):
        bits, e = ((SUBNORMAL, LARGE, ORDINARY, ORDINARY)[n % 4] if not ordinary else ORDINARY)[kind]
        s[:, n] = np.ldexp(2.0 * rng.integers(0, 1 << (bits - 1), (E, G)) + 1, e)
    if kind == "f16" and N > 1 and not ordinary:
        s[0, 0, 0], s[0, 1, 0] = 2.0 ** -24, 65504.0  # the least and the largest
    return s


def sparse(rng, shape):
    """Rows of zeros but for up to four integers, two of them neighbours; the first
    row's last value is one of them."""
    x = np.zeros(shape)
    rows, K = x.reshape(-1, shape[-1]), shape[-1]
    for i, r in enumerate(rows):
        at = rng.integers(0, K, 3)
        at[2] = K - 1 if i == 0 else at[2]
        for c in (*at, min(at[0] + 1, K - 1)):
            r[c] = rng.choice([-3, -2, -1, 1, 2, 3])
    return x


def halves(rng, shape):
    return rng.choice([0.5, 1.0], shape)


# (T, k, E, N, K, group): every group length's form, odd sizes, few and many rows per expert
EXACT = [(1, 1, 1, 5, 64, 32), (3, 2, 4, 36, 192, 64), (16, 1, 1, 70, 1024, 256), (9, 3, 7, 50, 416, 32),
         (40, 2, 3, 64, 640, 128), (100, 1, 1, 130, 288, 32), (16, 8, 24, 48, 256, 128), (128, 1, 1, 2130, 384, 128)]


# rms error of an fp32 product of standard normal x and normal weights, over the rms of
# the results. A group of g terms sums (16 + q) x, about 24 |x| each, in at most g
# roundings of 2^-24 of a partial sum of about 24 sqrt(g) (x's signs being even);
# independent of each other they give 24 g 2^-24, the sum of x times 16 + z as much
# again; over n groups sqrt(n) times that. The results are 4 to 5 sqrt(g n). With g at
# most 128: below 2 * 24 / 4 * sqrt(128) * 2^-24 < 2^-16; the sums over at most 128 groups add less than
# sqrt(128) 2^-24. Weights or a group's sums rounded to bf16 give about 2^-10.
NORMAL_RMS = 2.0 ** -15
NORMAL = [(1, 1, 512, 4096, 128), (33, 1, 130, 2080, 32), (7, 4, 96, 14336, 128), (64, 2, 64, 1024, 64)]
