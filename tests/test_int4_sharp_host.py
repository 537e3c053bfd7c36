"""That the checks of int4_cases.py see what they are there for, on the CPU: results
formed with a rounding too many differ from the exact ones, or from the normal
values' bound, and plain fp32 sums do neither."""
import numpy as np
import pytest

import int4_cases
import int4_ref


def f32(v):
    return v.astype(np.float32).astype(np.float64)


def by_group(x, q, s, z, group_sum):
    """y [T][N] with group_sum on what a group adds."""
    G = s.shape[-1]
    xg, qg = x.reshape(len(x), G, -1), q.reshape(len(q), G, -1).astype(np.float64)
    zz = np.full(s.shape, 8.0) if z is None else z.astype(np.float64)
    y = np.zeros((len(x), len(q)))
    for g in range(G):
        y = f32(y + group_sum((xg[:, g] @ (qg[:, g] - zz[:, g, None]).T) * s[:, g]))
    return y


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T,k,E,N,K,group", int4_cases.EXACT)
def test_a_rounding_too_many_shows(T, k, E, N, K, group, kind):
    rng = np.random.default_rng(T + N + K)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    z = rng.integers(0, 16, (N, K // group)).astype(np.uint8)
    s = int4_cases.whole_scales(rng, (1, N, K // group), kind)[0]
    held = np.float16 if kind == "f16" else np.float64
    assert (s.astype(held) == s).all() and (kind == "f16" or (int4_ref.to_bf16(s) == s).all())
    x = int4_cases.sparse(rng, (T, K))
    want = x @ int4_ref.values(q, s, z).T
    assert (f32(want) == want).all() and (by_group(x, q, s, z, f32) == want).all()
    assert (x @ int4_ref.to_bf16(int4_ref.values(q, s, z)).T != want).any()
    assert (by_group(x, q, s, z, int4_ref.to_bf16) != want).any()
    if kind == "f16":
        assert (x @ int4_ref.values(q, int4_ref.to_bf16(s), z).T != want).any()
        flushed = np.where(s < 2.0 ** -14, 0.0, s)
        assert (x @ int4_ref.values(q, flushed, z).T != want).any()


@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("T,E,N,K,group", int4_cases.NORMAL)
def test_normal_values_bound_lies_between(T, E, N, K, group, symmetric):
    rng = np.random.default_rng(K + T)
    w = int4_ref.to_bf16(rng.normal(0, K ** -0.5, (N, K)))
    q, s, z, _ = int4_ref.quantize(w, group, symmetric)
    z = None if symmetric else z
    x = int4_ref.to_bf16(rng.normal(0, 1, (T, K)))
    want = x @ int4_ref.values(q, s, z).T

    def rms(y):
        return np.sqrt(((y - want) ** 2).mean() / (want ** 2).mean())

    # as the kernel forms it, its sums one after the other
    G = s.shape[-1]
    xg, qg = x.reshape(T, G, -1), q.reshape(N, G, -1)
    y = np.zeros((T, N), np.float32)
    for g in range(G):
        acc, ones = np.zeros((T, N), np.float32), np.zeros((T, 1), np.float32)
        for c in range(xg.shape[-1]):
            acc += (xg[:, g, c, None] * (16 + qg[None, :, g, c].astype(np.float64))).astype(np.float32)
            ones += xg[:, g, c, None].astype(np.float32)
        zz = 24.0 if z is None else 16.0 + z[:, g]
        y += (f32(acc - zz * ones.astype(np.float64)) * s[:, g]).astype(np.float32)
    assert rms(y) < int4_cases.NORMAL_RMS / 4
    assert rms(x @ int4_ref.to_bf16(int4_ref.values(q, s, z)).T) > 4 * int4_cases.NORMAL_RMS
    assert rms(by_group(x, q, s, np.full(s.shape, 8.0) if z is None else z, int4_ref.to_bf16)) > 4 * int4_cases.NORMAL_RMS
