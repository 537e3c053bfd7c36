// topk.hpp - selection of the k largest logits of a token and the softmax over
// them, shared by the router kernels and the layer kernels for a few tokens.
#pragma once

#include "common.hpp"

namespace cmoe {

// Monotone map of a float to an unsigned key (larger float -> larger key).
// -0 is first turned into +0 so that the two zeros tie, as they compare equal.
__device__ __forceinline__ uint32_t order_key(float f)
{
    if (f == 0.0f)
        f = 0.0f;
    uint32_t u = __float_as_uint(f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Inverse of order_key (a -0 logit comes back as +0, which compares equal).
__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// One step of the wave maximum: v and the value of the lane that the DPP
// control CTRL names (lanes outside ROW_MASK, or without a source lane, take
// 0, the smallest key).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v)
{
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false));
}

// Largest v over the wave, in a scalar register: within each row of 16 lanes
// by swaps of neighbours, of quads and of half rows, then across the rows by
// the row broadcasts of lane 15 and lane 31, so that lane 63 holds the
// maximum. (DPP moves data between lanes without an LDS round trip.)
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    v = dpp_max<0xB1, 0xF>(v);   // quad_perm [1,0,3,2]
    v = dpp_max<0x4E, 0xF>(v);   // quad_perm [2,3,0,1]
    v = dpp_max<0x141, 0xF>(v);  // row_half_mirror
    v = dpp_max<0x140, 0xF>(v);  // row_mirror: every lane holds its row's maximum
    v = dpp_max<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
    v = dpp_max<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Top-k + softmax for the block's bt tokens, reading logits (bias included)
// from LDS `lg` laid out [bt][ldl]. Wave w of W handles tokens w, w+W, ...;
// lane l holds the keys of experts l + 64q (q < NQ, NQ = ceil(E / 64) at
// most) and, once they are chosen, slot l's expert and logit (l < k), so
// that the k softmax weights are computed and stored by k lanes at once.
template <int NQ>
__device__ inline void topk_softmax_epilogue(const float* lg, int ldl, int bt, int t0, int T, int E, int k,
                                      int32_t* ids, float* wout)
{
    const int lane = threadIdx.x % kWave;
    const int wv = threadIdx.x / kWave;
    for (int r = wv; r < bt; r += (int)blockDim.x / kWave) {
        const int t = t0 + r;
        if (t >= T)
            break;
        // Order keys of the token's logits (expert e = lane + 64q); an expert
        // not present, or already taken, has key 0, below every logit's key.
        // The largest key wins; among equal keys the lowest expert index.
        uint32_t key[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int e = lane + q * kWave;
            key[q] = e < E ? order_key(lg[r * ldl + e]) : 0u;
        }
        int my_id = 0;
        float my_l = 0.0f;
        for (int j = 0; j < k; ++j) {
            uint32_t best = key[0];
#pragma unroll
            for (int q = 1; q < NQ; ++q)
                best = max(best, key[q]);
            best = wave_max_u32(best);
            int e = E - 1;
#pragma unroll
            for (int q = NQ - 1; q >= 0; --q) {
                const uint64_t m = __ballot(key[q] == best && lane + q * kWave < E);
                if (m != 0)
                    e = q * kWave + __builtin_ctzll(m);
            }
            if (lane == j) {
                my_id = e;
                my_l = key_value(best);
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if (lane + q * kWave == e)
                    key[q] = 0u;
        }
        // w_j = exp(l_j - l_0) / sum_j' exp(l_j' - l_0), the sum taken in slot
        // order (the same value in every lane).
        const float l0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_l), 0));
        const float ex = __expf(my_l - l0);
        float sum = 0.0f;
        for (int j = 0; j < k; ++j)
            sum += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ex), j));
        const float inv = 1.0f / sum;
        if (lane < k) {
            ids[(int64_t)t * k + lane] = my_id;
            wout[(int64_t)t * k + lane] = ex * inv;
        }
    }
}

__device__ inline void store_logits(const float* lg, int ldl, int bt, int t0, int T, int E, float* logits)
{
    if (!logits)
        return;
    for (int i = threadIdx.x; i < bt * E; i += (int)blockDim.x) {
        const int r = i / E, e = i % E;
        if (t0 + r < T)
            logits[(int64_t)(t0 + r) * E + e] = lg[r * ldl + e];
    }
}

}  // namespace cmoe
