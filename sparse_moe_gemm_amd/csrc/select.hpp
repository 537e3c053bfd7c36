// select.hpp - a token's experts and weights under a selection rule, shared by
// the router kernels and the routing of given logits.
//
//   s_e  = sigmoid(l_e), or the softmax over all E logits
//   c_e  = s_e + b_e                      (the choice; b optional)
//   the top_groups of the groups of E / groups consecutive experts whose best
//     choice (or whose two best choices' sum) is largest stay
//   ids  = the k largest c among them, in descending order
//   w_j  = scale * s_ids[j] / sum_j' s_ids[j']   (or without the division)
// Ties go to the lower index, for groups and for experts. An expert whose
// logit is -inf or NaN (or whose choice is) is out: it is chosen only when the
// groups that stay hold fewer than k others, after them, and with weight 0.
// (Groups first, experts within them: the two-level expert topologies of
// «Colibri 是什么» (nxbn.cn) §2.3.)
#pragma once

#include "topk.hpp"

namespace cmoe {

constexpr uint32_t kOutKey = 0x007FFFFFu;  // order_key(-inf)

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROW_MASK, 0xF, false));
}

// Sum over the wave, the same bits in every lane (steps as in wave_max_u32).
__device__ __forceinline__ float wave_sum(float v)
{
    v = dpp_add<0xB1, 0xF>(v);
    v = dpp_add<0x4E, 0xF>(v);
    v = dpp_add<0x141, 0xF>(v);
    v = dpp_add<0x140, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);
    v = dpp_add<0x143, 0xC>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Lowest expert (lane + 64 q) whose key is `best`, which some lane holds.
template <int NQ>
__device__ __forceinline__ int lowest_of(const uint32_t (&key)[NQ], uint32_t best)
{
    int e = 0;
#pragma unroll
    for (int q = NQ - 1; q >= 0; --q) {
        const uint64_t m = __ballot(key[q] == best);
        if (m != 0)
            e = q * kWave + __builtin_ctzll(m);
    }
    return e;
}

template <int NQ>
__device__ __forceinline__ uint32_t largest_of(const uint32_t (&key)[NQ])
{
    uint32_t best = key[0];
#pragma unroll
    for (int q = 1; q < NQ; ++q)
        best = max(best, key[q]);
    return wave_max_u32(best);
}

// One wave selects for one token; lane l holds experts l + 64 q. logit(e)
// reads a logit (e < E).
template <int NQ, class Logit>
__device__ __forceinline__ void select_token(Logit logit, int E, int k, const SelectRule& r, int32_t* ids, float* w)
{
    const int lane = threadIdx.x % kWave;
    float s[NQ];
    uint32_t key[NQ];
    float l[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const int e = lane + q * kWave;
        const float v = e < E ? logit(e) : -INFINITY;
        l[q] = v > -INFINITY ? v : -INFINITY;  // NaN too
    }
    if (r.sigmoid) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            s[q] = 1.0f / (1.0f + expf(-l[q]));
    } else {
        uint32_t mk = 0;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            mk = max(mk, order_key(l[q]));
        const float m = key_value(wave_max_u32(mk));
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            // equal infinities count as a difference of 0
            s[q] = l[q] == -INFINITY ? 0.0f : expf(l[q] == m ? 0.0f : l[q] - m);
            sum += s[q];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            s[q] = s[q] > 0.0f ? s[q] / sum : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const int e = lane + q * kWave;
        float c = s[q];
        if (r.bias && e < E)
            c += r.bias[e];
        const bool in = l[q] > -INFINITY && c > -INFINITY;
        key[q] = in ? order_key(c) : e < E ? kOutKey : 0u;
        s[q] = in ? s[q] : 0.0f;
    }
    if (r.top_groups < r.groups) {
        const int size = E / r.groups;
        uint32_t gkey = 0;  // lane g: group g
        for (int g = 0; g < r.groups; ++g) {
            uint32_t mine[NQ];
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int e = lane + q * kWave;
                mine[q] = e >= g * size && e < (g + 1) * size ? key[q] : 0u;
            }
            const uint32_t k1 = largest_of(mine);
            float v = key_value(k1);  // -inf: the whole group is out
            if (r.pair && size > 1) {
                const int e1 = lowest_of(mine, k1);
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    if (lane + q * kWave == e1)
                        mine[q] = 0u;
                const uint32_t k2 = largest_of(mine);
                if (k2 > kOutKey)
                    v += key_value(k2);
            }
            if (lane == g)
                gkey = order_key(v);
        }
        uint64_t kept = 0;
        for (int h = 0; h < r.top_groups; ++h) {
            const uint32_t best = wave_max_u32(gkey);
            const int g = __builtin_ctzll(__ballot(gkey == best));
            kept |= 1ull << g;
            if (lane == g)
                gkey = 0u;
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int e = lane + q * kWave;
            if (e < E && !((kept >> (e / size)) & 1))
                key[q] = 0u;
        }
    }
    int my_id = 0;
    float my_s = 0.0f;
    for (int j = 0; j < k; ++j) {
        const int e = lowest_of(key, largest_of(key));
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            if (q == e / kWave)
                v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s[q]), e % kWave));
        if (lane == j) {
            my_id = e;
            my_s = v;
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            if (lane + q * kWave == e)
                key[q] = 0u;
    }
    if (r.normalize) {
        float sum = 0.0f;
        for (int j = 0; j < k; ++j)
            sum += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_s), j));
        my_s = sum > 0.0f ? my_s / sum : 0.0f;
    }
    if (lane < k) {
        ids[lane] = my_id;
        w[lane] = my_s * r.scale;
    }
}

// The block's bt tokens from LDS logits [bt][ldl] (bias of the projection
// included), a wave per token, as topk_softmax_epilogue.
template <int NQ>
__device__ inline void select_epilogue(const float* lg, int ldl, int bt, int t0, int T, int E, int k,
                                       const SelectRule& rule, int32_t* ids, float* wout)
{
    for (int r = threadIdx.x / kWave; r < bt && t0 + r < T; r += (int)blockDim.x / kWave) {
        const int64_t t = t0 + r;
        select_token<NQ>([&](int e) { return lg[r * ldl + e]; }, E, k, rule, ids + t * k, wout + t * k);
    }
}

}  // namespace cmoe
