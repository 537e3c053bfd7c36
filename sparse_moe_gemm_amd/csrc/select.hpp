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
//
// Sixteen lanes (a DPP row) serve one token, lane r holding the experts
// r * NQ .. r * NQ + NQ - 1 in registers, so that a wave selects for four tokens at
// once and a reduction over a token is four steps within the row. Instruction
// issue bounds it: 16384 tokens, 256 experts, 8 of them in 4 of 8 groups took
// 30 us with a wave per token and take 13 us so (reading the logits: 3.3 us); 2047
// tokens of 128 experts 3.9 us, 32 of 8 3.0 us. In a layer's router, whose waves that have
// no token of their own repeat the last one's selection, a rule adds 4 us to a
// call of 1 to 1024 tokens on 128 experts (11.6 -> 15.4 us for one token), 1.6 at 4096.
#pragma once

#include "topk.hpp"

namespace cmoe {

constexpr uint32_t kOutKey = 0x007FFFFFu;  // order_key(-inf)
constexpr int kRow = 16;                   // lanes of a token

template <int CTRL>
__device__ __forceinline__ uint32_t row_move(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// Steps of a reduction over the 16 lanes of a row, after which each of them
// holds the result.
template <class F>
__device__ __forceinline__ void row_steps(F step)
{
    step(std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
    step(std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
    step(std::integral_constant<int, 0x141>{});  // row_half_mirror
    step(std::integral_constant<int, 0x140>{});  // row_mirror
}

__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    row_steps([&](auto c) { v = max(v, row_move<c()>(v)); });
    return v;
}

__device__ __forceinline__ uint32_t row_or(uint32_t v)
{
    row_steps([&](auto c) { v |= row_move<c()>(v); });
    return v;
}

__device__ __forceinline__ float row_sum(float v)
{
    row_steps([&](auto c) { v += __uint_as_float(row_move<c()>(__float_as_uint(v))); });
    return v;
}

// First lane of the row where p holds, 0..15, or 16.
__device__ __forceinline__ int row_first(bool p)
{
    const uint32_t m = (uint32_t)(__ballot(p) >> (threadIdx.x % kWave & ~(kRow - 1))) & 0xFFFFu;
    return __builtin_ctz(m | 0x10000u);
}

// The two largest keys of a lane, a row part, a row: n1 >= n2.
struct Two {
    uint32_t n1 = 0, n2 = 0;
    __device__ __forceinline__ void add(uint32_t x)
    {
        n2 = max(n2, min(n1, x));
        n1 = max(n1, x);
    }
    template <int CTRL>
    __device__ __forceinline__ void join()
    {
        const uint32_t o1 = row_move<CTRL>(n1), o2 = row_move<CTRL>(n2);
        n2 = max(max(n2, o2), min(n1, o1));
        n1 = max(n1, o1);
    }
    // What a group whose choices these are counts as.
    __device__ __forceinline__ uint32_t group_key(bool pair) const
    {
        return pair && n2 > kOutKey ? order_key(key_value(n1) + key_value(n2)) : n1;
    }
};

// Zeroes the keys of the experts whose group doesn't stay.
template <int NQ>
__device__ __forceinline__ void keep_groups(uint32_t (&key)[NQ], int E, const SelectRule& r)
{
    const int lane = threadIdx.x % kRow;
    const int size = E / r.groups;
    const int lanes = size / NQ;
    if (lanes * NQ == size && (lanes & (lanes - 1)) == 0) {
        // A group is 1, 2, 4 or 8 neighbouring lanes: all groups at once.
        Two t;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            t.add(key[q]);
        if (lanes > 1)
            t.join<0xB1>();
        if (lanes > 2)
            t.join<0x4E>();
        if (lanes > 4)
            t.join<0x141>();
        uint32_t gkey = lane * NQ < E ? t.group_key(r.pair) : 0u;
        bool kept = false;
        for (int h = 0; h < r.top_groups; ++h) {
            const int first = row_first(gkey == row_max(gkey));
            if (lane >= first && lane < first + lanes) {
                kept = true;
                gkey = 0u;
            }
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            key[q] = kept ? key[q] : 0u;
        return;
    }
    // Groups that end within a lane: one after the other.
    uint32_t gkey[4] = {};  // groups lane + 16 i
    for (int g = 0; g < r.groups; ++g) {
        Two t;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            t.add((unsigned)(lane * NQ + q - g * size) < (unsigned)size ? key[q] : 0u);
        t.join<0xB1>();
        t.join<0x4E>();
        t.join<0x141>();
        t.join<0x140>();
        const uint32_t v = t.group_key(r.pair);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (g == lane + i * kRow)
                gkey[i] = v;
    }
    uint64_t kept = 0;
    for (int h = 0; h < r.top_groups; ++h) {
        const uint32_t best = row_max(max(max(gkey[0], gkey[1]), max(gkey[2], gkey[3])));
        int g = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = row_first(gkey[i] == best);
            if (g < 0 && f < kRow)
                g = f + i * kRow;
        }
        kept |= 1ull << g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (g == lane + i * kRow)
                gkey[i] = 0u;
    }
    int g = lane * NQ / size, next = (g + 1) * size;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        if (lane * NQ + q == next) {
            ++g;
            next += size;
        }
        key[q] = g < r.groups && ((kept >> g) & 1) ? key[q] : 0u;
    }
}

template <int NQ>
__device__ __forceinline__ float tree_sum(const float* v)
{
    if constexpr (NQ == 1)
        return v[0];
    else
        return tree_sum<NQ / 2>(v) + tree_sum<NQ / 2>(v + NQ / 2);
}

__device__ __forceinline__ float element(const float* p, int i) { return p[i]; }
__device__ __forceinline__ float element(const uint16_t* p, int i) { return bf16_to_f32(p[i]); }

// Elements e0 .. e0 + NQ - 1 of a row of E, `behind` behind its end. VEC: the row
// starts at a multiple of 16 bytes and is read so.
template <bool VEC, typename T, int NQ>
__device__ __forceinline__ void load_row(const T* row, int e0, int E, float behind, float (&v)[NQ])
{
    constexpr int kStep = VEC ? (NQ < 16 / (int)sizeof(T) ? NQ : 16 / (int)sizeof(T)) : 1;
    typedef T Part __attribute__((ext_vector_type(kStep)));
#pragma unroll
    for (int q = 0; q < NQ; q += kStep) {
        if (kStep > 1 && e0 + q + kStep <= E) {
            const Part p = *(const Part*)(row + e0 + q);
            T t[kStep];
            __builtin_memcpy(t, &p, sizeof(t));
#pragma unroll
            for (int i = 0; i < kStep; ++i)
                v[q + i] = element(t, i);
        } else {
#pragma unroll
            for (int i = 0; i < kStep; ++i)
                v[q + i] = e0 + q + i < E ? element(row, e0 + q + i) : behind;
        }
    }
}

// exp(x) of x <= 0: 2^(x log2 e) with the product in two parts, so that the
// reduced argument is good to 2^-26 whatever x is.
__device__ __forceinline__ float exp_of(float x)
{
#pragma clang fp contract(off)
    constexpr float kHi = 1.44269504f, kLo = 1.92596299e-8f;  // log2 e
    x = fmaxf(x, -150.0f);                                    // 0 from there on
    const float t = x * kHi;
    const float n = rintf(t);
    const float f = (t - n) + fmaf(x, kLo, fmaf(x, kHi, -t));
    return ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

// A score from a logit that is in (greater than -inf).
struct Score {
    bool sigmoid;
    float m, inv;  // softmax: the largest logit, 1 / the sum
    // equal infinities count as a difference of 0
    __device__ __forceinline__ float exponential(float l) const { return exp_of(l == m ? 0.0f : l - m); }
    // In the form that has no large exponential: the reciprocal is of a number
    // in 1..2, and one correction rounds it.
    __device__ __forceinline__ float logistic(float l) const
    {
#pragma clang fp contract(off)
        const float e = exp_of(-fabsf(l));
        const float d = 1.0f + e;
        float r = __builtin_amdgcn_rcpf(d);
        r = fmaf(fmaf(-d, r, 1.0f), r, r);
        return l < 0.0f ? e * r : r;
    }
    __device__ __forceinline__ float operator()(float l) const { return sigmoid ? logistic(l) : exponential(l) * inv; }
};

// The row of lanes selects for one token: `logits` reads them (one(e), e < E, and
// all(e0, l): NQ of them, -inf behind E). `store`: the token exists.
template <int NQ, class Logits>
__device__ __forceinline__ void select_token(const Logits& logits, int E, int k, const SelectRule& r, bool store,
                                             int32_t* ids, float* w)
{
    // The choice adds the bias to the rounded score, in every kernel alike.
#pragma clang fp contract(off)
    static_assert(kRow * NQ <= kMaxExperts && kMaxExperts <= 256 && kMaxTopK <= 8, "a pick is a byte of 64 bits");
    const int lane = threadIdx.x % kRow;
    const int e0 = lane * NQ;
    float l[NQ], s[NQ], b[NQ];
    logits.all(e0, l);
    if (r.bias && ((uintptr_t)r.bias & 15u) == 0)
        load_row<true>(r.bias, e0, E, 0.0f, b);
    else if (r.bias)
        load_row<false>(r.bias, e0, E, 0.0f, b);
    Score score{r.sigmoid != 0, 0.0f, 0.0f};
    if (score.sigmoid) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            s[q] = score.logistic(l[q]);
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            m = fmaxf(m, l[q]);  // not NaN
        row_steps([&](auto c) { m = fmaxf(m, __uint_as_float(row_move<c()>(__float_as_uint(m)))); });
        score.m = m;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            s[q] = l[q] > -INFINITY ? score.exponential(l[q]) : 0.0f;
        const float sum = row_sum(tree_sum<NQ>(s));
        score.inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            s[q] *= score.inv;
    }
    if (r.bias) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            s[q] += b[q];
    }
    uint32_t key[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const uint32_t u = __float_as_uint(s[q]);  // not -0: a score is +0 or larger
        key[q] = l[q] > -INFINITY && s[q] > -INFINITY ? u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u) : kOutKey;
    }
    if (e0 + NQ > E) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            key[q] = e0 + q < E ? key[q] : 0u;
    }
    if (r.top_groups < r.groups)
        keep_groups<NQ>(key, E, r);
    uint32_t my_key = 0;  // lane j: pick j
    uint64_t picks = 0;   // byte j: pick j, in the lane that held it
    for (int j = 0; j < k; ++j) {
        uint32_t mine = key[0];
#pragma unroll
        for (int q = 1; q < NQ; ++q)
            mine = max(mine, key[q]);
        const uint32_t best = row_max(mine);
        bool look = lane == row_first(mine == best);
        uint32_t e = 0;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const bool hit = look && key[q] == best;
            look = look && !hit;
            e = hit ? (uint32_t)(e0 + q) : e;
            key[q] = hit ? 0u : key[q];
        }
        picks |= (uint64_t)e << (8 * j);
        if (lane == j)
            my_key = best;
    }
    picks = (uint64_t)row_or((uint32_t)(picks >> 32)) << 32 | row_or((uint32_t)picks);
    const int id = (int)(picks >> (8 * (lane & 7))) & 0xFF;
    float v = 0.0f;
    if (lane < k && my_key > kOutKey)
        v = r.bias ? score(logits.one(id)) : key_value(my_key);  // without a bias the choice is the score
    if (r.normalize) {
        const float sum = row_sum(v);
        v = sum > 0.0f ? v / sum : 0.0f;
    }
    if (store && lane < k) {
        ids[lane] = id;
        w[lane] = v * r.scale;
    }
}

// Experts of a lane for E experts: the same in every kernel, as it is part of
// the order of a softmax's sum.
__host__ __device__ constexpr int select_width(int E)
{
    return E <= 4 * kRow ? 4 : E <= 8 * kRow ? 8 : 16;
}

struct LdsLogits {
    const float* row;
    int E;
    __device__ __forceinline__ float one(int e) const { return row[e]; }
    template <int NQ>
    __device__ __forceinline__ void all(int e0, float (&l)[NQ]) const
    {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            l[q] = e0 + q < E ? row[e0 + q] : -INFINITY;
    }
};

// The block's bt tokens from LDS logits [bt][ldl] (bias of the projection
// included).
template <int NQ>
__device__ inline void select_epilogue(const float* lg, int ldl, int bt, int t0, int T, int E, int k,
                                       const SelectRule& rule, int32_t* ids, float* wout)
{
    const int n = min(bt, T - t0);
    for (int r0 = 0; r0 < n; r0 += (int)blockDim.x / kRow) {
        const int r = r0 + (int)threadIdx.x / kRow;
        const int64_t t = t0 + r;
        select_token<NQ>(LdsLogits{lg + min(r, n - 1) * ldl, E}, E, k, rule, r < n, ids + t * k, wout + t * k);
    }
}

}  // namespace cmoe
