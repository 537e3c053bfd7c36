// router.hip - fused router: projection, top-k and softmax over the winners.
//
// One launch computes, for a block of 16 tokens,
//   logits[t][e] = sum_i x[t][i] * W_r[i][e] + b_r[e]      (fp32 accumulation)
// then selects the k largest logits per token (equal logits -> lower expert
// index, slot 0 = largest) and the renormalised softmax over those k:
//   w[t][j] = exp(l_j - l_0) / sum_j' exp(l_j' - l_0).
// This is the router of «Colibri 是什么» (xxqk.cn) §3.2 (a linear projection plus
// router bias, then a top-k selection on the logits) fused the way
// «Colibri：面向MoE模型的高性能C语言推理引擎» (zskr.cn) §2.2 and
// «Colibri不是一只蜂鸟» (discosf.com) §5.1 describe (projection, softmax and
// top-k in one pass with the intermediates kept on chip). Selection only needs
// the order of the logits, so exponentials are taken for the k winners only.
//
// bf16 path: the projection runs on v_mfma_f32_16x16x32_bf16 (16 tokens x 16
// experts per MFMA; init stores the router weights as 1 KiB operand blocks,
// one per 16 experts and 32-wide K step, so that each B fragment is one
// contiguous load); the 16 waves of a block (8 for more than 128 experts)
// split the reduction dimension in interleaved 32-wide steps and add their
// partial sums through LDS in a fixed order, so results are bit-reproducible
// and do not depend on the number of tokens in the call.
// fp32 path: plain FMA dot products (gfx950 has no faster fp32 matrix rate).
#include "select.hpp"

namespace cmoe {

namespace {

constexpr int kTok = 16;     // tokens per block
constexpr int kThreads = 256;  // fp32 path

// NG = number of 16-expert column groups (E <= 16 * NG); TG = number of
// 16-token groups per block; W = waves per block, which split the reduction
// dimension. Each wave's loads form a chain of dependent batches (one memory
// round trip each, and the router's inputs are usually cold: the expert GEMMs
// stream gigabytes through the caches between two calls), so W is as large as
// the register budget allows: 16 waves (8 for 256 experts). A token's logits
// do not depend on T or TG: every token is reduced by the same interleaving
// of K over the W waves and the same LDS summation order.
template <int NG, int TG, int W, bool RULE>
__global__ __launch_bounds__(W * kWave) void router_bf16_kernel(RouterArgs a)
{
    constexpr int EP = 16 * NG;      // padded expert count
    constexpr int LDL = EP + 1;      // LDS row stride (floats)
    constexpr int BT = kTok * TG;    // tokens per block
    __shared__ float part[BT][LDL];

    const int lane = threadIdx.x % kWave;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);  // wave-uniform
    const int t0 = blockIdx.x * BT;
    const int d = a.d;

    // A fragment rows: token rows, clamped (padded rows read valid memory and
    // their results are dropped); B fragments: whole blocks of the blocked
    // router weights (experts past E are zero rows there).
    const int kq = (lane >> 4) * 8;
    const uint16_t* xr[TG];
#pragma unroll
    for (int g = 0; g < TG; ++g)
        xr[g] = (const uint16_t*)a.x + (int64_t)min(t0 + g * kTok + (lane & 15), a.T - 1) * d + kq;
    // Router weights in MFMA operand blocks: the fragment of expert group n at
    // K step s is the 1 KiB block n * steps + s, lane l's 16 bytes at l*16.
    const int steps = d / 32;
    const Vec16* wb = (const Vec16*)a.w_rt + lane;

    floatx4 acc[TG][NG];
#pragma unroll
    for (int g = 0; g < TG; ++g)
#pragma unroll
        for (int n = 0; n < NG; ++n)
            acc[g][n] = floatx4{0.f, 0.f, 0.f, 0.f};

    // Wave w takes steps w, w+W, w+2W, ... in order; the loads of U of its
    // steps are issued before their MFMAs. The summation order does not
    // depend on U. Past the last step a batch reloads the last step with a
    // zero token fragment (adding exact zeros), so that every MFMA and every
    // load is unconditional: a step under a branch lets the compiler move its
    // loads into the branch and wait for each of them there.
    constexpr int U = NG * TG >= 8 ? 1 : 8 / (NG * TG);
    for (int s0 = wv; s0 < steps; s0 += W * U) {
        Vec16 av[U][TG], bv[U][NG];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int st = min(s0 + W * u, steps - 1);
#pragma unroll
            for (int g = 0; g < TG; ++g)
                av[u][g] = *(const Vec16*)(xr[g] + st * 32);
#pragma unroll
            for (int n = 0; n < NG; ++n)
                bv[u][n] = wb[(int64_t)(n * steps + st) * kWave];
        }
        __builtin_amdgcn_sched_barrier(0);  // all loads of the batch first
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool past = s0 + W * u >= steps;  // wave-uniform
#pragma unroll
            for (int g = 0; g < TG; ++g) {
                const Vec16 z = {0u, 0u, 0u, 0u};
                const Vec16 a_ = past ? z : av[u][g];
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    acc[g][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a_), as_bf16x8(bv[u][n]), acc[g][n],
                                                                        0, 0, 0);
            }
        }
    }

    // D layout of a 16x16 MFMA: lane holds rows 4*(lane/16)+i, column lane%16.
    // The W partial sums are added in wave order (((w0 + w1) + w2) + ...):
    // groups of up to 8 waves store their partials to LDS side by side, then
    // every thread adds the group's partials of its elements in wave order.
    constexpr int WG = W < 8 ? W : 8;
    constexpr int NE = BT * EP;                       // logits of the block (padded)
    constexpr int NS = (NE + W * kWave - 1) / (W * kWave);  // elements per thread
    __shared__ float red[WG][NE];
    float sum[NS];
    for (int wg = 0; wg < W; wg += WG) {
        if (wv >= wg && wv < wg + WG) {
            float* dst = red[wv - wg];
#pragma unroll
            for (int g = 0; g < TG; ++g)
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[(g * kTok + (lane >> 4) * 4 + i) * EP + n * 16 + (lane & 15)] = acc[g][n][i];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int idx = threadIdx.x + j * W * kWave;
            if (idx < NE) {
#pragma unroll
                for (int w = 0; w < WG; ++w)
                    sum[j] = (wg + w == 0) ? red[w][idx] : sum[j] + red[w][idx];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int idx = threadIdx.x + j * W * kWave;
        const int e = idx % EP;
        if (idx < NE)
            part[idx / EP][e] = e < a.E ? sum[j] + a.b[e] : sum[j];  // then the bias
    }
    __syncthreads();
    store_logits(&part[0][0], LDL, BT, t0, a.T, a.E, a.logits);
    if constexpr (RULE)
        select_epilogue<select_width(EP)>(&part[0][0], LDL, BT, t0, a.T, a.E, a.k, a.rule, a.ids, a.w);
    else
        topk_softmax_epilogue<(EP + kWave - 1) / kWave>(&part[0][0], LDL, BT, t0, a.T, a.E, a.k, a.ids, a.w);
}

template <bool RULE>
__global__ __launch_bounds__(kThreads) void router_f32_kernel(RouterArgs a)
{
    __shared__ float lg[kTok][kMaxExperts + 1];
    const int t0 = blockIdx.x * kTok;
    const float* x = (const float*)a.x;
    const float* wt = (const float*)a.w_rt;
    for (int i = threadIdx.x; i < kTok * a.E; i += kThreads) {
        const int r = i / a.E, e = i % a.E;
        const int t = min(t0 + r, a.T - 1);
        const float* xr = x + (int64_t)t * a.d;
        const float* wr = wt + (int64_t)e * a.d;
        float s = 0.0f;
        for (int c = 0; c < a.d; ++c)
            s = fmaf(xr[c], wr[c], s);
        lg[r][e] = s + a.b[e];
    }
    __syncthreads();
    store_logits(&lg[0][0], kMaxExperts + 1, kTok, t0, a.T, a.E, a.logits);
    if constexpr (RULE) {
        auto select = [&](auto nq) {
            select_epilogue<nq()>(&lg[0][0], kMaxExperts + 1, kTok, t0, a.T, a.E, a.k, a.rule, a.ids, a.w);
        };
        switch (select_width(a.E)) {
        case 4: select(std::integral_constant<int, 4>{}); break;
        case 8: select(std::integral_constant<int, 8>{}); break;
        default: select(std::integral_constant<int, 16>{}); break;
        }
    } else
        topk_softmax_epilogue<kMaxExperts / kWave>(&lg[0][0], kMaxExperts + 1, kTok, t0, a.T, a.E, a.k, a.ids, a.w);
}

__global__ void transpose_router_kernel(const uint8_t* src, uint8_t* dst, int d, int E, int esize)
{
    // dst[e][i] = src[i][e]
    const int64_t n = (int64_t)d * E;
    for (int64_t idx = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; idx < n;
         idx += (int64_t)gridDim.x * blockDim.x) {
        const int64_t e = idx / d, i = idx % d;
        const uint8_t* s = src + (i * E + e) * esize;
        uint8_t* o = dst + idx * esize;
        for (int b = 0; b < esize; ++b)
            o[b] = s[b];
    }
}

// Groups of 16 experts the bf16 router kernel multiplies (its NG).
int router_groups(int E)
{
    return E <= 16 ? 1 : E <= 32 ? 2 : E <= 64 ? 4 : E <= 128 ? 8 : 16;
}

// bf16 router weights [d][E] -> MFMA operand blocks for router_groups(E)
// groups of 16 experts (the layout router_weight_bytes sizes).
__global__ void block_router_kernel(const uint16_t* src, uint16_t* dst, int d, int E, int groups)
{
    const int steps = d / 32;
    const int64_t n = (int64_t)groups * steps * 512;
    for (int64_t idx = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; idx < n;
         idx += (int64_t)gridDim.x * blockDim.x) {
        const int j = (int)(idx & 7), lane = (int)((idx >> 3) & 63);
        const int64_t blk = idx >> 9;
        const int st = (int)(blk % steps), g = (int)(blk / steps);
        const int e = g * 16 + (lane & 15), i = st * 32 + (lane >> 4) * 8 + j;
        dst[idx] = e < E ? src[(int64_t)i * E + e] : (uint16_t)0;
    }
}

template <int NG, int TG>
hipError_t launch_router_tg(const RouterArgs& a, hipStream_t s)
{
    constexpr int W = NG >= 16 ? 8 : 16;  // 16 waves need <= 128 registers
    const int bt = kTok * TG;
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((a.T + bt - 1) / bt), dim3(W * kWave), 0, s, a); };
    if (a.rule.on)
        go(router_bf16_kernel<NG, TG, W, true>);
    else
        go(router_bf16_kernel<NG, TG, W, false>);
    return hipGetLastError();
}

// Token groups per block: with many experts and many tokens, blocks of 32
// (128 experts) or 64 tokens (64 experts) read the router weights fewer
// times (measured on MI355X: 16384 tokens x 64 experts 99 -> 68 us, 8192 x 128
// 58 -> 46 us); with few tokens or experts, 16-token blocks keep more blocks
// in flight.
template <int NG>
hipError_t launch_router_ng(const RouterArgs& a, hipStream_t s)
{
    if constexpr (NG == 4 || NG == 8) {
        if (a.T >= 4096)
            return launch_router_tg<NG, NG == 4 ? 4 : 2>(a, s);
    }
    return launch_router_tg<NG, 1>(a, s);
}

}  // namespace

hipError_t launch_router_bf16(const RouterArgs& a, hipStream_t s)
{
    // NG = router_groups(E): the weight blocks hold exactly that many groups
    switch (router_groups(a.E)) {
    case 1:
        return launch_router_ng<1>(a, s);
    case 2:
        return launch_router_ng<2>(a, s);
    case 4:
        return launch_router_ng<4>(a, s);
    case 8:
        return launch_router_ng<8>(a, s);
    default:
        return launch_router_ng<16>(a, s);
    }
}

hipError_t launch_router_f32(const RouterArgs& a, hipStream_t s)
{
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((a.T + kTok - 1) / kTok), dim3(kThreads), 0, s, a); };
    if (a.rule.on)
        go(router_f32_kernel<true>);
    else
        go(router_f32_kernel<false>);
    return hipGetLastError();
}

size_t router_weight_bytes(int d, int E, int esize)
{
    return esize == 2 ? (size_t)router_groups(E) * 16 * d * 2 : (size_t)E * d * esize;
}

hipError_t launch_transpose_router(const void* w_r, void* w_rt, int d, int E, int esize, hipStream_t s)
{
    if (esize == 2)
        hipLaunchKernelGGL(block_router_kernel, dim3(256), dim3(256), 0, s, (const uint16_t*)w_r, (uint16_t*)w_rt,
                           d, E, router_groups(E));
    else
        hipLaunchKernelGGL(transpose_router_kernel, dim3(256), dim3(256), 0, s, (const uint8_t*)w_r,
                           (uint8_t*)w_rt, d, E, esize);
    return hipGetLastError();
}

}  // namespace cmoe
