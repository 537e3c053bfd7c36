// few.hip - the whole layer for at most 16 tokens in two launches.
//
//   few_gate_up_kernel: logits, top-k and softmax (as router.hip), then
//     h[t][j][c] = SiLU(sum_i x[t][i] Wg[e][c][i]) * (sum_i x[t][i] Wu[e][c][i]),   e = ids[t][j]
//   few_down_kernel:
//     y[t][o] = sum_j w[t][j] sum_c Wd[e][o][c] h[t][j][c]
// for bf16, 8-bit (E4M3, row scales) and 4-bit (MXFP4) expert weights in the
// layouts of the other GEMM paths.
//
// For so few tokens the work is reading the active experts' weights once, and
// the six or seven dependent launches of the general path cost more than many
// layers' weights. Two launches are the fewest without a barrier across
// workgroups (which could wait for ever beside another such call): the down
// product needs every h of an expert.
//   * The 16 tokens are the second operand of v_mfma_f32_16x16x32_bf16, 16
//     weight rows the first. Every active expert's rows are multiplied with all
//     tokens and the tokens that did not choose it drop out at the end, so no
//     token is gathered and the matrix work (a sixteenth of the pipe's rate) is
//     free.
//   * A workgroup is 16 waves that split K in interleaved steps and add their
//     sums through LDS in wave order; its work item is 16 weight rows (gate and
//     up rows of 16 columns; 32 columns of 4-bit weights). A wave thus reads the
//     same K steps in every item, and keeps its token fragments in registers
//     over all of them (d_model up to 4096).
//   * Every workgroup computes the routing itself, in the order of the router
//     kernel (the same logits bit for bit), from router weights that its XCD's
//     L2 holds after the first; the first workgroup writes the routing outputs.
//   * h is kept as a pair of bf16 (value and remainder, 16 significant bits):
//     the second MFMA it costs is free here, and h adds no error to speak of.
//   * Weights are read with non-temporal loads, two register sets in flight.
// Measured (GPU time of the two kernels, bytes of the experts that were active):
// 1 token, bf16, 8 experts of 4096 x 14336, k = 2: 77 + 41 us for 470 + 235 MB
// (6.1 and 5.8 TB/s; a plain read of memory reaches 5.7 - 6.2); 16 tokens, bf16,
// 128 of 2048 x 768, k = 4, 50 active: 69 + 31 us for 315 + 157 MB, 9 us of it the
// routing's 512 KB per workgroup; 7 tokens, 4-bit, 8 of 4096 x 14336, 6 active: 73
// + 41 us for 374 + 187 MB (5.1 and 4.5 TB/s); 3 tokens, 8-bit, 64 of 4096 x 1408:
// 19 + 11 us for 29 + 14 MB, bound by latency (start, routing, two reductions). A
// very small layer takes 8 + 4 us. Against the general path (whole calls, us, 1 / 7
// / 16 tokens, 8 experts of 4096 x 14336): bf16 122 / 320 / 438 and 170 / 364 /
// 440, 8-bit 72 / 184 / 251 and 109 / 212 / 250, 4-bit 52 / 115 / 158 and 67 / 133
// / 155: 16 tokens on few large experts gain nothing. Reading the down weights
// ahead into the caches at the end of the first kernel cost 1 - 5 us instead of
// saving any.
#include "mxfp4.hpp"
#include "topk.hpp"

namespace cmoe {

namespace {

constexpr int kTok = 16;
constexpr int kWaves = 16;
constexpr int kThreads = kWaves * kWave;
constexpr int kMaxAssign = kTok * kMaxTopK;
constexpr int kXV = 8;  // token fragments a wave keeps: 4096 k over the 16 waves

enum Format { kBf16 = 0, kFp8 = 1, kMx4 = 2 };

// A unit: the K range whose weight fragments are one 16-byte load per lane (16
// rows), M MFMAs of 32 k. Lane l holds row l%16 and, of the unit, the M * 8
// consecutive k from M * 8 * (l/16).
template <int FMT>
struct Unit {
    static constexpr int M = FMT == kBf16 ? 1 : FMT == kFp8 ? 2 : 4;
    static constexpr int K = 32 * M;
    static constexpr int kCG = FMT == kMx4 ? 2 : 1;  // gate/up: 16-column groups per item
    static constexpr int kXU = kXV / M;              // units of token fragments kept
    static constexpr int kUPS = FMT == kBf16 ? 4 : FMT == kFp8 ? 2 : 1;  // units per step
};

// Byte offset of lane l's 16 bytes for rows 16 cj .. +16 of a 32-row block from
// the start of a unit of it, in any of the three blocked layouts (1 KiB blocks
// of 32 rows x half a unit of k, two to a unit).
__device__ __forceinline__ uint32_t unit_lane(int cj, int lane)
{
    const int o = lane >> 4;
    return (uint32_t)((o >> 1) * kWave + (o & 1) * 32 + 16 * cj + (lane & 15)) * 16u;
}

// MXFP4: the scale byte of that lane's 32 codes, from the row block's part of
// the unit's scales (its two blocks kb are lane halves o/2 here).
__device__ __forceinline__ uint32_t unit_scale_lane(int cj, int lane)
{
    const int o = lane >> 4;
    return (uint32_t)((o & 1) * 32 + 16 * cj + (lane & 15)) * 2u + (uint32_t)(o >> 1);
}

// A wave-uniform address in scalar registers, so that the loads from it take a
// 32-bit offset per lane.
__device__ __forceinline__ const uint8_t* uniform(const void* p)
{
    const uint64_t a = (uint64_t)(uintptr_t)p;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
    return (const uint8_t*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

// MFMA fragment s of a unit's 16 bytes; sc: the row's or the block's scale.
template <int FMT>
__device__ __forceinline__ bf16x8 unit_frag(const Vec16& w, int s, float sc)
{
    if constexpr (FMT == kBf16)
        return as_bf16x8(w);
    else if constexpr (FMT == kFp8)
        return fp8x8_to_bf16(w[2 * s], w[2 * s + 1], sc);
    else
        return mx8_to_bf16(w[s], sc);
}

// Barrier for LDS data; loads from global memory stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Which experts are active (ascending) and who chose them.
struct Choice {
    int row;  // t * k + j, or -1: token t did not choose the expert
    float w;
};
struct Routes {
    int32_t ids[kMaxAssign];
    float w[kMaxAssign];
    uint32_t mask[kMaxExperts / 32];
    int32_t act[kMaxAssign];
    Choice tab[kMaxAssign][kTok];
};

// Builds r.act and r.tab from r.ids and r.w (filled before the call, by any
// threads; the first barrier is here). Returns the number of active experts.
__device__ __forceinline__ int build_routes(Routes& r, int T, int k)
{
    const int tid = threadIdx.x, A = T * k;
    if (tid < kMaxExperts / 32)
        r.mask[tid] = 0;
    for (int i = tid; i < A * kTok; i += kThreads)
        r.tab[i / kTok][i % kTok] = Choice{-1, 0.f};
    lds_barrier();
    int e = 0;
    if (tid < A) {
        e = r.ids[tid];
        atomicOr(&r.mask[e >> 5], 1u << (e & 31));
    }
    lds_barrier();
    int below = 0, n = 0;
#pragma unroll
    for (int q = 0; q < kMaxExperts / 32; ++q) {
        const uint32_t m = r.mask[q];
        n += __popc(m);
        below += q < (e >> 5) ? __popc(m) : q == (e >> 5) ? __popc(m & ((1u << (e & 31)) - 1u)) : 0;
    }
    if (tid < A) {
        r.act[below] = e;
        r.tab[below][tid / k] = Choice{tid, r.w[tid]};
    }
    lds_barrier();
    return __builtin_amdgcn_readfirstlane(n);
}

// The routing of the call's tokens into r.ids / r.w, as router_bf16_kernel
// computes it: wave w takes K steps w, w + 16, ..., the waves' sums are added
// in wave order, then the bias. lds holds the partial sums and the logits.
constexpr int kRouteFloats = kTok * 129 + 8 * kTok * 128;

template <int NG>
__device__ __forceinline__ void route(const FewArgs& g, float* lds, Routes& r, bool first)
{
    constexpr int EP = 16 * NG, LDL = EP + 1, NE = kTok * EP;
    constexpr int NS = (NE + kThreads - 1) / kThreads;
    constexpr int U = NG >= 8 ? 2 : 16 / NG > 8 ? 8 : 16 / NG;  // steps whose loads are in flight
    static_assert(kTok * LDL + 8 * NE <= kRouteFloats, "LDS");
    float* part = lds;              // [kTok][LDL]
    float* red = lds + kTok * LDL;  // [8][NE]
    const int lane = threadIdx.x % kWave;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int steps = g.d / 32;
    const uint16_t* xr = (const uint16_t*)g.x + (int64_t)min(lane & 15, g.T - 1) * g.d + (lane >> 4) * 8;
    const Vec16* wb = (const Vec16*)g.w_rt + lane;
    floatx4 acc[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n)
        acc[n] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = wv; s0 < steps; s0 += kWaves * U) {
        Vec16 av[U], bv[U][NG];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int st = min(s0 + kWaves * u, steps - 1);
            av[u] = *(const Vec16*)(xr + st * 32);
#pragma unroll
            for (int n = 0; n < NG; ++n)
                bv[u][n] = wb[(int64_t)(n * steps + st) * kWave];
        }
        __builtin_amdgcn_sched_barrier(0);  // all loads of the batch first
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Vec16 z = {0u, 0u, 0u, 0u};
            const Vec16 a = s0 + kWaves * u >= steps ? z : av[u];  // past the last step: exact zeros
#pragma unroll
            for (int n = 0; n < NG; ++n)
                acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(bv[u][n]), acc[n], 0, 0, 0);
        }
    }
    float sum[NS];
    for (int wg = 0; wg < kWaves; wg += 8) {
        if (wv >= wg && wv < wg + 8) {
            float* dst = red + (wv - wg) * NE;
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dst[((lane >> 4) * 4 + i) * EP + n * 16 + (lane & 15)] = acc[n][i];
        }
        lds_barrier();
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int idx = threadIdx.x + j * kThreads;
            if (idx < NE) {
#pragma unroll
                for (int w = 0; w < 8; ++w)
                    sum[j] = wg + w == 0 ? red[w * NE + idx] : sum[j] + red[w * NE + idx];
            }
        }
        lds_barrier();
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int idx = threadIdx.x + j * kThreads;
        const int e = idx % EP;
        if (idx < NE)
            part[idx / EP * LDL + e] = e < g.E ? sum[j] + g.b[e] : sum[j];
    }
    lds_barrier();
    if (first)
        store_logits(part, LDL, kTok, 0, g.T, g.E, g.logits);
    topk_softmax_epilogue<(EP + kWave - 1) / kWave>(part, LDL, kTok, 0, g.T, g.E, g.k, r.ids, r.w);
}

// Routing outputs of the call (one workgroup): ids and weights, which the
// second kernel reads, and the dispatch a general forward reports (a stable
// counting sort of the assignments by expert).
__device__ __forceinline__ void store_routes(const FewArgs& g, const Routes& r)
{
    const int tid = threadIdx.x, A = g.T * g.k;
    if (tid < A) {
        const int e = r.ids[tid];
        if (!g.routed) {
            g.ids[tid] = e;
            g.w[tid] = r.w[tid];
        }
        int pos = 0;
        for (int a = 0; a < A; ++a)
            pos += r.ids[a] < e || (r.ids[a] == e && a < tid) ? 1 : 0;
        if (g.perm)
            g.perm[pos] = tid / g.k;
        if (g.perm_slot)
            g.perm_slot[pos] = tid % g.k;
        if (g.inv)
            g.inv[tid] = pos;
    }
    if ((g.counts || g.offsets) && tid <= g.E) {
        int below = 0, at = 0;
        for (int a = 0; a < A; ++a) {
            below += r.ids[a] < tid ? 1 : 0;
            at += r.ids[a] == tid ? 1 : 0;
        }
        if (g.counts && tid < g.E)
            g.counts[tid] = at;
        if (g.offsets)
            g.offsets[tid] = below;
    }
}

// Token fragments of the experts' products, quantized where the layer
// quantizes its token rows: exponent byte of the row (8-bit) or of the lane's
// block of 32 (4-bit), the code, and the value it stands for, exact in bf16.
__device__ __forceinline__ void widen8(const Vec16& v, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t abs_max8(const Vec16& v, uint32_t m)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(m, max((v[i] << 16) & 0x7FFFFFFFu, v[i] & 0x7FFF0000u));
    return m;
}

__device__ __forceinline__ Vec16 fp8_round(const Vec16& v, int e)
{
    float f[8];
    widen8(v, f);
    const float inv = ldexpf(1.0f, -e), sc = ldexpf(1.0f, e);
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inv, f[1] * inv, 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inv, f[3] * inv, lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * inv, f[5] * inv, 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * inv, f[7] * inv, hi, true);
    return __builtin_bit_cast(Vec16, fp8x8_to_bf16((uint32_t)lo, (uint32_t)hi, sc));
}

// The two register sets of weight loads of the gate/up kernel.
template <int FMT>
struct Step {
    using U = Unit<FMT>;
    Vec16 w[U::kUPS][2][U::kCG];
    uint32_t mx[FMT == kMx4 ? U::kUPS : 1][2][U::kCG];
    float sc[2];
};

template <int FMT>
__global__ __launch_bounds__(kThreads) void few_gate_up_kernel(FewArgs g)
{
    using U = Unit<FMT>;
    constexpr int M = U::M, CG = U::kCG, UPS = U::kUPS, XU = U::kXU;
    constexpr int NP = 2 * CG * 256;  // partial sums of a wave per item
    __shared__ Routes r;
    // the waves' sums of two items; before that the router's, of up to 128 experts
    constexpr int kLds = 2 * kWaves * NP > kRouteFloats ? 2 * kWaves * NP : kRouteFloats;
    __shared__ __align__(16) float lds[kLds];

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wv = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int A = g.T * g.k;

    if (g.routed) {  // the router kernel ran before
        if (tid < A) {
            r.ids[tid] = g.ids[tid];
            r.w[tid] = g.w[tid];
        }
    } else {
        const bool first = blockIdx.x == 0;
        if (g.E <= 16)
            route<1>(g, lds, r, first);
        else if (g.E <= 32)
            route<2>(g, lds, r, first);
        else if (g.E <= 64)
            route<4>(g, lds, r, first);
        else
            route<8>(g, lds, r, first);
    }
    // Token fragments of units wv + 16 i, i < XU, of K chunk ch.
    const int NU = g.d / U::K;
    const uint16_t* xr = (const uint16_t*)g.x + (int64_t)min(lane & 15, g.T - 1) * g.d + (lane >> 4) * (8 * M);
    Vec16 x[kXV];
    int xe = 0;  // 8-bit token rows: exponent of this lane's token
    auto load_x = [&](int ch) {
#pragma unroll
        for (int i = 0; i < XU; ++i) {
            const int u = min(wv + kWaves * (ch * XU + i), NU - 1);
#pragma unroll
            for (int s = 0; s < M; ++s)
                x[i * M + s] = *(const Vec16*)(xr + u * U::K + s * 8);
        }
    };
    auto round_x = [&]() {
        if constexpr (FMT == kFp8) {
            if (g.act_quant)
#pragma unroll
                for (int i = 0; i < kXV; ++i)
                    x[i] = fp8_round(x[i], xe);
        }
        if constexpr (FMT == kMx4) {
            if (g.act_quant)
#pragma unroll
                for (int i = 0; i < XU; ++i) {
                    uint32_t m = 0;
#pragma unroll
                    for (int s = 0; s < M; ++s)
                        m = abs_max8(x[i * M + s], m);
                    const uint32_t b = mx_scale_byte(m);
                    const float inv = mx_inv_scale(b == kMxNan ? 127u : b), sc = mx_scale(b);
#pragma unroll
                    for (int s = 0; s < M; ++s) {
                        float f[8];
                        widen8(x[i * M + s], f);
                        x[i * M + s] = __builtin_bit_cast(Vec16, mx8_to_bf16(b == kMxNan ? 0u : mx_encode8(f, inv), sc));
                    }
                }
        }
    };
    load_x(0);  // on their way while the routes are built
    const int nact = build_routes(r, g.T, g.k);
    if (blockIdx.x == 0)
        store_routes(g, r);

    if constexpr (FMT == kFp8) {
        if (g.act_quant) {  // the row's largest magnitude, over the lanes and waves that hold it
            uint32_t m = 0;
            for (int u = wv; u < NU; u += kWaves)
#pragma unroll
                for (int s = 0; s < M; ++s)
                    m = abs_max8(*(const Vec16*)(xr + u * U::K + s * 8), m);
            m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
            m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
            uint32_t* mx = (uint32_t*)lds;
            if (lane < 16)
                mx[wv * 16 + lane] = m;
            lds_barrier();
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                m = max(m, mx[w * 16 + (lane & 15)]);
            lds_barrier();
            // smallest e >= -126 with amax <= 448 * 2^e = 1.75 * 2^(e + 8); 0 for a row of zeros
            const int E = (int)(m >> 23);
            xe = m == 0 ? 0 : max(-126, E - 127 - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0));
        }
    }

    // Steps of an item: UPS units per wave each. One where the units fit, else
    // an even number (two steps to a chunk of kept fragments).
    const int P = NU <= kWaves * UPS ? 1 : (NU + kWaves * XU - 1) / (kWaves * XU) * (XU / UPS);
    const bool one_chunk = NU <= kWaves * XU;
    round_x();
    const int groups = g.f / (16 * CG);
    const int items = nact * groups;
    const int mine = (int)blockIdx.x < items ? (items - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    const int Q = mine * P;
    const int KB = 2 * NU, NBK = g.f / 16;  // 32-row blocks of [2f]

    const uint32_t lane_w = unit_lane(0, lane), lane_m = unit_scale_lane(0, lane);

    floatx4 acc[2][CG];
    auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c = 0; c < CG; ++c)
                acc[n][c] = floatx4{0.f, 0.f, 0.f, 0.f};
    };
    clear();

    auto load = [&](Step<FMT>& t, int q) {
        q = min(q, Q - 1);
        const int p = q % P, it = (int)blockIdx.x + (int)gridDim.x * (q / P);
        const int a = it / groups, c = it - a * groups;
        const int e = __builtin_amdgcn_readfirstlane(r.act[a]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int64_t rb = (int64_t)e * NBK + 2 * (CG == 2 ? c : c / 2) + n;
            const int cj = CG == 2 ? 0 : c & 1;
#pragma unroll
            for (int i = 0; i < UPS; ++i) {
                const int u = min(wv + kWaves * (p * UPS + i), NU - 1);
                const uint8_t* wp = uniform((const uint8_t*)g.w_gu + (rb * KB + 2 * u) * 1024 + cj * 256);
#pragma unroll
                for (int h = 0; h < CG; ++h)
                    t.w[i][n][h] = __builtin_nontemporal_load((const Vec16*)(wp + lane_w + h * 256));
                if constexpr (FMT == kMx4) {
                    const int nb = 2 * c + n;
                    const uint8_t* mp = uniform(g.m_gu + mx_scale_group(e, nb, u, 2 * g.f, g.d) + mx_scale_at(nb, 0, 0));
#pragma unroll
                    for (int h = 0; h < CG; ++h)
                        t.mx[i][n][h] = mp[lane_m + h * 32];
                }
            }
            if constexpr (FMT == kFp8)
                t.sc[n] = g.s_gu[rb * 32 + 16 * cj + (lane & 15)];
        }
    };
    auto multiply = [&](const Step<FMT>& t, int p, auto x0_const) {
        constexpr int x0 = decltype(x0_const)::value;
#pragma unroll
        for (int i = 0; i < UPS; ++i)
            if (wv + kWaves * (p * UPS + i) < NU)
#pragma unroll
                for (int s = 0; s < M; ++s)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int h = 0; h < CG; ++h) {
                            const float sc = FMT == kMx4 ? mx_scale(t.mx[FMT == kMx4 ? i : 0][n][h]) : t.sc[n];
                            acc[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                unit_frag<FMT>(t.w[i][n][h], s, sc), as_bf16x8(x[x0 + i * M + s]), acc[n][h], 0, 0, 0);
                        }
    };
    int buf = 0;
    // Step q from set t; the item's sums leave after its last step.
    auto take = [&](const Step<FMT>& t, int q) {
        const int p = q % P;
        if (!one_chunk && p % (XU / UPS) == 0) {
            load_x(p / (XU / UPS));
            round_x();
        }
        if (XU / UPS == 1 || (p & 1) == 0)
            multiply(t, p, std::integral_constant<int, 0>{});
        else
            multiply(t, p, std::integral_constant<int, (XU / UPS == 1 ? 0 : UPS * M)>{});
        if (p != P - 1)
            return;
        // Result lane: token lane%16, weight rows 4 (lane/16) + i. The item
        // after next writes this buffer again, when every thread has passed the
        // next item's barrier and so has read it.
        float* sums = lds + buf * kWaves * NP;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < CG; ++h)
                *(floatx4*)(sums + wv * NP + (h * 2 + n) * 256 + lane * 4) = acc[n][h];
        clear();
        lds_barrier();
        if (tid < 256 * CG) {
            const int h = tid / 256, el = tid % 256;
            float gs = 0.f, us = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                gs += sums[w * NP + h * 512 + el];
                us += sums[w * NP + h * 512 + 256 + el];
            }
            const int it = (int)blockIdx.x + (int)gridDim.x * (q / P);
            const int a = it / groups, c = it - a * groups;
            const int t16 = (el / 4) % 16, col = (c * CG + h) * 16 + 4 * (el / 64) + el % 4;
            const int row = r.tab[a][t16].row;
            if (row >= 0) {
                const float hv = silu(gs) * us;
                const uint16_t hi = f32_to_bf16_bits(hv);
                uint16_t* hp = g.h + (int64_t)row * g.f + col;
                hp[0] = hi;
                // the remainder (0 for a non-finite h, whose high part says it all)
                const float lo = hv - bf16_to_f32(hi);
                hp[(int64_t)A * g.f] = f32_to_bf16_bits(fabsf(hv) < INFINITY && fabsf(lo) < INFINITY ? lo : 0.f);
            }
        }
        buf ^= 1;
    };
    if (Q == 0)
        return;
    Step<FMT> t0, t1;
    load(t0, 0);
    for (int q = 0; q < Q; q += 2) {
        load(t1, q + 1);
        take(t0, q);
        load(t0, q + 2);
        if (q + 1 < Q)
            take(t1, q + 1);
    }
}

// 16-row groups of W_down per item of the down kernel.
__host__ __device__ constexpr int down_groups(int fmt)
{
    return fmt == kMx4 ? 4 : 2;
}

// What the low parts of h add to a sum of weights times h. An infinite weight
// decides such a sum by the high parts alone: times a low part it would give
// NaN (0 * inf) or the opposite infinity.
__device__ __forceinline__ float low_sum(float v)
{
    return fabsf(v) < INFINITY ? v : 0.f;
}

// Loads of B units of the down kernel: weights and scales of both 16-row
// halves, and the token fragments of h (lanes whose token did not choose the
// expert load nothing and hold zeros). H = 2: high and low parts apart, for 16
// tokens; H = 1: at most 8 tokens, whose high parts are columns 0..7 and low
// parts columns 8..15 of one fragment.
template <int FMT, int B, int H, int W>
struct DownStep {
    static constexpr int M = Unit<FMT>::M;
    static constexpr bool LATE = FMT == kMx4 && H == 2;  // (two sets of 16 fragments spill)
    Vec16 w[B][W];
    uint32_t mx[FMT == kMx4 ? B : 1][W];
    float sc[FMT == kFp8 ? B : 1][W];
    Vec16 x[LATE ? 1 : B][M][H];
    uint32_t row[LATE ? B : 1];  // LATE: where x is, loaded just before it is multiplied
    int at[LATE ? B : 1];
    float wt[B];  // routing weight, -1 if the lane's token did not choose the expert
};

// A work item is 16 W output columns: an h fragment costs as much to load as a
// weight fragment, so each serves both halves of a row block, on 4-bit weights
// (four h fragments to a weight load) two row blocks, and up to 8 tokens take
// one fragment instead of two (7 tokens on 4-bit weights: 16 columns 77 us, 32
// 56, with one fragment 45, 64 columns 41). An item is one of g.split parts of
// the units of all active experts, which its 16 waves take in interleaved
// order. With more than one part the parts' sums go to memory
// and the workgroup that finishes the column block last adds them in the order
// of the parts: nobody waits, and the result does not depend on who is last.
template <int FMT, int H>
__global__ __launch_bounds__(kThreads) void few_down_kernel(FewArgs g)
{
    using U = Unit<FMT>;
    constexpr int M = U::M;
    constexpr int B = FMT == kBf16 ? (H == 1 ? 4 : 3) : FMT == kFp8 && H == 1 ? 2 : 1;
    __shared__ Routes r;
    constexpr int W = down_groups(FMT), NC = 16 * W;  // 16-row groups, columns of an item
    __shared__ __align__(16) float red[kWaves][W * 256];
    __shared__ int last;

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wv = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int A = g.T * g.k;
    if (tid < A) {
        r.ids[tid] = g.ids[tid];
        r.w[tid] = g.w[tid];
    }
    const int nact = build_routes(r, g.T, g.k);
    const int NU = g.f / U::K;  // units per expert
    const int KB = 2 * NU, NBK = g.d / 32;
    const uint32_t plane = (uint32_t)A * (uint32_t)g.f * 2u;
    const __amdgpu_buffer_rsrc_t rh = __builtin_amdgcn_make_buffer_rsrc((void*)g.h, 0, (int)(2 * plane), 0x00020000);
    const uint32_t lane_w = unit_lane(0, lane), lane_m = unit_scale_lane(0, lane);

    const int nb = (int)blockIdx.x / g.split, part = (int)blockIdx.x - nb * g.split;
    const int v0 = (int)((int64_t)part * nact * NU / g.split);
    const int V = (int)((int64_t)(part + 1) * nact * NU / g.split);  // units v0 .. V of the item
    floatx4 total[W];
#pragma unroll
    for (int h = 0; h < W; ++h)
        total[h] = floatx4{0.f, 0.f, 0.f, 0.f};
    // The wave's next unit to load: unit cu of active expert ca, of whose
    // tokens and weights cwt, crow, cw, cm, cs tell.
    int cv = v0 + wv, ca = -1, cu = 0;
    float cwt = 0.f, cs[2] = {1.f, 1.f};  // (8-bit weights: W = 2)
    uint32_t crow = 0;
    const uint8_t *cw = nullptr, *cm = nullptr;
    auto open = [&](int a) {
        ca = a;
        const int e = __builtin_amdgcn_readfirstlane(r.act[a]);
        const int64_t rb = (int64_t)e * NBK + nb * (W / 2);
        const Choice ch = r.tab[a][H == 1 ? lane & 7 : lane & 15];
        cwt = ch.row < 0 ? -1.f : ch.w;
        // past the buffer for lanes that hold zeros
        crow = ch.row < 0 ? 0x80000000u : ((uint32_t)ch.row * (uint32_t)g.f + (uint32_t)((lane >> 4) * 8 * M)) * 2u;
        if (H == 1 && (lane & 8))
            crow += plane;
        cw = uniform((const uint8_t*)g.w_d + rb * KB * 1024);
        if constexpr (FMT == kMx4)
            cm = uniform(g.m_d + mx_scale_group(e, nb * (W / 2), 0, g.d, g.f) + mx_scale_at(nb * (W / 2), 0, 0));
        if constexpr (FMT == kFp8)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                cs[h] = ((const float*)uniform(g.s_d + rb * 32))[16 * h + (lane & 15)];
    };
    auto load_x = [&](Vec16 (&x)[M][H], uint32_t row, int at) {
#pragma unroll
        for (int s = 0; s < M; ++s)
#pragma unroll
            for (int h = 0; h < H; ++h)
                x[s][h] = __builtin_bit_cast(
                    Vec16, __builtin_amdgcn_raw_buffer_load_b128(rh, (int)(row + 16u * s), at + h * (int)plane, 0));
    };
    constexpr bool LATE = DownStep<FMT, B, H, W>::LATE;
    auto load = [&](DownStep<FMT, B, H, W>& t) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            t.wt[b] = cwt;
            const uint8_t* wp = cw + (int64_t)cu * 2048;
#pragma unroll
            for (int h = 0; h < W; ++h) {
                t.w[b][h] = __builtin_nontemporal_load(
                    (const Vec16*)(wp + (int64_t)(h / 2) * KB * 1024 + lane_w + h % 2 * 256));
                if constexpr (FMT == kMx4)
                    t.mx[b][h] = (cm + (int64_t)cu * 1024)[lane_m + h / 2 * 128 + h % 2 * 32];
                if constexpr (FMT == kFp8)
                    t.sc[b][h] = cs[h];
            }
            const int at = cu * U::K * 2;
            if constexpr (LATE) {
                t.row[b] = crow;
                t.at[b] = at;
            } else {
                load_x(t.x[b], crow, at);
            }
            if (cv + kWaves < V) {  // else this unit again, not multiplied
                cv += kWaves;
                cu += kWaves;
                int a = ca;
                while (cu >= NU) {
                    cu -= NU;
                    ++a;
                }
                if (a != ca)
                    open(a);
            }
        }
    };
    auto multiply = [&](const DownStep<FMT, B, H, W>& t, int i0) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (v0 + wv + kWaves * (i0 + b) >= V)
                continue;
            floatx4 acc[W];
#pragma unroll
            for (int h = 0; h < W; ++h)
                acc[h] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < M; ++s)
#pragma unroll
                for (int h = 0; h < W; ++h) {
                    const float sc = FMT == kMx4 ? mx_scale(t.mx[FMT == kMx4 ? b : 0][h]) : t.sc[FMT == kFp8 ? b : 0][h];
                    const bf16x8 f = unit_frag<FMT>(t.w[b][h], s, sc);
#pragma unroll
                    for (int p = 0; p < H; ++p)
                        acc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, as_bf16x8(t.x[b][s][p]), acc[h], 0, 0, 0);
                }
            // A sum that is not finite is taken again without the low parts
            // (low_sum). H = 1 keeps the parts' sums apart to the end.
            if constexpr (H == 2) {
                float bad = 0.f;
#pragma unroll
                for (int h = 0; h < W; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        bad = fmaf(acc[h][i], 0.f, bad);
                if (__ballot(bad != 0.f) != 0) {  // NaN: some sum is not finite
#pragma unroll
                    for (int h = 0; h < W; ++h) {
                        floatx4 hi = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int s = 0; s < M; ++s) {
                            float sc = FMT == kMx4 ? mx_scale(t.mx[FMT == kMx4 ? b : 0][h]) : t.sc[FMT == kFp8 ? b : 0][h];
                            if constexpr (FMT != kBf16)  // converts again: fragments kept for this would spill
                                asm volatile("" : "+v"(sc));
                            hi = __builtin_amdgcn_mfma_f32_16x16x32_bf16(unit_frag<FMT>(t.w[b][h], s, sc),
                                                                         as_bf16x8(t.x[b][s][0]), hi, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[h][i] = fabsf(acc[h][i]) < INFINITY ? acc[h][i] : hi[i];
                    }
                }
            }
            // only the tokens that chose this expert take its rows (whose
            // weights may be infinite or NaN)
#pragma unroll
            for (int h = 0; h < W; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    total[h][i] = t.wt[b] < 0.f ? total[h][i] : fmaf(t.wt[b], acc[h][i], total[h][i]);
        }
    };
    const int I = (V - v0 + kWaves - 1) / kWaves;  // units per wave, at most
    if (cv < V) {
        cu = cv;
        int a = 0;
        while (cu >= NU) {
            cu -= NU;
            ++a;
        }
        open(a);
        DownStep<FMT, B, H, W> t0, t1;
        load(t0);
        for (int i = 0; i < I; i += 2 * B) {
            if constexpr (LATE)
                load_x(t0.x[0], t0.row[0], t0.at[0]);  // before the next weights: the wait for it leaves them in flight
            load(t1);
            multiply(t0, i);
            if constexpr (LATE)
                load_x(t1.x[0], t1.row[0], t1.at[0]);
            load(t0);
            multiply(t1, i + B);
        }
    }
#pragma unroll
    for (int h = 0; h < W; ++h)
        *(floatx4*)(&red[wv][h * 256 + lane * 4]) = total[h];
    lds_barrier();
    float sum = 0.f;
    if (tid < W * 256)
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            sum += H == 1 ? red[w][tid] + low_sum(red[w][tid ^ 32]) : red[w][tid];  // ^ 32: eight columns on
    if (g.split > 1) {
        // Parts and counts are accessed at device scope (written through and
        // read past the XCDs' separate L2s), ordered by the wait for the stores
        // and the barrier before the count. Fences would do the same by
        // flushing every L2 from every wave, which took 115 us here.
        float* mine = g.part + (int64_t)blockIdx.x * (W * 256);
        if (tid < W * 256)
            __hip_atomic_store(mine + tid, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        lds_barrier();
        if (tid == 0)
            last = __hip_atomic_fetch_add(&g.count[nb], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == g.split - 1;
        lds_barrier();
        if (!last)
            return;
        if (tid == 0)  // for the next call
            __hip_atomic_store(&g.count[nb], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        float v[kFewMaxSplit];
        sum = 0.f;
        if (tid < W * 256) {
#pragma unroll
            for (int p = 0; p < kFewMaxSplit; ++p)
                if (p < g.split)
                    v[p] = __hip_atomic_load(g.part + ((int64_t)nb * g.split + p) * (W * 256) + tid, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int p = 0; p < kFewMaxSplit; ++p)
                if (p < g.split)
                    sum += v[p];
        }
    }
    if (tid < W * 256) {
        const int el = tid % 256, t = (el / 4) % 16, col = nb * NC + tid / 256 * 16 + 4 * (el / 64) + el % 4;
        if (t < g.T)
            ((uint16_t*)g.y)[(int64_t)t * g.d + col] = f32_to_bf16_bits(sum);
    }
}

}  // namespace

bool few_routes_itself(int d, int E)
{
    // Routing in every workgroup against the router as a launch before (4-bit
    // layers, 8 tokens, us): d = 1024, E = 128 22.5 / 24.0; 2048, 64 34.0 / 35.8;
    // 2048, 128 37.0 / 38.4; 4096, 64 47.9 / 49.5; 4096, 128 52.2 / 53.5; 4096, 96
    // with 2 tokens 30.6 / 30.9. The gain shrinks with the router's size, which
    // every workgroup reads; beyond these sizes, and for more than 128 experts
    // (the LDS sums above), the router is launched.
    return E <= 128 && (int64_t)d * E <= (int64_t)1 << 19;
}

hipError_t launch_few_gate_up(const FewArgs& a, int cus, hipStream_t s)
{
    const dim3 grid(cus), block(kThreads);
    if (a.m_gu)
        hipLaunchKernelGGL(few_gate_up_kernel<kMx4>, grid, block, 0, s, a);
    else if (a.s_gu)
        hipLaunchKernelGGL(few_gate_up_kernel<kFp8>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(few_gate_up_kernel<kBf16>, grid, block, 0, s, a);
    return hipGetLastError();
}

int few_down_columns(int mx4)
{
    return 16 * down_groups(mx4 ? kMx4 : kBf16);
}

int few_down_split(int d, int mx4, int cus)
{
    // A workgroup per compute unit, in at most kFewMaxSplit parts: reading the
    // weights at full rate takes them all (d = 2048: 49 us with 128 workgroups of
    // whole columns, 30 with 256).
    return std::max(1, std::min(kFewMaxSplit, cus / (d / few_down_columns(mx4))));
}

hipError_t launch_few_down(const FewArgs& a, hipStream_t s)
{
    const dim3 grid(a.d / few_down_columns(a.m_gu != nullptr) * a.split), block(kThreads);
    auto k = a.m_gu   ? (a.T <= 8 ? few_down_kernel<kMx4, 1> : few_down_kernel<kMx4, 2>)
             : a.s_gu ? (a.T <= 8 ? few_down_kernel<kFp8, 1> : few_down_kernel<kFp8, 2>)
                      : (a.T <= 8 ? few_down_kernel<kBf16, 1> : few_down_kernel<kBf16, 2>);
    hipLaunchKernelGGL(k, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace cmoe
