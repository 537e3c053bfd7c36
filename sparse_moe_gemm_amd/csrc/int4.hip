// int4.hip - products of a few rows with 4-bit integer weights that have a scale
// and a zero point per group (quant_int4.hip), dense or through expert ids.
//
//   y[a][n] = sum_k (q[e][n][k] - z[e][n][k/g]) * s[e][n][k/g] * x[row(a)][k]
// for assignments a = t * k_slots + j with expert e = ids[a] (dense: a = t, one
// matrix), then one of
//   plain:    y[a][n]
//   SwiGLU:   y[a][c] = SiLU(y[a][c]) * y[a][f + c]       (rows 0..f-1 gate, f..2f-1 up)
//   weighted: y[t][n] = sum_j w[t][j] * y[t * k_slots + j][n]
//
// As few.hip, the work is reading the weights of the experts in use once: 16
// weight rows are the second operand of v_mfma_f32_16x16x32_bf16, up to 16 rows
// of x (assignments of one expert) the first.
//   * A code q becomes the bf16 value 16 + q, exact, by placing its four bits in
//     the mantissa of 16 (a shift and an and-or for two codes). The matrix unit
//     sums (16 + q) x over a group in fp32; with the group's sum of x, from a
//     product with ones, the group adds s * (sum (16 + q) x - (16 + z) sum x) to
//     the row's total. So the weights are never rounded: each term is exact
//     before the fp32 sums.
//   * A unit is 16 rows x 128 k: one KiB in which lane l's 16 bytes are row l%16,
//     k = 32 s + 8 (l/16) .. +8 for the four MFMA steps s, so that a step's 32 k
//     lie in one group; its scales and zero points are a dword per row and group.
//   * The waves of a work item split its units and add their totals through LDS
//     in wave order: the result does not depend on what else runs.
#include "common.hpp"

namespace cmoe {

namespace {

constexpr int kUnitK = 128;
constexpr int kMaxRows = kInt4Rows;

enum Form { kPlain = 0, kSwiglu = 1, kWeighted = 2 };

__host__ __device__ __forceinline__ int units_of(int K) { return (K + kUnitK - 1) / kUnitK; }

// Tiles of 16 rows, an even number (a work item takes one or two). SwiGLU: gate
// and up tiles of the same 16 columns in turn.
__host__ __device__ __forceinline__ int tiles_of(int N, int swiglu)
{
    return swiglu ? 2 * ((N / 2 + 15) / 16) : ((N + 15) / 16 + 1) / 2 * 2;
}

// Groups of a unit: 32, 64 or 128 k each (longer groups repeat).
__host__ __device__ __forceinline__ int unit_groups(int group) { return group == 32 ? 4 : group == 64 ? 2 : 1; }

// Eight codes of a word as bf16 16 + q: element 2p is nibble p, 2p + 1 nibble p + 4.
__device__ __forceinline__ bf16x8 codes8(uint32_t w)
{
    const uint32_t m = 0x00780078u, b = 0x41804180u;
    const Vec16 v = {((w << 3) & m) | b, ((w >> 1) & m) | b, ((w >> 5) & m) | b, ((w >> 9) & m) | b};
    return as_bf16x8(v);
}

// Codes and groups of the caller's rows in the layout above; one thread per
// word of codes, then one per scale.
__global__ __launch_bounds__(256) void int4_pack_kernel(Int4Pack p, int units, int tiles, int mg)
{
    const int64_t words = (int64_t)p.E * tiles * units * 256;
    const int64_t metas = (int64_t)p.E * tiles * units * 16 * mg;
    const int gpr = p.K / p.group;
    const int f = p.N / 2;
    auto source_row = [&](int tile, int r) {  // -1: none
        if (p.swiglu) {
            const int c = (tile >> 1) * 16 + r;
            return c < f ? (tile & 1) * f + c : -1;
        }
        const int n = tile * 16 + r;
        return n < p.N ? n : -1;
    };
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words + metas; i += (int64_t)gridDim.x * 256) {
        if (i < words) {
            const int s = (int)(i & 3), lane = (int)(i >> 2) & 63;
            const int64_t block = i >> 8;
            const int u = (int)(block % units), tile = (int)(block / units % tiles);
            const int64_t e = block / units / tiles;
            const int n = source_row(tile, lane & 15), k = u * kUnitK + 32 * s + 8 * (lane >> 4);
            uint32_t out = 0;
            if (n >= 0 && k < p.K) {
                const uint8_t* src = p.codes + ((e * p.N + n) * p.K + k) / 2;
#pragma unroll
                for (int b = 0; b < 4; ++b) {  // codes 2b and 2b + 1
                    out |= (uint32_t)(src[b] & 15) << (4 * b);
                    out |= (uint32_t)(src[b] >> 4) << (4 * b + 16);
                }
            }
            p.out_codes[i] = out;
        } else {
            const int64_t m = i - words;
            const int g = (int)(m % mg), r = (int)(m / mg) & 15;
            const int64_t block = m / mg / 16;
            const int u = (int)(block % units), tile = (int)(block / units % tiles);
            const int64_t e = block / units / tiles;
            const int n = source_row(tile, r), k = u * kUnitK + g * (kUnitK / mg);
            uint32_t out = 0;
            if (n >= 0 && k < p.K) {
                const int64_t at = (e * p.N + n) * gpr + k / p.group;
                const uint32_t z = p.zeros ? p.zeros[at] & 15u : 8u;
                out = p.scales[at] | (0x4180u | (z << 3)) << 16;  // scale, 16 + z as bf16
            }
            p.out_meta[m] = out;
        }
    }
}

// Assignments by expert: order[] lists them expert by expert; pass i is up to
// CP of them, from order[start[i]], with the same expert.
struct Passes {
    int32_t id[kMaxRows];
    uint32_t mask[kMaxRows / 32];
    int16_t order[kMaxRows], start[kMaxRows], count[kMaxRows], expert[kMaxRows];
};

// Number of passes. An id outside 0..E-1 is no expert's: in no pass.
template <int CP>
__device__ __forceinline__ int build_passes(Passes& p, const Int4Args& a)
{
    const int tid = threadIdx.x, A = a.T * a.k;
    if (!a.ids) {
        if (tid < A)
            p.order[tid] = (int16_t)tid;
        if (tid * CP < A) {
            p.start[tid] = (int16_t)(tid * CP);
            p.count[tid] = (int16_t)min(CP, A - tid * CP);
            p.expert[tid] = 0;
        }
        __syncthreads();
        return (A + CP - 1) / CP;
    }
    if (tid < kMaxRows / 32)
        p.mask[tid] = 0;
    int e = a.E;
    if (tid < A) {
        e = a.ids[tid];
        e = e < 0 || e >= a.E ? a.E : e;
        p.id[tid] = e;
    }
    __syncthreads();
    int below = 0, before = 0, same = 0;
    if (tid < A) {
        for (int b = 0; b < A; ++b) {
            const int o = p.id[b];
            below += o < e;
            same += o == e;
            before += o == e && b < tid;
        }
        p.order[below + before] = (int16_t)tid;
    }
    const bool starts = tid < A && e < a.E && before % CP == 0;
    const int rank = below + before;
    if (starts)
        atomicOr(&p.mask[rank >> 5], 1u << (rank & 31));
    __syncthreads();
    int n = 0, at = 0;
#pragma unroll
    for (int q = 0; q < kMaxRows / 32; ++q) {
        const uint32_t m = p.mask[q];
        n += __popc(m);
        at += q < (rank >> 5) ? __popc(m) : q == (rank >> 5) ? __popc(m & ((1u << (rank & 31)) - 1u)) : 0;
    }
    if (starts) {
        p.start[at] = (int16_t)rank;
        p.count[at] = (int16_t)min(CP, same - before);
        p.expert[at] = (int16_t)e;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(n);
}

// SiLU to a few fp32 steps over the whole range (outputs may be fp32): the
// exponential never overflows.
__device__ __forceinline__ float silu_f32(float z)
{
    const float e = expf(-fabsf(z));
    return (z < 0.0f ? z * e : z) / (1.0f + e);
}

__device__ __forceinline__ void store_y(const Int4Args& a, int64_t at, float v)
{
    if (a.y_f32)
        ((float*)a.y)[at] = v;
    else
        ((uint16_t*)a.y)[at] = f32_to_bf16_bits(v);
}

// A work item is a pass and RT tiles of 16 rows; kw of the workgroup's W waves
// (a power of two) share an item, the workgroup runs W / kw items side by side.
// Weighted: the workgroup takes RT tiles and all passes, keeps every
// assignment's sums in LDS and adds a token's at the end, in slot order.
template <int FORM, int NT, int RT, int MG, int W>
__global__ __launch_bounds__(W * kWave) void int4_kernel(Int4Args a, int kw)
{
    constexpr int CP = 16 * NT;
    constexpr int NV = RT * NT * 256;  // totals of a wave
    __shared__ Passes ps;
    __shared__ float red[W][NV];
    __shared__ float res[FORM == kWeighted ? kMaxRows : 1][16 * RT];
    typedef uint32_t Meta __attribute__((ext_vector_type(MG)));

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wv = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int slot = wv / kw, part = wv % kw, slots = W / kw;
    const int units = units_of(a.K), tiles = tiles_of(a.N, FORM == kSwiglu), groups = tiles / RT;
    const int passes = build_passes<CP>(ps, a);
    const int M = FORM == kSwiglu ? a.N / 2 : a.N;
    const bf16x8 ones = as_bf16x8(Vec16{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};

    // items of this workgroup: plain and SwiGLU: (pass, tiles) pairs in turn;
    // weighted: the passes of one pair of tiles after another
    const int total = FORM == kWeighted ? passes : passes * groups;
    for (int own = blockIdx.x; own < (FORM == kWeighted ? groups : (total + slots - 1) / slots); own += gridDim.x) {
        for (int first = FORM == kWeighted ? 0 : own * slots; first < (FORM == kWeighted ? total : own * slots + 1);
             first += slots) {
            const int item = first + slot;
            const bool live = item < total;
            const int pass = !live ? 0 : FORM == kWeighted ? item : item / groups;
            const int tg = FORM == kWeighted ? own : live ? item % groups : 0;
            const int count = ps.count[pass], start = ps.start[pass];
            floatx4 tot[RT][NT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    tot[r][n] = zero;
            if (live) {
                const int64_t tile0 = (int64_t)ps.expert[pass] * tiles + tg * RT;
                const Vec16* wc = (const Vec16*)a.codes + tile0 * units * kWave + lane;
                const Meta* wm = (const Meta*)a.meta + tile0 * units * 16 + (lane & 15);
                const uint16_t* xr[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int at = ps.order[start + min(n * 16 + (lane & 15), count - 1)];
                    xr[n] = (const uint16_t*)a.x + (int64_t)(a.x_per_slot ? at : at / a.k) * a.K + (lane >> 4) * 8;
                }
                for (int u = part; u < units; u += kw) {
                    Vec16 c[RT], x[NT][4];
                    Meta m[RT];
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        c[r] = __builtin_nontemporal_load(wc + ((int64_t)r * units + u) * kWave);
                        m[r] = wm[((int64_t)r * units + u) * 16];
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            // behind the row (K % 128): any of it, times a scale of 0, with x as 0
                            const int k = u * kUnitK + 32 * s;
                            x[n][s] = *(const Vec16*)(xr[n] + min(k, a.K - 32));
                            if (k >= a.K)
                                x[n][s] = Vec16{0u, 0u, 0u, 0u};
                        }
#pragma unroll
                    for (int g = 0; g < MG; ++g) {
                        floatx4 acc[RT][NT], sum[NT];
#pragma unroll
                        for (int s4 = 0; s4 < 4 / MG; ++s4) {
                            const int s = g * (4 / MG) + s4;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                sum[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x[n][s]), ones,
                                                                                s4 ? sum[n] : zero, 0, 0, 0);
#pragma unroll
                            for (int r = 0; r < RT; ++r) {
                                const bf16x8 q = codes8(c[r][s]);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                        as_bf16x8(x[n][s]), q, s4 ? acc[r][n] : zero, 0, 0, 0);
                            }
                        }
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            uint32_t w;
                            if constexpr (MG == 1)
                                w = m[r][0];
                            else
                                w = m[r][g];
                            const float z = __uint_as_float(w & 0xFFFF0000u);
                            const float s = a.scales_f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)w)
                                                         : __uint_as_float(w << 16);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    tot[r][n][i] = fmaf(s, fmaf(-z, sum[n][i], acc[r][n][i]), tot[r][n][i]);
                        }
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        red[wv][(r * NT + n) * 256 + i * kWave + lane] = tot[r][n][i];
            __syncthreads();
            // value v of a tile: x row 16 n + 4 (l / 16) + i, weight row l % 16
            auto added = [&](int r, int v) {
                float s = red[slot * kw][r * NT * 256 + v];
                for (int w = 1; w < kw; ++w)
                    s += red[slot * kw + w][r * NT * 256 + v];
                return s;
            };
            if (live)
                for (int v = part * kWave + lane; v < NT * 256; v += kw * kWave) {
                    const int row = (v >> 8) * 16 + ((v & 63) >> 4) * 4 + ((v >> 6) & 3), col = v & 15;
                    if (row >= count)
                        continue;
                    const int at = ps.order[start + row];
                    if constexpr (FORM == kSwiglu) {
                        const int n = tg * 16 + col;
                        if (n < M)
                            store_y(a, (int64_t)at * M + n, silu_f32(added(0, v)) * added(1, v));
                    } else {
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const int n = (tg * RT + r) * 16 + col;
                            if constexpr (FORM == kWeighted)
                                res[at][r * 16 + col] = added(r, v);
                            else if (n < M)
                                store_y(a, (int64_t)at * M + n, added(r, v));
                        }
                    }
                }
            __syncthreads();
        }
        if constexpr (FORM == kWeighted) {
            for (int v = tid; v < a.T * 16 * RT; v += W * kWave) {
                const int t = v / (16 * RT), n = own * RT * 16 + v % (16 * RT);
                if (n >= M)
                    continue;
                float s = 0.0f;
                for (int j = 0; j < a.k; ++j) {
                    const int at = t * a.k + j;
                    if ((uint32_t)ps.id[at] < (uint32_t)a.E)
                        s = fmaf(a.w[at], res[at][v % (16 * RT)], s);
                }
                store_y(a, (int64_t)t * M + n, s);
            }
            __syncthreads();  // res is written again
        }
    }
    // assignments of no expert: rows of zeros
    if constexpr (FORM != kWeighted) {
        if (a.ids)
            for (int at = 0; at < a.T * a.k; ++at)
                if (ps.id[at] >= a.E)
                    for (int n = blockIdx.x * W * kWave + tid; n < M; n += gridDim.x * W * kWave)
                        store_y(a, (int64_t)at * M + n, 0.0f);
    }
}

template <int FORM, int NT, int RT, int W>
hipError_t launch(const Int4Args& a, int cus, hipStream_t s)
{
    const int units = units_of(a.K), groups = tiles_of(a.N, FORM == kSwiglu) / RT, A = a.T * a.k;
    int kw = 1;
    while (kw * 2 <= W && kw * 2 <= units)
        kw *= 2;
    // at most: every expert's passes
    const int64_t passes = a.ids ? std::min(a.E, A) + A / (16 * NT) : (A + 16 * NT - 1) / (16 * NT);
    const int64_t items = FORM == kWeighted ? groups : (passes * groups + W / kw - 1) / (W / kw);
    const unsigned grid = (unsigned)std::min<int64_t>(items, (int64_t)cus * (W == 4 ? 8 : 2));
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(grid), dim3(W * kWave), 0, s, a, kw); };
    switch (unit_groups(a.group)) {
    case 4:
        go(int4_kernel<FORM, NT, RT, 4, W>);
        break;
    case 2:
        go(int4_kernel<FORM, NT, RT, 2, W>);
        break;
    default:
        go(int4_kernel<FORM, NT, RT, 1, W>);
    }
    return hipGetLastError();
}

template <int NT>
hipError_t launch_form(const Int4Args& a, int cus, hipStream_t s)
{
    if (a.swiglu)
        return launch<kSwiglu, NT, 2, 4>(a, cus, s);
    if (a.w)
        return launch<kWeighted, NT, 2, NT == 1 ? 16 : 8>(a, cus, s);
    return launch<kPlain, NT, 2, 4>(a, cus, s);
}

}  // namespace

size_t int4_code_bytes(int E, int N, int K, int swiglu)
{
    return (size_t)E * tiles_of(N, swiglu) * units_of(K) * 1024;
}

size_t int4_meta_bytes(int E, int N, int K, int group, int swiglu)
{
    return (size_t)E * tiles_of(N, swiglu) * units_of(K) * 64 * unit_groups(group);
}

hipError_t launch_int4_pack(const Int4Pack& p, hipStream_t s)
{
    hipLaunchKernelGGL(int4_pack_kernel, dim3(4096), dim3(256), 0, s, p, units_of(p.K), tiles_of(p.N, p.swiglu),
                       unit_groups(p.group));
    return hipGetLastError();
}

hipError_t launch_int4_linear(const Int4Args& a, int cus, hipStream_t s)
{
    // x rows of a pass: one group of 16 while an expert has few of them
    const int rows = !a.ids ? a.T : a.T <= 16 ? 1 : 2 * a.T * a.k / a.E;
    if (rows <= 16)
        return launch_form<1>(a, cus, s);
    if (rows <= 32)
        return launch_form<2>(a, cus, s);
    return launch_form<4>(a, cus, s);
}

}  // namespace cmoe
