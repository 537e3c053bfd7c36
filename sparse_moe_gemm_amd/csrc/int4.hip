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
// (m: the place of four mantissa bits in both halves, b: 16.0 in both).
__device__ __forceinline__ bf16x8 codes8(uint32_t w, uint32_t m, uint32_t b)
{
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

// Assignments by expert: row r is the r-th of them, expert by expert; a pass is
// up to CP of them with the same expert.
struct Pass {
    int16_t expert, start, count, unused;
};
struct Row {
    uint32_t x;       // byte offset of its row of x
    int16_t assigned;  // t * k + j
    int16_t token;
    float w;
    uint32_t unused;
};
struct __align__(16) Passes {
    Row row[kMaxRows];
    Pass pass[kMaxRows];
    int32_t key[kMaxRows];
    uint32_t counts[kMaxRows];
    uint32_t mask[kMaxRows / 32];
    int32_t none;    // some assignment is of no expert
    int32_t twins;   // some token has an expert in two slots
};

constexpr int kKeyBits = 7;  // an assignment's key: expert, then index
static_assert(kMaxRows == 1 << kKeyBits, "keys");

// Number of passes. An id outside 0..E-1 is no expert's: in no pass. An
// assignment's rank is the number of smaller keys; the threads share the
// comparisons, W / 2 of them for each assignment.
template <int CP, int W>
__device__ __forceinline__ int build_passes(Passes& p, const Int4Args& a)
{
    const int tid = threadIdx.x, A = a.T * a.k;
    const uint32_t pitch = (uint32_t)a.K * 2;
    if (!a.ids) {
        if (tid < A)
            p.row[tid] = Row{(uint32_t)tid * pitch, (int16_t)tid, (int16_t)tid, 0.0f, 0u};
        if (tid * CP < A)
            p.pass[tid] = Pass{0, (int16_t)(tid * CP), (int16_t)min(CP, A - tid * CP), 0};
        if (tid == 0)
            p.none = 0;
        __syncthreads();
        return (A + CP - 1) / CP;
    }
    int e = a.E + 1;  // behind the last assignment
    float weight = 0.0f;
    if (tid < A) {
        const int id = a.ids[tid];
        if (a.w)
            weight = a.w[tid];
        e = (uint32_t)id < (uint32_t)a.E ? id : a.E;
    }
    if (tid < kMaxRows) {
        p.key[tid] = (e << kKeyBits) | tid;
        p.counts[tid] = 0;
    }
    if (tid < kMaxRows / 32)
        p.mask[tid] = 0;
    if (tid == 0)
        p.none = p.twins = 0;
    __syncthreads();
    if (tid < A && e == a.E)
        p.none = 1;
    const int mine = tid % kMaxRows;
    if (mine < A) {
        const int key = p.key[mine], lo = key & -kMaxRows, hi = lo + kMaxRows;
        uint32_t n = 0;  // keys below mine, of lower experts, of experts up to mine
        for (int b = tid / kMaxRows * 4; b < A; b += W / 2 * 4) {
            const int4 o = *(const int4*)&p.key[b];
            n += (o.x < key) + (o.y < key) + (o.z < key) + (o.w < key);
            n += ((o.x < lo) + (o.y < lo) + (o.z < lo) + (o.w < lo)) << 8;
            n += ((o.x < hi) + (o.y < hi) + (o.z < hi) + (o.w < hi)) << 16;
        }
        atomicAdd(&p.counts[mine], n);
    }
    __syncthreads();
    int rank = 0, before = 0, same = 0;
    bool starts = false;
    if (tid < A) {
        const uint32_t n = p.counts[tid];
        rank = n & 255;
        before = rank - (int)(n >> 8 & 255);
        same = (int)(n >> 16) - (int)(n >> 8 & 255);
        const int t = (int)((uint32_t)tid / (uint32_t)a.k), slot = tid - t * a.k;
        p.row[rank] = Row{(uint32_t)(a.x_per_slot ? tid : t) * pitch, (int16_t)tid, (int16_t)t, weight, 0u};
        starts = e < a.E && before % CP == 0;
        if (starts)
            atomicOr(&p.mask[rank >> 5], 1u << (rank & 31));
        for (int j = 1; j <= slot; ++j)
            if (e < a.E && p.key[tid - j] >> kKeyBits == e)
                p.twins = 1;
    }
    __syncthreads();
    int n = 0, at = 0;
#pragma unroll
    for (int q = 0; q < kMaxRows / 32; ++q) {
        const uint32_t m = p.mask[q];
        n += __popc(m);
        at += q < (rank >> 5) ? __popc(m) : q == (rank >> 5) ? __popc(m & ((1u << (rank & 31)) - 1u)) : 0;
    }
    if (starts)
        p.pass[at] = Pass{(int16_t)e, (int16_t)rank, (int16_t)min(CP, same - before), 0};
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

// A wave-uniform address in scalar registers, named as global memory (a generic
// one would be loaded through the flat path, whose waits are for everything).
typedef const __attribute__((address_space(1))) uint8_t* Global;
__device__ __forceinline__ Global uniform(const uint8_t* p)
{
    const uint64_t a = (uint64_t)(uintptr_t)p;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
    return (Global)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

// Barrier for LDS data; loads from global memory stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What a wave holds of a unit: RT tiles of codes with their groups, NT groups of
// RL rows of x in RL / 4 loads each.
template <int RL, int NT, int RT, int MG>
struct Unit {
    typedef uint32_t Meta __attribute__((ext_vector_type(MG)));
    Vec16 c[RT], x[NT][RL / 4];
    Meta m[RT];
};

// Where a wave loads next: unit u of RT tiles, its codes and groups at scalar
// addresses (32-bit offsets per lane), x rows at the offsets xo.
template <int NT>
struct Cursor {
    Global c, m;
    int u;
    uint32_t xo[NT];
};

template <int NT, int MG>
__device__ __forceinline__ void aim(Cursor<NT>& at, const Int4Args& a, int64_t tile, int units, int u)
{
    at.c = uniform((const uint8_t*)a.codes + (tile * units + u) * 1024);
    at.m = uniform((const uint8_t*)a.meta + (tile * units + u) * (64 * MG));
    at.u = u;
}

// x as a buffer: loads past its end give zeros and touch no memory; a lane
// without a row gets such an offset.
constexpr uint32_t kNoRow = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t x_buffer(const Int4Args& a)
{
    const uint32_t rows = (uint32_t)(a.x_per_slot ? a.T * a.k : a.T);
    return __builtin_amdgcn_make_buffer_rsrc((void*)a.x, 0, (int)(rows * (uint32_t)a.K * 2), 0x00020000);
}

// Loads unit at.u + j (behind the tile's last unit that one again, times a scale
// of 0). A load of x takes 64 lanes x 16 bytes whatever the rows are, and
// at 16 rows the four steps' loads cost more than the codes; with RL = 4 (8)
// rows one load holds all four (two) steps, lanes l%16 = RL i + row those of the
// i-th, and row_rotate brings a step to lanes 0..RL-1 of each 16 (7 tokens on 8
// experts, down: 62 -> XX us). Unconditional, also behind the row (K % 128: its
// end again, times a scale of 0), so that waits count exactly.
template <int RL, int NT, int RT, int MG>
__device__ __forceinline__ void load_unit(Unit<RL, NT, RT, MG>& v, const Int4Args& a, __amdgpu_buffer_rsrc_t xb,
                                          const Cursor<NT>& at, int units, int j)
{
    typedef const __attribute__((address_space(1))) Vec16* Codes;
    typedef const __attribute__((address_space(1))) typename Unit<RL, NT, RT, MG>::Meta* Metas;
    const uint32_t lane = threadIdx.x % kWave, co = lane * 16, mo = (lane & 15) * 4 * MG;
    const int u = min(at.u + j, units - 1), d = u - at.u;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        v.c[r] = __builtin_nontemporal_load((Codes)(at.c + ((int64_t)r * units + d) * 1024 + co));
        v.m[r] = *(Metas)(at.m + ((int64_t)r * units + d) * (64 * MG) + mo);
    }
#pragma unroll
    for (int i = 0; i < RL / 4; ++i) {
        if constexpr (RL == 16) {
            const int k = min(u * kUnitK + 32 * i, a.K - 32) * 2;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                v.x[n][i] = __builtin_bit_cast(Vec16, __builtin_amdgcn_raw_buffer_load_b128(xb, (int)at.xo[n], k, 0));
        } else {
            const int k = min(u * kUnitK + 32 * (i * (16 / RL) + (int)(lane & 15) / RL), a.K - 32) * 2;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                v.x[n][i] = __builtin_bit_cast(Vec16, __builtin_amdgcn_raw_buffer_load_b128(xb, (int)at.xo[n] + k, 0, 0));
        }
    }
}

// Lane i of each 16 gets lane (i + N) % 16's.
template <int N>
__device__ __forceinline__ Vec16 row_rotate(const Vec16& v)
{
    if constexpr (N == 0) {
        return v;
    } else {
        Vec16 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // row_ror: lane i from lane i - (16 - N)
            o[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[i], 0x120 + 16 - N, 0xF, 0xF, false);
        return o;
    }
}

// The x fragment of step S.
template <int RL, int S>
__device__ __forceinline__ bf16x8 x_step(const Vec16 (&x)[RL / 4])
{
    constexpr int per = 16 / RL;
    return as_bf16x8(row_rotate<RL % 16 * (S % per)>(x[S / per]));
}

struct Consts {
    uint32_t fields, sixteen;  // as codes8 takes them, in vector registers
    uint32_t f16;              // all ones: the scales are fp16
    __device__ __forceinline__ explicit Consts(const Int4Args& a)
        : fields(0x00780078u), sixteen(0x41804180u), f16(a.scales_f16 ? ~0u : 0u)
    {
        asm volatile("" : "+v"(fields), "+v"(sixteen));
    }
};

// tot += s * sum (q - z) x over the unit's groups (live 0: times 0 instead). A
// group's sums are done with before the next one's begin, and the set before it
// is loaded again: fewer registers, and no copies of what is in flight.
template <int RL, int NT, int RT, int MG>
__device__ __forceinline__ void multiply_unit(const Unit<RL, NT, RT, MG>& v, const Consts& k, floatx4 (&tot)[RT][NT],
                                              uint32_t live)
{
    const bf16x8 ones = as_bf16x8(Vec16{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};
    floatx4 acc[RT][NT], sum[NT];
    auto step = [&](auto sc) {
        constexpr int S = decltype(sc)::value;
        constexpr bool begins = S % (4 / MG) == 0, ends = S % (4 / MG) == 4 / MG - 1;
        bf16x8 x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            x[n] = x_step<RL, S>(v.x[n]);
            sum[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[n], ones, begins ? zero : sum[n], 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const bf16x8 q = codes8(v.c[r][S], k.fields, k.sixteen);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[n], q, begins ? zero : acc[r][n], 0, 0, 0);
        }
        if constexpr (ends) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t w = v.m[r][S / (4 / MG)];
                const float z = __uint_as_float(w & 0xFFFF0000u);
                // the scale of either type by a bit select: no branch between the loads
                const uint32_t half = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)w));
                const float s = __uint_as_float(((half & k.f16) | ((w << 16) & ~k.f16)) & live);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tot[r][n][i] = fmaf(s, fmaf(-z, sum[n][i], acc[r][n][i]), tot[r][n][i]);
                    asm volatile("" : "+v"(tot[r][n]));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    step(std::integral_constant<int, 0>());
    step(std::integral_constant<int, 1>());
    step(std::integral_constant<int, 2>());
    step(std::integral_constant<int, 3>());
}

template <int NT, int RT>
__device__ __forceinline__ void clear(floatx4 (&tot)[RT][NT])
{
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            tot[r][n] = floatx4{0.f, 0.f, 0.f, 0.f};
}

// Lane l's element i of a tile's totals: x row 16 n + 4 (l / 16) + i, weight row l % 16.
template <int NT, int RT>
__device__ __forceinline__ void store_totals(float* red, const floatx4 (&tot)[RT][NT])
{
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[(r * NT + n) * 256 + i * kWave + lane] = tot[r][n][i];
}

// x row and weight row of value v of a tile's totals.
__device__ __forceinline__ int total_row(int v) { return (v >> 8) * 16 + ((v & 63) >> 4) * 4 + ((v >> 6) & 3); }
__device__ __forceinline__ int total_col(int v) { return v & 15; }

// Plain and SwiGLU. A work item is a pass and RT tiles of 16 rows. A workgroup
// takes a contiguous share of the items; of these every wave takes whole ones, one
// after another, and stores them itself, as long as there are W more. The units
// of the rest are one line, cut into W pieces: a piece is part of two items at
// most, and what the waves summed of an item is added through LDS, in wave order.
// So all waves stream all the time, and meet once. Units go by Q in a turn (the
// last ones past the row count for nothing): as the products of one are done,
// the same one of the next turn is loaded.
template <bool SWIGLU, int RL, int NT, int RT, int MG, int W, int Q>
__global__ __launch_bounds__(W * kWave) void int4_kernel(Int4Args a)
{
    static_assert(NT == 1 || RL == 16, "rows");
    constexpr int CP = RL * NT, NV = RT * NT * 256;
    __shared__ Passes ps;
    __shared__ int first_item[W];
    __shared__ float red[W][2][NV];

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wv = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int units = units_of(a.K), turns = (units + Q - 1) / Q, tiles = tiles_of(a.N, SWIGLU), groups = tiles / RT;
    const uint32_t items = (uint32_t)(build_passes<CP, W>(ps, a) * groups);
    const int M = SWIGLU ? a.N / 2 : a.N;
    const Consts consts(a);
    const __amdgpu_buffer_rsrc_t xb = x_buffer(a);

    const uint32_t share = items / gridDim.x, more = items % gridDim.x;
    const int mine = (int)(share + (blockIdx.x < more ? 1 : 0));
    const int i0 = (int)(blockIdx.x * share + min(blockIdx.x, more));
    const int full = mine / W, rest = mine % W, rest0 = i0 + full * W;
    const uint32_t line = (uint32_t)(rest * turns);
    const int cut0 = (int)(line * wv / W), cut1 = (int)(line * (wv + 1) / W);  // this wave's piece
    const int first = (int)((uint32_t)cut0 / (uint32_t)turns);               // its first item of the rest
    const int segments = full + (cut1 > cut0) + (cut1 > (first + 1) * turns);
    if (lane == 0)
        first_item[wv] = first;
    struct Segment {
        int item, q0, q1;
    };
    auto segment = [&](int k) {
        if (k < full)
            return Segment{i0 + k * W + wv, 0, turns};
        const int m = first + k - full;
        return Segment{rest0 + m, max(cut0 - m * turns, 0), min(cut1 - m * turns, turns)};
    };

    // The load cursor. Past the last segment it stays where it is.
    Cursor<NT> at;
    int lk = 0, lend = 0;
    auto aim_at = [&]() {
        const Segment s = segment(lk);
        const int pass = (int)((uint32_t)s.item / (uint32_t)groups), tg = s.item - pass * groups;
        const Pass p = ps.pass[pass];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = n * 16 + (lane % RL);
            at.xo[n] = row >= p.count ? kNoRow : ps.row[p.start + row].x + (lane >> 4) * 16;
        }
        aim<NT, MG>(at, a, (int64_t)__builtin_amdgcn_readfirstlane((int)p.expert) * tiles + tg * RT, units, s.q0 * Q);
        lend = s.q1 * Q;
    };
    auto advance = [&]() {
        if (at.u + Q < lend) {
            at.u += Q;
            at.c += Q * 1024;
            at.m += Q * 64 * MG;
        } else if (lk + 1 < segments) {
            ++lk;
            aim_at();
        }
    };
    // Row `row` of a pass, weight rows col of the item's RT tiles: sums v[r].
    auto store = [&](int pass, int tg, int row, int col, const float (&v)[RT]) {
        const Pass p = ps.pass[pass];
        if (row >= p.count)
            return;
        const int64_t y = (int64_t)ps.row[p.start + row].assigned * M;
        if constexpr (SWIGLU) {
            const int n = tg * 16 + col;
            if (n < M)
                store_y(a, y + n, silu_f32(v[0]) * v[1]);
        } else {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int n = (tg * RT + r) * 16 + col;
                if (n < M)
                    store_y(a, y + n, v[r]);
            }
        }
    };

    if (segments > 0) {
        aim_at();
        Unit<RL, NT, RT, MG> v[Q];
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            load_unit(v[j], a, xb, at, units, j);
            __builtin_amdgcn_sched_barrier(0);  // in this order, for the waits in the loop
        }
        floatx4 tot[RT][NT];
        clear(tot);
        int k = 0;
        Segment now = segment(0);
        for (;;) {
            advance();
#pragma unroll
            for (int j = 0; j < Q; ++j) {
                multiply_unit(v[j], consts, tot, j == 0 || now.q0 * Q + j < units ? ~0u : 0u);
                load_unit(v[j], a, xb, at, units, j);
            }
            if (++now.q0 < now.q1)
                continue;
            if (k < full) {
                const int pass = (int)((uint32_t)now.item / (uint32_t)groups), tg = now.item - pass * groups;
#pragma unroll 1
                for (int t = 0; t < NT; ++t)
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        float w[RT];
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            w[r] = NT == 1 ? tot[r][0][i] : tot[r][t][i];
                        store(pass, tg, t * 16 + (lane >> 4) * 4 + i, lane & 15, w);
                    }
            } else {
                store_totals(red[wv][k - full], tot);
            }
            clear(tot);
            if (++k == segments)
                break;
            now = segment(k);
        }
    }
    if (rest > 0) {
        lds_barrier();
        const int firsts = first_item[lane % W];
        for (int i = tid; i < rest * NT * 256; i += W * kWave) {
            const int m = __builtin_amdgcn_readfirstlane(i / (NT * 256)), v = i % (NT * 256);
            float sum[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
                sum[r] = 0.0f;
#pragma unroll 1
            for (int w0 = 0; w0 < W; w0 += 4) {  // the waves with a piece of item m, in order
                float p[4][RT];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int w = w0 + j, c0 = (int)(line * w / W), c1 = (int)(line * (w + 1) / W);
                    const bool has = c0 < c1 && c0 < (m + 1) * turns && c1 > m * turns;
                    const float* t = &red[w][has ? m - __builtin_amdgcn_readlane(firsts, w) : 0][v];
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        p[j][r] = has ? t[r * NT * 256] : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        sum[r] += p[j][r];
            }
            const int pass = (int)((uint32_t)(rest0 + m) / (uint32_t)groups);
            store(pass, rest0 + m - pass * groups, total_row(v), total_col(v), sum);
        }
    }
    if (ps.none)  // assignments of no expert: rows of zeros
        for (int p = 0; p < a.T * a.k; ++p)
            if (ps.key[p] >> kKeyBits == a.E)
                for (int n = blockIdx.x * W * kWave + tid; n < M; n += gridDim.x * W * kWave)
                    store_y(a, (int64_t)p * M + n, 0.0f);
}

// y[t] = sum_j w[t][j] W[ids[t][j]] x. A workgroup takes RT tiles and all tokens;
// the units of all passes are one line, cut into W pieces, one per wave. At the
// end of a pass, or of its piece, a wave adds w times what it summed to its own
// sums of the tokens in LDS, and these are added once, in wave order.
template <int RL, int RT, int MG, int W, int Q>
__global__ __launch_bounds__(W * kWave) void int4_sum_kernel(Int4Args a)
{
    __shared__ Passes ps;
    extern __shared__ float sums[];  // [W][T][16 RT]
    constexpr int C = 16 * RT;

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wv = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int units = units_of(a.K), turns = (units + Q - 1) / Q, tiles = tiles_of(a.N, 0);
    const int tg = blockIdx.x;
    for (int i = tid; i < W * a.T * C; i += W * kWave)
        sums[i] = 0.0f;
    const uint32_t line = (uint32_t)(build_passes<RL, W>(ps, a) * turns);
    const int cut0 = (int)(line * wv / W), cut1 = (int)(line * (wv + 1) / W);
    const Consts consts(a);
    const __amdgpu_buffer_rsrc_t xb = x_buffer(a);

    if (cut1 > cut0) {
        // The load cursor: `left` turns to the end of the piece, where it stays.
        Cursor<1> at;
        int lp = (int)((uint32_t)cut0 / (uint32_t)turns), left = cut1 - cut0;
        auto aim_at = [&](int q) {
            const Pass p = ps.pass[lp];
            at.xo[0] = lane % RL >= p.count ? kNoRow : ps.row[p.start + lane % RL].x + (lane >> 4) * 16;
            aim<1, MG>(at, a, (int64_t)__builtin_amdgcn_readfirstlane((int)p.expert) * tiles + tg * RT, units, q * Q);
        };
        auto advance = [&]() {
            if (--left <= 0)
                return;
            if (at.u + Q < units) {
                at.u += Q;
                at.c += Q * 1024;
                at.m += Q * 64 * MG;
            } else {
                ++lp;
                aim_at(0);
            }
        };
        int p = lp, q = cut0 - p * turns, todo = cut1 - cut0;
        aim_at(q);
        Unit<RL, 1, RT, MG> v[Q];
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            load_unit(v[j], a, xb, at, units, j);
            __builtin_amdgcn_sched_barrier(0);  // in this order, for the waits in the loop
        }
        floatx4 sum[RT][1];
        clear(sum);
        for (;;) {
            advance();
#pragma unroll
            for (int j = 0; j < Q; ++j) {
                multiply_unit(v[j], consts, sum, j == 0 || q * Q + j < units ? ~0u : 0u);
                load_unit(v[j], a, xb, at, units, j);
            }
            if (++q < turns && --todo > 0)
                continue;
            // a token has one row in a pass, unless it has the expert twice: then
            // the lane groups take turns
            const Pass now = ps.pass[p];
            const int groups = ps.twins ? 4 : 1;
#pragma unroll 1
            for (int g = 0; g < groups; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = (lane >> 4) * 4 + i;
                    if (row < now.count && (groups == 1 || (lane >> 4) == g)) {
                        const Row o = ps.row[now.start + row];
                        float* y = sums + (wv * a.T + o.token) * C + (lane & 15);
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            y[r * 16] = fmaf(o.w, sum[r][0][i], y[r * 16]);
                    }
                }
            clear(sum);
            if (q == turns) {
                q = 0;
                ++p;
                if (--todo <= 0)
                    break;
            } else {
                break;
            }
        }
    }
    lds_barrier();
    for (int v = tid; v < a.T * C; v += W * kWave) {
        const int n = tg * C + v % C;
        float s = sums[v];
#pragma unroll
        for (int w = 1; w < W; ++w)
            s += sums[w * a.T * C + v];
        if (n < a.N)
            store_y(a, (int64_t)(v / C) * a.N + n, s);
    }
}

// go(MG): with the number of groups of a unit at compile time.
template <class Go>
hipError_t by_groups(int group, Go go)
{
    switch (unit_groups(group)) {
    case 4:
        go(std::integral_constant<int, 4>());
        break;
    case 2:
        go(std::integral_constant<int, 2>());
        break;
    default:
        go(std::integral_constant<int, 1>());
    }
    return hipGetLastError();
}

template <bool SWIGLU, int RL, int NT, int RT, int W, int Q = 2>
hipError_t launch(const Int4Args& a, int per_cu, int cus, hipStream_t s)
{
    const int groups = tiles_of(a.N, SWIGLU) / RT, A = a.T * a.k, CP = RL * NT;
    // at most: every expert's passes
    const int64_t passes = a.ids ? std::min(a.E, A) + A / CP : (A + CP - 1) / CP;
    const unsigned grid = (unsigned)std::min<int64_t>(passes * groups, (int64_t)cus * per_cu);
    return by_groups(a.group, [&](auto mg) {
        hipLaunchKernelGGL((int4_kernel<SWIGLU, RL, NT, RT, decltype(mg)::value, W, Q>), dim3(grid), dim3(W * kWave), 0, s, a);
    });
}

template <int RL, int RT, int Q>
hipError_t launch_sum(const Int4Args& a, hipStream_t s)
{
    constexpr int W = 16;
    const unsigned grid = (unsigned)(tiles_of(a.N, 0) / RT);
    const size_t lds = (size_t)W * a.T * 16 * RT * sizeof(float);
    return by_groups(a.group, [&](auto mg) {
        hipLaunchKernelGGL((int4_sum_kernel<RL, RT, decltype(mg)::value, W, Q>), dim3(grid), dim3(W * kWave), lds, s, a);
    });
}

// Two tiles per workgroup where that leaves one for every compute unit and the
// sums of the tokens fit (N = 8192: 36.7 -> 27.7 us; with too few, N = 4096, 53 ->
// 67). Four units in a turn for long rows (K = 14336: 53 -> 49 us; K = 2048: 8.6 ->
// 9.8).
template <int RL>
hipError_t launch_sums(const Int4Args& a, int cus, hipStream_t s)
{
    if (tiles_of(a.N, 0) / 2 >= cus && a.T <= 64)
        return launch_sum<RL, 2, 2>(a, s);
    if constexpr (RL < 16) {
        if (a.K >= 8192)
            return launch_sum<RL, 1, 4>(a, s);
    }
    return launch_sum<RL, 1, 2>(a, s);
}

// Many items: four workgroups of four waves per compute unit, whose starts and
// ends overlap the others' streaming (16 tokens over 128 experts of 1536 x 2048:
// 23.3 us, two of eight waves 24.7, one of sixteen 28; 8 experts of 28672 x 4096, one
// token: 26.5, 29.6, 31.6). Few: eight waves for an item (one token, 4096 x 4096: 5.8
// us, 6.5 with four; K = 14336: 10.8, 14.2).
template <int RL, int NT>
hipError_t launch_items(const Int4Args& a, int cus, hipStream_t s)
{
    const int A = a.T * a.k, CP = RL * NT;
    const int64_t passes = a.ids ? std::min(a.E, A) : (A + CP - 1) / CP;
    const int64_t tiles = passes * tiles_of(a.N, a.swiglu);
    if constexpr (NT == 1) {
        if (a.swiglu)
            return tiles / 2 >= 2 * cus ? launch<true, RL, 1, 2, 4>(a, 4, cus, s) : launch<true, RL, 1, 2, 8>(a, 2, cus, s);
        if (tiles / 2 >= 2 * cus)
            return launch<false, RL, 1, 2, 4>(a, 4, cus, s);
        return tiles >= 2 * cus ? launch<false, RL, 1, 1, 4>(a, 4, cus, s) : launch<false, RL, 1, 1, 8>(a, 2, cus, s);
    } else {
        if (a.swiglu)
            return launch<true, 16, NT, 2, 4, 1>(a, 2, cus, s);
        if (tiles / 2 >= 2 * cus)
            return launch<false, 16, NT, 2, 4, 1>(a, 2, cus, s);
        return launch<false, 16, NT, 1, 4, 1>(a, 3, cus, s);
    }
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
    const int A = a.T * a.k;
    // The rows that passes hold: with ids, the mean of the chosen experts' (if all
    // choose alike), in eighths. Fewer rows per pass make loads of x cheaper, but
    // an expert of more is read again: passes of 4 up to 1.6 rows, of 8 up to 4.5 (16
    // tokens on 8 experts, 4 rows each: 8 rows 91.6 us, 4 rows 122, 16 rows 91.8).
    const int rows = !a.ids ? a.T * 8 : a.T <= 4 ? 8 : std::min(a.T * 8, A * 8 / std::min(a.E, A));
    if (a.w) {
        if (rows <= 13)
            return launch_sums<4>(a, cus, s);
        return rows <= 36 ? launch_sums<8>(a, cus, s) : launch_sums<16>(a, cus, s);
    }
    if (rows <= (a.ids ? 13 : 32))
        return launch_items<4, 1>(a, cus, s);
    if (rows <= (a.ids ? 36 : 64))
        return launch_items<8, 1>(a, cus, s);
    if (rows <= 128)
        return launch_items<16, 1>(a, cus, s);
    return rows <= 256 ? launch_items<16, 2>(a, cus, s) : launch_items<16, 4>(a, cus, s);
}

}  // namespace cmoe
