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
// As few.hip, the work is reading the weights of the experts in use once (from 16
// rows of x on, the products): 16 weight rows are the second operand of
// v_mfma_f32_16x16x32_bf16, 16 rows of x (assignments of one expert) the first.
//   * A code q becomes the bf16 value 16 + q, exact, by placing its four bits in
//     the mantissa of 16 (a shift and an and-or for two codes). The matrix unit
//     sums (16 + q) x over a group in fp32; with the group's sum of x, from a
//     product with ones, the group adds s * (sum (16 + q) x - (16 + z) sum x) to
//     the row's total. So the weights are never rounded: each term is exact
//     before the fp32 sums.
//   * A unit is 16 rows x 128 k: one KiB in which lane l's 16 bytes are row l%16,
//     k = 32 s + 8 (l/16) .. +8 for the four MFMA steps s, so that a step's 32 k
//     lie in one group; its scales and zero points are a dword per row and group.
//   * The waves of a workgroup split its units and add their totals through LDS in
//     wave order: the result does not depend on what else runs.
// One token x 4096 x 4096: 4.9 us with the launch, of which 1.6 are the weights' 9 MB;
// 16 tokens on 8 experts of 28672 x 4096 (SwiGLU, 4 rows each): 86 us, 5.7 TB/s.
// All times here are a call's in a replayed graph of such calls, three sets of inputs
// in turn. Times of two choices are of one card at the time the choice was made; other
// cards, and later changes to what both share, move them by up to a tenth.
#include "common.hpp"

namespace cmoe {

namespace {

constexpr int kUnitK = 128;
constexpr int kMaxRows = kInt4Rows;

__host__ __device__ __forceinline__ int units_of(int K) { return (K + kUnitK - 1) / kUnitK; }

// Tiles of 16 rows, an even number (a work item takes one, two or four). SwiGLU:
// gate and up tiles of the same 16 columns in turn.
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
// exponential never overflows, and a sum that did, to -infinity, gives -0.
__device__ __forceinline__ float silu_f32(float z)
{
    const float e = expf(-fabsf(z));
    return (z < 0.0f ? fmaxf(z, -0x1.fffffep127f) * e : z) / (1.0f + e);
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

// x as a buffer: loads past its end give zeros and touch no memory; a lane
// without a row gets such an offset.
constexpr uint32_t kNoRow = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t x_buffer(const Int4Args& a)
{
    const uint32_t rows = (uint32_t)(a.x_per_slot ? a.T * a.k : a.T);
    return __builtin_amdgcn_make_buffer_rsrc((void*)a.x, 0, (int)(rows * (uint32_t)a.K * 2), 0x00020000);
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

// tot += s * sum (q - z) x over the unit's groups, the x
// fragments from x_of(step, n). A group's sums are done with before the next
// one's begin: fewer registers.
template <int NT, int RT, int MG, class X, class Meta>
__device__ __forceinline__ void multiply_unit(X x_of, const Vec16 (&c)[RT], const Meta (&m)[RT], const Consts& k,
                                              floatx4 (&tot)[RT][NT])
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
            x[n] = x_of(sc, n);
            sum[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[n], ones, begins ? zero : sum[n], 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const bf16x8 q = codes8(c[r][S], k.fields, k.sixteen);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[n], q, begins ? zero : acc[r][n], 0, 0, 0);
        }
        if constexpr (ends) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t w = m[r][S / (4 / MG)];
                const float z = __uint_as_float(w & 0xFFFF0000u);
                // the scale of either type by a bit select, without a branch
                const uint32_t half = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)w));
                const float s = __uint_as_float((half & k.f16) | ((w << 16) & ~k.f16));
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

// A wave's way through units of weights and the x rows that go with them: Q units
// are in flight, and a unit's registers are loaded again before it is multiplied.
//
// In the order of the products' operands, 64 lanes of a load of x would read 16
// rows in pieces of 16 bytes, at four times the cache's time for whole lines, and
// that was most of the work from 8 rows on. So a load takes 256 bytes (a unit's k)
// of each of four rows, L loads for the 4 L rows of a pass (NT times 16 with L = 4),
// and the wave turns them in its own 4 KiB of LDS per 16 rows: piece p of row r is at
// place p ^ r of its row, so that neither side has bank conflicts. Rows of the 16
// that were not loaded hold anything: a row of the products depends on its own
// row of x. (4096 x 4096, 12 rows: 7.9 us in the operands' order, 5.4 so; 64: 20.2, 9.4;
// 14336 x 4096, 128 rows: 69.5, 35.8.)
template <int L, int NT, int RT, int MG, int Q>
struct Stream {
    static_assert(NT == 1 || L == 4, "rows");
    typedef uint32_t Meta __attribute__((ext_vector_type(MG)));
    typedef const __attribute__((address_space(1))) Vec16* Codes;
    typedef const __attribute__((address_space(1))) Meta* Metas;
    struct Slot {
        Vec16 c[RT], x[NT][L];
        Meta m[RT];
    };

    const Int4Args& a;
    const Passes& ps;
    const Consts& consts;
    __amdgpu_buffer_rsrc_t xb;
    int units, lane;
    Vec16* turn;         // [NT][16 rows][16 pieces]
    int to[L], from[4];  // places of load i's piece, of step i's
    uint32_t xo[NT][L];  // offsets of the rows of x
    Global c, m;         // the next unit's codes and groups
    int u;               // and its number

    __device__ __forceinline__ Stream(const Int4Args& args, const Passes& passes, const Consts& k, Vec16* place)
        : a(args), ps(passes), consts(k), xb(x_buffer(args)), units(units_of(args.K)), lane(threadIdx.x % kWave),
          turn(place)
    {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int row = 4 * i + (lane >> 4);
            to[i] = row * 16 + ((lane & 15) ^ row);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            from[i] = (lane & 15) * 16 + ((4 * i + (lane >> 4)) ^ (lane & 15));
    }
    // Next: unit `unit` of pass p and tiles t.. of its expert's `tiles`.
    __device__ __forceinline__ void aim(const Pass& p, int tiles, int t, int unit)
    {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int row = n * 16 + 4 * i + (lane >> 4);
                xo[n][i] = row >= p.count ? kNoRow : ps.row[p.start + row].x + (lane & 3) * 16;
            }
        const int64_t tile = (int64_t)__builtin_amdgcn_readfirstlane((int)p.expert) * tiles + t;
        c = uniform((const uint8_t*)a.codes + (tile * units + unit) * 1024);
        m = uniform((const uint8_t*)a.meta + (tile * units + unit) * (64 * MG));
        u = unit;
    }
    __device__ __forceinline__ void load(Slot& v)
    {
        const uint32_t co = lane * 16, mo = (lane & 15) * 4 * MG;
        // behind the row (K % 128): its end again, times a scale of 0
        const int k = min(u * kUnitK + 32 * ((lane & 15) >> 2), a.K - 32) * 2;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < L; ++i)
                v.x[n][i] = __builtin_bit_cast(Vec16, __builtin_amdgcn_raw_buffer_load_b128(xb, (int)xo[n][i] + k, 0, 0));
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            v.c[r] = __builtin_nontemporal_load((Codes)(c + (int64_t)r * units * 1024 + co));
            v.m[r] = *(Metas)(m + (int64_t)r * units * (64 * MG) + mo);
        }
        c += 1024;
        m += 64 * MG;
        ++u;
        __builtin_amdgcn_sched_barrier(0);  // here and in this order, not behind the products that follow
    }
    // n units from where it aims: next() before each but the first is loaded,
    // done(tot, last) after each is multiplied.
    template <class Next, class Done>
    __device__ __forceinline__ void run(int n, floatx4 (&tot)[RT][NT], Next next, Done done)
    {
        Slot v[Q];
#pragma unroll
        for (int j = 0; j < Q; ++j)
            if (j < n) {
                if (j > 0)
                    next();
                load(v[j]);
            }
        auto step = [&](Slot& slot, bool more, bool last) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < L; ++i)
                    turn[t * 256 + to[i]] = slot.x[t][i];
            Vec16 codes[RT];
            Meta groups[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                codes[r] = slot.c[r];
                groups[r] = slot.m[r];
            }
            if (more) {
                next();
                load(slot);
            }
            multiply_unit<NT, RT, MG>([&](auto s, int t) { return as_bf16x8(turn[t * 256 + from[s()]]); }, codes, groups,
                                      consts, tot);
            done(tot, last);
        };
        int i = 0;
        for (; i + 2 * Q <= n; i += Q) {
#pragma unroll
            for (int j = 0; j < Q; ++j)
                step(v[j], true, false);
        }
#pragma unroll
        for (int j = 0; j < Q; ++j)
            if (i + j < n)
                step(v[j], i + j + Q < n, i + j + 1 == n);
#pragma unroll
        for (int j = 0; j < Q - 1; ++j)
            if (i + Q + j < n)
                step(v[j], false, i + Q + j + 1 == n);
    }
};

// Plain and SwiGLU. A work item is a pass and RT tiles; the waves cut its units
// into W pieces and add their sums in wave order.
template <bool SWIGLU, int L, int NT, int RT, int MG, int W, int Q>
__global__ __launch_bounds__(W * kWave, 2) void int4_kernel(Int4Args a)
{
    static_assert(RT <= 4, "a wave's sums fit where x was");
    __shared__ Passes ps;
    __shared__ Vec16 turn[W][NT * 256];

    const int tid = threadIdx.x;
    const int wv = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int units = units_of(a.K), tiles = tiles_of(a.N, SWIGLU), groups = (tiles + RT - 1) / RT;
    const int items = build_passes<4 * L * NT, W>(ps, a) * groups;
    const int M = SWIGLU ? a.N / 2 : a.N;
    const int u0 = units * wv / W, u1 = units * (wv + 1) / W;
    const Consts consts(a);
    Stream<L, NT, RT, MG, Q> stream(a, ps, consts, turn[wv]);

    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int pass = (int)((uint32_t)item / (uint32_t)groups);
        // the last tiles: a few of the group before again, with the same results
        const int t = min((item - pass * groups) * RT, tiles - RT);
        const Pass p = ps.pass[pass];
        floatx4 tot[RT][NT];
        clear(tot);
        if (u0 < u1) {
            stream.aim(p, tiles, t, u0);
            stream.run(u1 - u0, tot, [] {}, [](auto&, bool) {});
        }
        store_totals((float*)turn[wv], tot);
        lds_barrier();
        for (int v = tid; v < NT * 256; v += W * kWave) {
            float sum[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
                sum[r] = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    sum[r] += ((const float*)turn[w])[r * NT * 256 + v];
            if (total_row(v) < p.count) {
                const int64_t y = (int64_t)ps.row[p.start + total_row(v)].assigned * M;
#pragma unroll
                for (int r = 0; r < RT; r += SWIGLU ? 2 : 1) {
                    const int n = (SWIGLU ? (t + r) / 2 : t + r) * 16 + total_col(v);
                    if (n < M)
                        store_y(a, y + n, SWIGLU ? silu_f32(sum[r]) * sum[r + SWIGLU] : sum[r]);
                }
            }
        }
        lds_barrier();
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
template <int L, int RT, int MG, int W>
__global__ __launch_bounds__(W * kWave) void int4_sum_kernel(Int4Args a)
{
    constexpr int C = 16 * RT;
    __shared__ Passes ps;
    __shared__ Vec16 turn[W][256];
    extern __shared__ float sums[];  // [W][T][C]

    const int tid = threadIdx.x, lane = tid % kWave;
    const int wv = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int units = units_of(a.K), tiles = tiles_of(a.N, 0), t = blockIdx.x * RT;
    for (int i = tid; i < W * a.T * C; i += W * kWave)
        sums[i] = 0.0f;
    const uint32_t line = (uint32_t)(build_passes<4 * L, W>(ps, a) * units);
    const int cut0 = (int)(line * wv / W), cut1 = (int)(line * (wv + 1) / W);
    const Consts consts(a);
    Stream<L, 1, RT, MG, 2> stream(a, ps, consts, turn[wv]);

    if (cut1 > cut0) {
        int loading = (int)((uint32_t)cut0 / (uint32_t)units);  // the pass whose units are loaded next
        int pass = loading, to_end = units - (cut0 - pass * units);
        stream.aim(ps.pass[pass], tiles, t, cut0 - pass * units);
        floatx4 tot[RT][1];
        clear(tot);
        auto next = [&] {
            if (stream.u == units)
                stream.aim(ps.pass[++loading], tiles, t, 0);
        };
        auto done = [&](floatx4(&tot)[RT][1], bool last) {
            if (--to_end > 0 && !last)
                return;
            // a token has one row in a pass, unless it has the expert twice: then
            // the lane groups take turns
            const Pass now = ps.pass[pass++];
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
                            y[r * 16] = fmaf(o.w, tot[r][0][i], y[r * 16]);
                    }
                }
            clear(tot);
            to_end = units;
        };
        stream.run(cut1 - cut0, tot, next, done);
    }
    lds_barrier();
    for (int v = tid; v < a.T * C; v += W * kWave) {
        const int n = t * 16 + v % C;
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

template <bool SWIGLU, int L, int NT, int RT, int W, int Q>
hipError_t launch(const Int4Args& a, int per_cu, int cus, hipStream_t s)
{
    const int groups = (tiles_of(a.N, SWIGLU) + RT - 1) / RT, A = a.T * a.k, CP = 4 * L * NT;
    // at most: every expert's passes
    const int64_t passes = a.ids ? std::min(a.E, A) + A / CP : (A + CP - 1) / CP;
    const unsigned grid = (unsigned)std::min<int64_t>(passes * groups, (int64_t)cus * per_cu);
    return by_groups(a.group, [&](auto mg) {
        hipLaunchKernelGGL((int4_kernel<SWIGLU, L, NT, RT, decltype(mg)::value, W, Q>), dim3(grid), dim3(W * kWave), 0, s,
                           a);
    });
}

template <int L, int RT, int W>
hipError_t launch_sum(const Int4Args& a, hipStream_t s)
{
    const unsigned grid = (unsigned)(tiles_of(a.N, 0) / RT);
    const size_t lds = (size_t)W * a.T * 16 * RT * sizeof(float);
    return by_groups(a.group, [&](auto mg) {
        hipLaunchKernelGGL((int4_sum_kernel<L, RT, decltype(mg)::value, W>), dim3(grid), dim3(W * kWave), lds, s, a);
    });
}

// Two tiles per workgroup where that leaves one for every compute unit and the
// sums of the tokens fit (4 tokens on 8 experts of 14336 x 4096: 32.0 us, one tile
// 38.6). Else sixteen waves, for the units in flight (16 tokens on 128 experts
// of 2048 x 768: 19.3 us, eight waves 24.3), but for the loads of many rows (64 tokens
// on 8 experts of 4096 x 1408: 15.6, sixteen 16.1) and sums that don't fit so.
template <int L>
hipError_t launch_sums(const Int4Args& a, int cus, hipStream_t s)
{
    if (tiles_of(a.N, 0) / 2 >= cus && a.T <= 64)
        return launch_sum<L, 2, 8>(a, s);
    if constexpr (L < 4) {
        if (a.T <= 64)
            return launch_sum<L, 1, 16>(a, s);
    }
    return launch_sum<L, 1, 8>(a, s);
}

// Tiles times the passes of `rows` rows: with ids, if all experts are chosen alike.
int64_t tile_passes(const Int4Args& a, int rows)
{
    const int A = a.T * a.k;
    return (int64_t)(a.ids ? std::min(a.E, A) : (A + rows - 1) / rows) * tiles_of(a.N, a.swiglu);
}

// The more items, the more tiles each, so that x is read less often, and the fewer
// waves, so that starts and ends of workgroups overlap the others' streaming.
// One token, K = 4096: N = 4096 (256 tiles) 4.8 us with one tile and eight waves, 5.8
// with two; 14336: 8.4 with two tiles and four waves, 9.2 and 9.5 with one and
// four; 28672: 13.1 with four, 13.5 with two. Of long rows each wave has enough:
// four tiles and eight waves (12 rows, 14336 x 14336: 24.1 us, two and four 29.5).
template <int L>
hipError_t launch_items(const Int4Args& a, int cus, hipStream_t s)
{
    const int64_t tiles = tile_passes(a, 4 * L);
    const bool four = tiles_of(a.N, a.swiglu) >= 4;
    if (!a.swiglu && tiles <= cus)
        return launch<false, L, 1, 1, 8, 2>(a, 2, cus, s);
    if (tiles <= 2 * cus)
        return a.swiglu ? launch<true, L, 1, 2, 8, 1>(a, 2, cus, s) : launch<false, L, 1, 2, 8, 1>(a, 2, cus, s);
    if (four && a.K >= 8192)
        return a.swiglu ? launch<true, L, 1, 4, 8, 1>(a, 1, cus, s) : launch<false, L, 1, 4, 8, 1>(a, 1, cus, s);
    if (four && tiles > 6 * cus)
        return a.swiglu ? launch<true, L, 1, 4, 4, 1>(a, 2, cus, s) : launch<false, L, 1, 4, 4, 1>(a, 2, cus, s);
    return a.swiglu ? launch<true, L, 1, 2, 4, 1>(a, 4, cus, s) : launch<false, L, 1, 2, 4, 1>(a, 4, cus, s);
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
    // choose alike), in eighths. Fewer rows per pass need fewer loads of x, but
    // an expert of more is read again, from a cache: passes of 4 up to 1.6 rows, of 8 up to 4.5, of
    // 16 up to 12. A weighted sum stays at 16, whose tokens' sums take the LDS. Ids that
    // crowd get the passes of the mean (64 tokens, k = 2, 1536 x 2048, 128 experts, passes of 4:
    // 83 experts in use 35.4 us, 32 20.1, 8 16.9, 2 13.0).
    const int rows = !a.ids ? a.T * 8 : a.T <= 4 ? 8 : std::min(a.T * 8, A * 8 / std::min(a.E, A));
    const int few = a.ids ? 13 : 32, some = a.ids ? 36 : 64, more = a.ids ? 96 : 128;
    if (a.w) {
        if (rows <= few)
            return launch_sums<1>(a, cus, s);
        return rows <= some ? launch_sums<2>(a, cus, s) : launch_sums<4>(a, cus, s);
    }
    if (rows <= few)
        return launch_items<1>(a, cus, s);
    if (rows <= some)
        return launch_items<2>(a, cus, s);
    // Passes of 32 rows spend less on each unit, but only where there are enough
    // of them for the card (64 rows, K = 4096: N = 8192 12.5 us, passes of 16 13.1; N = 2048
    // 6.7 and 6.1; 128 rows of 14336 x 4096 35.5 and 43.0).
    if (rows <= more || tile_passes(a, 16) <= 4 * cus || tiles_of(a.N, a.swiglu) < 4)
        return launch_items<4>(a, cus, s);
    return a.swiglu ? launch<true, 4, 2, 4, 4, 1>(a, 2, cus, s) : launch<false, 4, 2, 4, 4, 1>(a, 2, cus, s);
}

}  // namespace cmoe
