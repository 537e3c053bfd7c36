// quant_int4.hip - 4-bit integer groups: quantization and reading back.
//
// The other 4-bit form the converters know («Colibri 是什么» (nxbn.cn): 4-bit
// AWQ; «Colibri不是蜂鸟» (lshu.cn): group-wise scales): a weight row in groups of g
// consecutive values, each with a scale s (16-bit float) and a zero point z,
//   w = (q - z) * s,   q, z in 0..15.
// Quantization of a group (values w_i, lo = min(0, min w_i), hi = max(0, max w_i)):
//   s = bf16((hi - lo) / 15),  z = rint(-lo / s),  q_i = rint(w_i / s) + z,
// z and q clamped to 0..15 (s may round down); symmetric: s = bf16(max |w_i| / 7),
// z = 8. A group whose s would be 0 is a group of zeros (s = 1); one with an
// infinity or NaN gets the scale NaN. rint rounds ties to even. Reading back
// rounds (q - z) * s once (exact in fp32).
//
// Both directions move each byte once, but for quantization of groups of other
// lengths than 32 to 512 in powers of two, which are read twice. 14336 x 4096, groups of
// 128, there and back in turn: 53.4 us for 2 x 148 MB (5.6 TB/s). The same direction again
// and again: bf16 30.3 us (4.9 TB/s) and 34.8 back (4.3), fp32 50.5 (5.3) and 64.3 (4.1);
// groups of 1024 57 us, of 4096 86.
#include "common.hpp"

namespace cmoe {

namespace {

constexpr int kThreads = 256;

template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8])
{
    if constexpr (VEC) {
        const Vec16 w = *(const Vec16*)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = bf16_to_f32(p[i]);
    }
}

template <bool VEC>
__device__ __forceinline__ void load8(const float* p, float (&v)[8])
{
    if constexpr (VEC) {
        const floatx4 a = *(const floatx4*)p, b = *(const floatx4*)(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = p[i];
    }
}

struct Range {
    float lo = 0.0f, hi = 0.0f;  // with 0
    float odd = 0.0f;            // NaN once an infinity or NaN was seen
};

__device__ __forceinline__ void widen(Range& r, const float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r.lo = fminf(r.lo, v[i]);
        r.hi = fmaxf(r.hi, v[i]);
        r.odd = fmaf(v[i], 0.0f, r.odd);
    }
}

template <int CTRL>
__device__ __forceinline__ void join_step(Range& r)
{
    const auto other = [](float v) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
    };
    r.lo = fminf(r.lo, other(r.lo));
    r.hi = fmaxf(r.hi, other(r.hi));
    r.odd += other(r.odd);
}

// Over the L neighbouring lanes of a group: moves within a row of 16 lanes,
// without a pass through LDS.
template <int L>
__device__ __forceinline__ void join(Range& r)
{
    join_step<0xB1>(r);  // quad_perm [1,0,3,2]
    if constexpr (L >= 4)
        join_step<0x4E>(r);  // quad_perm [2,3,0,1]
    if constexpr (L >= 8)
        join_step<0x141>(r);  // row_half_mirror
    if constexpr (L == 16)
        join_step<0x140>(r);  // row_mirror
}

struct Group {
    uint16_t bits;       // scale
    float s, inv, lift;  // scale * lift, about its reciprocal; lift: a power of two
    float z;
    bool flat;  // every code is z
};

// v / s by the reciprocal and one correction, q + (v - q s) / s: the nearest
// float, as a division gives (v has 24 bits and s 8: a quotient is at least
// 2^-33 of itself away from every midpoint, and the correction is good to
// 2^-45), at a third of its cost: 14336 x 4096 in groups of 128 54.6 -> 44.2 us.
// |s| within 2^+-100, so that nothing underflows that a rounding to an integer
// could see.
__device__ __forceinline__ float quotient(float v, const Group& g)
{
    const float q = v * g.inv;
    return fmaf(fmaf(-q, g.s, v), g.inv, q);
}

__device__ __forceinline__ Group group_of(const Range& r, bool symmetric)
{
    Group g;
    const bool bad = r.odd != 0.0f;
    float range = r.hi - r.lo, back = 1.0f;
    if (range == INFINITY) {
        range = 0.5f * r.hi - 0.5f * r.lo;
        back = 2.0f;
    }
    const float s = symmetric ? fmaxf(r.hi, -r.lo) / 7.0f : range / 15.0f * back;
    g.bits = f32_to_bf16_bits(s);
    g.s = bf16_to_f32(g.bits);
    g.flat = bad || g.s == 0.0f;
    if (g.s == 0.0f) {
        g.s = 1.0f;
        g.bits = 0x3F80;
    }
    g.lift = g.s < 0x1p-100f ? 0x1p64f : g.s > 0x1p100f ? 0x1p-64f : 1.0f;
    g.s *= g.lift;
    g.inv = __builtin_amdgcn_rcpf(g.s);
    g.z = symmetric ? 8.0f : __builtin_amdgcn_fmed3f(rintf(quotient(-r.lo * g.lift, g)), 0.0f, 15.0f);
    if (bad) {
        g.bits = 0x7FC0;
        g.z = symmetric ? 8.0f : 0.0f;
    } else if (g.flat) {
        g.z = symmetric ? 8.0f : 0.0f;
    }
    return g;
}

__device__ __forceinline__ uint32_t encode8(float (&v)[8], const Group& g)
{
    if (g.lift != 1.0f)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] *= g.lift;
    uint32_t even = 0, odd = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = __builtin_amdgcn_fmed3f(rintf(quotient(v[i], g)) + g.z, 0.0f, 15.0f);  // an integer
        if (i & 1)
            odd = __builtin_amdgcn_cvt_pk_u8_f32(c, i / 2, odd);
        else
            even = __builtin_amdgcn_cvt_pk_u8_f32(c, i / 2, even);
    }
    return g.flat ? 0x11111111u * (uint32_t)g.z : even | odd << 4;
}

// L neighbouring lanes share a group of 8 L P m values, lane j of them holding
// values 8j .. +8 of its parts of 8 L. What a group costs beside its values (the
// range's exchange, scale and zero point) is thus shared by 16 or 32 values per
// lane; with 8 the instructions took longer than the memory (14336 x 4096, groups
// of 128: 16 lanes 36.0 us, 4 lanes 27.9; of 32, both ways: 4 lanes 59.9, 2 lanes 54.9, one,
// whose loads no longer share lines, 60.8). m = 1: the values stay in registers
// between the two steps, other groups are read again (of 256 so, both ways: 87.5 us,
// in registers 52.3).
// 32 values per thread are in flight.
template <typename T, bool VEC, int L, int P, bool ONE>
__global__ __launch_bounds__(kThreads) void int4_quantize_kernel(const T* w, int64_t groups, int per_row, int m,
                                                                 int64_t ld, uint32_t* codes, uint16_t* scales,
                                                                 uint8_t* zeros)
{
    constexpr int kFlight = 4 / P, kPart = 8 * L;
    const int j = threadIdx.x % L;
    const int parts = ONE ? P : P * m, group = kPart * parts;
    const int64_t step = (int64_t)gridDim.x * (kThreads / L);
    const int64_t first = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const bool dense = ld == (int64_t)per_row * group;  // rows without gaps
    for (int64_t g0 = first; g0 < groups; g0 += step * kFlight) {
        const T* src[kFlight];
        float v[kFlight][P][8];
        Range r[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t g = min(g0 + f * step, groups - 1);  // past the end: the last group again
            src[f] = w + g * group + 8 * j;
            if (!dense) {
                const int64_t row = (groups >> 32) == 0 ? (uint32_t)g / (uint32_t)per_row : g / per_row;
                src[f] += row * (ld - (int64_t)per_row * group);
            }
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
#pragma unroll
            for (int p = 0; p < P; ++p)
                load8<VEC>(src[f] + p * kPart, v[f][p]);
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
#pragma unroll
            for (int p = 0; p < P; ++p)
                widen(r[f], v[f][p]);
        if constexpr (!ONE)
            for (int p = P; p < parts; p += P)
#pragma unroll
                for (int f = 0; f < kFlight; ++f) {
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        load8<VEC>(src[f] + (p + q) * kPart, v[f][q]);
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        widen(r[f], v[f][q]);
                }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            join<L>(r[f]);
            const int64_t g = g0 + f * step;
            if (g >= groups)
                break;  // no exchange between lanes is left
            const Group q = group_of(r[f], zeros == nullptr);
            uint32_t* out = codes + g * (L * parts) + j;
            if constexpr (ONE) {
#pragma unroll
                for (int p = 0; p < P; ++p)
                    out[p * L] = encode8(v[f][p], q);
            } else {
                for (int p = 0; p < parts; ++p) {
                    float u[8];
                    load8<VEC>(src[f] + p * kPart, u);
                    out[p * L] = encode8(u, q);
                }
            }
            if (j == 0) {
                scales[g] = q.bits;
                if (zeros)
                    zeros[g] = (uint8_t)q.z;
            }
        }
    }
}

// Eight codes per thread and unit back to values; units of a group: per_group.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void int4_dequantize_kernel(const uint32_t* codes, const uint16_t* scales,
                                                                   int scales_f16, const uint8_t* zeros, int64_t units,
                                                                   int per_group, void* out)
{
    constexpr int kFlight = 4;
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t u0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; u0 < units; u0 += step * kFlight) {
        uint32_t c[kFlight];
        uint16_t sb[kFlight];
        float z[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t u = min(u0 + f * step, units - 1);
            const int64_t g = (units >> 32) == 0 ? (uint32_t)u / (uint32_t)per_group : u / per_group;
            c[f] = codes[u];
            sb[f] = scales[g];
            z[f] = zeros ? (float)(zeros[g] & 15) : 8.0f;  // as int4_pack_kernel reads them
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t u = u0 + f * step;
            if (u >= units)
                break;
            const float s = scales_f16 ? (float)__builtin_bit_cast(_Float16, sb[f]) : bf16_to_f32(sb[f]);
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = ((float)((c[f] >> (4 * i)) & 15u) - z[f]) * s;
            if constexpr (BF16) {
                Vec16 o;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = (uint32_t)f32_to_bf16_bits(v[2 * i]) | ((uint32_t)f32_to_bf16_bits(v[2 * i + 1]) << 16);
                ((Vec16*)out)[u] = o;
            } else {
                ((floatx4*)out)[2 * u] = floatx4{v[0], v[1], v[2], v[3]};
                ((floatx4*)out)[2 * u + 1] = floatx4{v[4], v[5], v[6], v[7]};
            }
        }
    }
}

template <typename T, bool VEC>
hipError_t launch_quantize(const T* w, int64_t rows, int64_t cols, int64_t ld, int group, uint8_t* codes,
                           uint16_t* scales, uint8_t* zeros, hipStream_t s)
{
    const int64_t groups = rows * (cols / group);
    auto go = [&](auto kern, int m, int L, int flight) {
        const int64_t blocks = std::min<int64_t>((groups + flight * (kThreads / L) - 1) / (flight * (kThreads / L)), 16384);
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, s, w, groups, (int)(cols / group), m, ld,
                           (uint32_t*)codes, scales, zeros);
    };
    switch (group) {
    case 32: go(int4_quantize_kernel<T, VEC, 2, 2, true>, 1, 2, 2); break;
    case 64: go(int4_quantize_kernel<T, VEC, 2, 4, true>, 1, 2, 1); break;
    case 128: go(int4_quantize_kernel<T, VEC, 4, 4, true>, 1, 4, 1); break;
    case 256: go(int4_quantize_kernel<T, VEC, 8, 4, true>, 1, 8, 1); break;
    case 512: go(int4_quantize_kernel<T, VEC, 16, 4, true>, 1, 16, 1); break;
    default: go(int4_quantize_kernel<T, VEC, 4, 4, false>, group / 128, 4, 1);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int4_quantize(const void* w, int bf16_in, int64_t rows, int64_t cols, int64_t ld, int group,
                                uint8_t* codes, uint16_t* scales, uint8_t* zeros, hipStream_t s)
{
    // 16-byte loads where every group starts at a multiple of 16 bytes
    const int es = bf16_in ? 2 : 4;
    const bool vec = ((uintptr_t)w & 15u) == 0 && (ld * es) % 16 == 0;
    auto go = [&](auto* p) {
        return vec ? launch_quantize<std::remove_const_t<std::remove_pointer_t<decltype(p)>>, true>(
                         p, rows, cols, ld, group, codes, scales, zeros, s)
                   : launch_quantize<std::remove_const_t<std::remove_pointer_t<decltype(p)>>, false>(
                         p, rows, cols, ld, group, codes, scales, zeros, s);
    };
    return bf16_in ? go((const uint16_t*)w) : go((const float*)w);
}

hipError_t launch_int4_dequantize(const uint8_t* codes, const uint16_t* scales, int scales_f16, const uint8_t* zeros,
                                  int64_t rows, int64_t cols, int group, int bf16_out, void* out, hipStream_t s)
{
    const int64_t units = rows * (cols / 8);
    const int64_t blocks = std::min<int64_t>((units + 4 * kThreads - 1) / (4 * kThreads), 16384);
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, s, (const uint32_t*)codes, scales, scales_f16,
                           zeros, units, group / 8, out);
    };
    if (bf16_out)
        go(int4_dequantize_kernel<true>);
    else
        go(int4_dequantize_kernel<false>);
    return hipGetLastError();
}

}  // namespace cmoe
