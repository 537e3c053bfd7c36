// quant_int4.hip - 4-bit integer groups: quantization and reading back.
//
// The other 4-bit form the converters know («Colibri 是什么» (nxbn.cn): 4-bit
// AWQ; «Colibri» (lshu.cn): group-wise scales): a weight row in groups of g
// consecutive values, each with a scale s (16-bit float) and a zero point z,
//   w = (q - z) * s,   q, z in 0..15.
// Quantization of a group (values w_i, lo = min(0, min w_i), hi = max(0, max w_i)):
//   s = bf16((hi - lo) / 15),  z = rint(-lo / s),  q_i = rint(w_i / s) + z,
// z and q clamped to 0..15 (s may round down); symmetric: s = bf16(max |w_i| / 7),
// z = 8. A group whose s would be 0 is a group of zeros (s = 1); one with an
// infinity or NaN gets the scale NaN. rint rounds ties to even. Reading back
// rounds (q - z) * s once (exact in fp32).
//
// Both directions move each byte once.
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
    uint32_t bits = 0;           // largest magnitude's bits: infinities and NaN show
};

__device__ __forceinline__ void widen(Range& r, const float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r.lo = fminf(r.lo, v[i]);
        r.hi = fmaxf(r.hi, v[i]);
        r.bits = max(r.bits, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
}

// Over the L neighbouring lanes of a group.
template <int L>
__device__ __forceinline__ void join(Range& r)
{
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        r.lo = fminf(r.lo, __shfl_xor(r.lo, o, kWave));
        r.hi = fmaxf(r.hi, __shfl_xor(r.hi, o, kWave));
        r.bits = max(r.bits, (uint32_t)__shfl_xor((int)r.bits, o, kWave));
    }
}

struct Group {
    uint16_t bits;  // scale
    float s, z;
    bool bad, empty;
};

__device__ __forceinline__ Group group_of(const Range& r, bool symmetric)
{
    Group g;
    g.bad = r.bits >= 0x7F800000u;
    const float range = r.hi - r.lo;
    float s = symmetric ? fmaxf(r.hi, -r.lo) / 7.0f : range < INFINITY ? range / 15.0f : r.hi / 15.0f - r.lo / 15.0f;
    g.bits = f32_to_bf16_bits(s);
    s = bf16_to_f32(g.bits);
    g.empty = s == 0.0f;
    if (g.empty) {
        s = 1.0f;
        g.bits = 0x3F80;
    }
    g.s = s;
    g.z = symmetric ? 8.0f : fminf(fmaxf(rintf(-r.lo / s), 0.0f), 15.0f);
    if (g.bad) {
        g.bits = 0x7FC0;
        g.z = symmetric ? 8.0f : 0.0f;
    }
    return g;
}

__device__ __forceinline__ uint32_t encode8(const float (&v)[8], const Group& g)
{
    if (g.bad || g.empty)
        return 0x11111111u * (uint32_t)g.z;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c |= (uint32_t)fminf(fmaxf(rintf(v[i] / g.s) + g.z, 0.0f), 15.0f) << (4 * i);
    return c;
}

// L neighbouring lanes share a group of 8 * L * m values, lane j of them holding
// values 8j .. +8 of each of its m parts: a wave reads whole lines and writes
// 256 bytes of codes. Groups of one part stay in registers between the two
// steps, longer ones are read again. Four groups per thread are in flight.
template <typename T, bool VEC, int L>
__global__ __launch_bounds__(kThreads) void int4_quantize_kernel(const T* w, int64_t groups, int per_row, int m,
                                                                 int64_t ld, uint32_t* codes, uint16_t* scales,
                                                                 uint8_t* zeros)
{
    constexpr int kFlight = 4;
    const int j = threadIdx.x % L;
    const int64_t step = (int64_t)gridDim.x * (kThreads / L);
    const int64_t first = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    for (int64_t g0 = first; g0 < groups; g0 += step * kFlight) {
        const T* src[kFlight];
        float v[kFlight][8];
        Range r[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t g = min(g0 + f * step, groups - 1);  // past the end: the last group again
            const int64_t row = (groups >> 32) == 0 ? (uint32_t)g / (uint32_t)per_row : g / per_row;
            src[f] = w + row * ld + (g - row * per_row) * (8 * L * m) + 8 * j;
            load8<VEC>(src[f], v[f]);
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
            widen(r[f], v[f]);
        for (int p = 1; p < m; ++p)
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                load8<VEC>(src[f] + p * 8 * L, v[f]);
                widen(r[f], v[f]);
            }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            join<L>(r[f]);
            const int64_t g = g0 + f * step;
            if (g >= groups)
                break;  // no exchange between lanes is left
            const Group q = group_of(r[f], zeros == nullptr);
            if (m == 1)
                codes[g * L + j] = encode8(v[f], q);
            else
                for (int p = 0; p < m; ++p) {
                    float u[8];
                    load8<VEC>(src[f] + p * 8 * L, u);
                    codes[(g * m + p) * L + j] = encode8(u, q);
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
            z[f] = zeros ? (float)zeros[g] : 8.0f;
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
    const int lanes = group >= 128 ? 16 : group / 8;
    const int64_t blocks = std::min<int64_t>((groups + 4 * (kThreads / lanes) - 1) / (4 * (kThreads / lanes)), 16384);
    auto go = [&](auto kern, int m) {
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, s, w, groups, (int)(cols / group), m, ld,
                           (uint32_t*)codes, scales, zeros);
    };
    if (group == 32)
        go(int4_quantize_kernel<T, VEC, 4>, 1);
    else if (group == 64)
        go(int4_quantize_kernel<T, VEC, 8>, 1);
    else
        go(int4_quantize_kernel<T, VEC, 16>, group / 128);
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
