// quant_mxfp4.hip - 4-bit microscaled rows: quantization, reading back, and the
// expert weights' GEMM layout.
//
// «Colibri 是什么» (xxqk.cn) §4.2 lets the converter keep the expert weights
// alone in fewer bits, the router in full precision; this is the 4-bit form of
// that idea in the open MXFP4 format (mxfp4.hpp). For every block of 32 values
// v_i of a row:
//   2^e  = smallest power of two, e >= -127, with max_i |v_i| <= 6 * 2^e
//          (e = 0 for a block of zeros), so that no value saturates,
//   code = v_i * 2^-e rounded to the nearest E2M1 value, ties to even,
// and a block that holds a NaN or an infinity gets the NaN scale. Reading
// back, code * 2^e, is exact in bf16 and f32 down to the subnormals (products of
// 2^128 and more overflow to infinity).
//
// Both directions move each byte once and are bound by HBM (a quantized bf16
// row: 2 bytes read and 17/32 written per value): a 14336 x 4096 bf16 matrix is
// quantized in 29 us and read back in 23 us, 5.1 and 6.3 TB/s (the library's
// copy: 5.1); a few rows take 2 - 4 us each way, mostly launch.
#include "mxfp4.hpp"

namespace cmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;  // 8-value units per thread in flight

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Eight consecutive values at p as f32. VEC: p is 16-byte aligned.
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

__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// Four neighbouring lanes share a block: lane j of the four holds its values
// 8j .. 8j+7, so a wave reads whole lines and writes 256 bytes of codes; the
// block maximum takes two exchanges between them. rows x upr units of 8 values
// (upr = cols / 8, a multiple of 4), row r at w + r * ld.
template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const T* w, int64_t units, int upr, int64_t ld,
                                                               uint32_t* codes, uint8_t* scales)
{
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t u0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; u0 < units; u0 += step * kUnits) {
        float v[kUnits][8];
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
            // past the end: the last unit again (all four lanes of a block
            // stay together, since units is a multiple of 4)
            const int64_t u = u0 + q * step < units ? u0 + q * step : units - 4 + (u0 & 3);
            int64_t r;
            if ((units >> 32) == 0)
                r = (uint32_t)u / (uint32_t)upr;
            else
                r = u / upr;
            load8<VEC>(w + r * ld + (u - r * upr) * 8, v[q]);
        }
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
            const int64_t u = u0 + q * step;
            uint32_t m = amax_bits8(v[q]);
            m = max(m, (uint32_t)__shfl_xor((int)m, 1, kWave));
            m = max(m, (uint32_t)__shfl_xor((int)m, 2, kWave));
            const uint32_t b = mx_scale_byte(m);
            const uint32_t c = b == kMxNan ? 0u : mx_encode8(v[q], mx_inv_scale(b));
            if (u < units) {
                codes[u] = c;
                if ((u & 3) == 0)
                    scales[u >> 2] = (uint8_t)b;
            }
        }
    }
}

// Eight codes per thread and unit back to values.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint32_t* codes, const uint8_t* scales,
                                                                 int64_t units, void* out)
{
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t u0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; u0 < units; u0 += step * kUnits) {
        uint32_t c[kUnits], b[kUnits];
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
            const int64_t u = min(u0 + q * step, units - 1);
            c[q] = codes[u];
            b[q] = scales[u >> 2];
        }
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
            const int64_t u = u0 + q * step;
            if (u >= units)
                break;
            const bf16x8 v = mx8_to_bf16(c[q], mx_scale(b[q]));
            if constexpr (BF16) {
                ((Vec16*)out)[u] = __builtin_bit_cast(Vec16, v);
            } else {
                floatx4 lo, hi;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo[i] = (float)v[i];
                    hi[i] = (float)v[4 + i];
                }
                ((floatx4*)out)[2 * u] = lo;
                ((floatx4*)out)[2 * u + 1] = hi;
            }
        }
    }
}

// bf16 expert weights into the GEMM layout (mxfp4.hpp), one lane's block of 32
// values per thread. With w1 != null the rows are gate/up rows interleaved by
// 32, as in the other layouts: combined row n of expert e is gate row
// (n/64)*32 + n%32 when n%64 < 32, else that up row.
__global__ __launch_bounds__(kThreads) void mx_pack_blocked_kernel(const uint16_t* w0, const uint16_t* w1, Vec16* out,
                                                                   uint8_t* scales, int E, int N, int K)
{
    const int NB = N / 32, KB = K / 64;
    const int64_t total = (int64_t)E * NB * KB * kWave;
    const int Nsrc = w1 ? N / 2 : N;
    for (int64_t idx = blockIdx.x * (int64_t)kThreads + threadIdx.x; idx < total;
         idx += (int64_t)gridDim.x * kThreads) {
        const int l = (int)(idx % kWave);
        const int64_t blk = idx / kWave;
        const int kb = (int)(blk % KB);
        const int64_t rb = blk / KB;  // e * NB + nb
        const int nb = (int)(rb % NB);
        const int64_t e = rb / NB;
        const int n = nb * 32 + (l % 32);
        const uint16_t* src = w0;
        int srow = n;
        if (w1) {
            srow = (n / 64) * 32 + (n % 32);
            src = n % 64 < 32 ? w0 : w1;
        }
        const uint16_t* p = src + (e * Nsrc + srow) * (int64_t)K + kb * 64 + 32 * (l / 32);
        float v[4][8];
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            load8<true>(p + 8 * q, v[q]);
            m = max(m, amax_bits8(v[q]));
        }
        const uint32_t b = mx_scale_byte(m);
        const float inv = mx_inv_scale(b == kMxNan ? 127u : b);
        Vec16 c;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            c[q] = b == kMxNan ? 0u : mx_encode8(v[q], inv);
        out[idx] = c;
        scales[mx_scale_group(e, nb, kb / 2, N, K) + mx_scale_at(nb, kb, l)] = (uint8_t)b;
    }
}

// Token rows [T][d] of a forward into the blocked 4-bit layout of the tiled
// GEMM (mxfp4.hpp), gathered by sorted position: a wave takes 32 rows x 128 k,
// a lane one block of 32 values at a time, so the maximum needs no exchange and
// codes leave as 1 KiB per store. Rows past an expert's last repeat it.
__global__ __launch_bounds__(kThreads) void mx_quantize_sorted_kernel(const uint16_t* x, const int32_t* offsets,
                                                                      const int32_t* perm, int A, int E, int d,
                                                                      Vec16* codes, uint16_t* scales)
{
    const int lane = threadIdx.x % kWave;
    const int MB = mx_row_blocks(A, E), KB = d / 64, KU = d / 128;
    TileTable tt;
    const int blocks = make_table<32>(offsets, E, lane, 1, tt);  // 32-row tiles are the blocks
    const int W = gridDim.x * (kThreads / kWave);
    const int w0 = blockIdx.x * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (int it = w0; it < blocks * KU; it += W) {
        const int b = it / KU, u = it - b * KU;
        const Tile t = decode<32>(tt, b, 1, 1, 1, 1);
        const int64_t row = perm[t.row0 + min(lane & 31, t.rows - 1)];
        const uint16_t* p = x + row * d + u * 128 + 32 * (lane >> 5);
        float v[2][4][8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                load8<true>(p + 64 * h + 8 * q, v[h][q]);
        uint32_t sb = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                m = max(m, amax_bits8(v[h][q]));
            const uint32_t s = mx_scale_byte(m);
            const float inv = mx_inv_scale(s == kMxNan ? 127u : s);
            Vec16 c;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                c[q] = s == kMxNan ? 0u : mx_encode8(v[h][q], inv);
            codes[((int64_t)b * KB + 2 * u + h) * kWave + lane] = c;
            sb |= s << (8 * h);
        }
        scales[((int64_t)u * MB + b) * kWave + lane] = (uint16_t)sb;
    }
}

unsigned unit_blocks(int64_t units)
{
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((units + kThreads * kUnits - 1) / (kThreads * kUnits), 8192));
}

}  // namespace

hipError_t launch_mx_quantize(const void* w, int bf16_in, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                              uint8_t* scales, hipStream_t s)
{
    if (rows < 1)
        return hipSuccess;
    const int64_t units = rows * (cols / 8);
    const int64_t es = bf16_in ? 2 : 4;
    // whole 16-byte loads where every row starts on 16 bytes, else one value
    // at a time
    const bool vec = ((uintptr_t)w % 16) == 0 && (rows == 1 || (ld * es) % 16 == 0);
    const dim3 grid(unit_blocks(units)), block(kThreads);
    const int upr = (int)(cols / 8);
    if (bf16_in) {
        if (vec)
            hipLaunchKernelGGL((mx_quantize_kernel<uint16_t, true>), grid, block, 0, s, (const uint16_t*)w, units, upr,
                               ld, (uint32_t*)codes, scales);
        else
            hipLaunchKernelGGL((mx_quantize_kernel<uint16_t, false>), grid, block, 0, s, (const uint16_t*)w, units,
                               upr, ld, (uint32_t*)codes, scales);
    } else {
        if (vec)
            hipLaunchKernelGGL((mx_quantize_kernel<float, true>), grid, block, 0, s, (const float*)w, units, upr, ld,
                               (uint32_t*)codes, scales);
        else
            hipLaunchKernelGGL((mx_quantize_kernel<float, false>), grid, block, 0, s, (const float*)w, units, upr, ld,
                               (uint32_t*)codes, scales);
    }
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int bf16_out,
                                void* out, hipStream_t s)
{
    if (rows < 1)
        return hipSuccess;
    const int64_t units = rows * (cols / 8);
    const dim3 grid(unit_blocks(units)), block(kThreads);
    if (bf16_out)
        hipLaunchKernelGGL(mx_dequantize_kernel<true>, grid, block, 0, s, (const uint32_t*)codes, scales, units, out);
    else
        hipLaunchKernelGGL(mx_dequantize_kernel<false>, grid, block, 0, s, (const uint32_t*)codes, scales, units, out);
    return hipGetLastError();
}

hipError_t launch_mx_quantize_sorted(const void* x, const int32_t* offsets, const int32_t* perm, int A, int E, int d,
                                     uint8_t* codes, uint8_t* scales, hipStream_t s)
{
    const int64_t waves = (int64_t)mx_row_blocks(A, E) * (d / 128);
    const unsigned blocks = (unsigned)std::min<int64_t>((waves + 3) / 4, 4096);
    hipLaunchKernelGGL(mx_quantize_sorted_kernel, dim3(blocks), dim3(kThreads), 0, s, (const uint16_t*)x, offsets, perm,
                       A, E, d, (Vec16*)codes, (uint16_t*)scales);
    return hipGetLastError();
}

size_t mx_row_bytes(int A, int E, int d)
{
    return (size_t)mx_row_blocks(A, E) * 32 * (d / 2);
}

size_t mx_row_scale_bytes(int A, int E, int d)
{
    return (size_t)mx_row_blocks(A, E) * d;
}

size_t mx_weight_bytes(int64_t E, int64_t N, int64_t K)
{
    return (size_t)(E * N * K / 2);
}

size_t mx_weight_scale_bytes(int64_t E, int64_t N, int64_t K)
{
    return (size_t)(E * mx_scale_tiles((int)N) * (K / 128) * 1024);
}

hipError_t launch_mx_pack_blocked(const void* w0, const void* w1, void* out, uint8_t* scales, int E, int N, int K,
                                  hipStream_t s)
{
    hipLaunchKernelGGL(mx_pack_blocked_kernel, dim3(4096), dim3(kThreads), 0, s, (const uint16_t*)w0,
                       (const uint16_t*)w1, (Vec16*)out, scales, E, N, K);
    return hipGetLastError();
}

}  // namespace cmoe
