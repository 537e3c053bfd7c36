// norm.hip - root-mean-square norm of token rows, with the residual's addition
// before it and 8-bit rows after it.
//
//   v  = x + r                       (r optional; the sum in fp32)
//   r' = v rounded to the row type   (the residual stream behind this point)
//   y  = v / sqrt(mean(v^2) + eps) * w
//   q  = E4M3 codes of y with one power-of-two scale per row, quant_fp8.hip's
//        rule, taken from the fp32 y: each output is rounded once.
//
// The step in front of an MoE layer: y goes to its router, q to products on
// 8-bit rows. One pass over memory: a row stays in registers between its two
// reductions (the squares, the largest |y|). The squares are summed in 64 bits,
// so that no finite row overflows or vanishes in its mean. 16384 rows of 4096 bf16
// with residual, y and codes: 119 us, 5.1 TB/s, a large copy's rate; one row 3.6 us.
#include "common.hpp"

namespace cmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// Eight consecutive values at any element's alignment (gfx950 reads and writes
// vectors at every address).
typedef Vec16 Vec16u __attribute__((aligned(2)));
typedef floatx4 floatx4u __attribute__((aligned(4)));
typedef uint32_t Vec8u __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8])
{
    const Vec16 w = *(const Vec16u*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8])
{
    const floatx4 a = *(const floatx4u*)p, b = *(const floatx4u*)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8])
{
    Vec16 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)f32_to_bf16_bits(v[2 * i]) | ((uint32_t)f32_to_bf16_bits(v[2 * i + 1]) << 16);
    *(Vec16u*)p = w;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8])
{
    *(floatx4u*)p = floatx4{v[0], v[1], v[2], v[3]};
    *(floatx4u*)(p + 4) = floatx4{v[4], v[5], v[6], v[7]};
}

__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = f32_to_bf16_bits(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

__device__ __forceinline__ void weights8(const NormArgs& a, int c, float (&w)[8])
{
    if (a.w_bf16)
        load8((const uint16_t*)a.w + c, w);
    else
        load8((const float*)a.w + c, w);
}

// |y| where it is finite, else 0: infinities and NaN become NaN codes and leave
// the scale to the others.
__device__ __forceinline__ float finite_abs(float y)
{
    const float m = fabsf(y);
    return m < INFINITY ? m : 0.0f;
}

__device__ __forceinline__ float fp8_input(float y, float inv)
{
    return fabsf(y) < INFINITY ? y * inv : NAN;
}

__device__ __forceinline__ Vec8u fp8x8(const float (&y)[8], float inv)
{
    Vec8u c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int r = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_input(y[4 * h], inv), fp8_input(y[4 * h + 1], inv), 0, false);
        c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fp8_input(y[4 * h + 2], inv), fp8_input(y[4 * h + 3], inv), r,
                                                         true);
    }
    return c;
}

// 1 / sqrt(mean + eps) of a row from the sum of its squares; and in two fp32
// factors, neither of them subnormal (rows near the largest float).
struct Scale {
    double s;
    float pre, inv;
};
__device__ __forceinline__ Scale row_scale(double sum, const NormArgs& a)
{
    const double s = 1.0 / sqrt(sum / a.d + (double)a.eps);
    const bool big = s < 0x1p-100;
    return Scale{s, big ? 0x1p-64f : 1.0f, (float)(big ? s * 0x1p64 : s)};
}

// y: of fp32 rows the nearest float, so that a code is off only where that
// rounding meets a tie; of bf16 rows within three roundings of it (as long as v * s
// is no subnormal float), which y's own bf16 hides and the codes' 4 bits nearly always do (in 64 bits 16384 rows of 4096
// with codes took 125.6 us, so 118.8).
template <typename T>
__device__ __forceinline__ float scaled(float v, const Scale& s, float w)
{
    if constexpr (sizeof(T) == 4)
        return (float)((double)v * s.s * (double)w);
    else
        return v * s.pre * s.inv * w;
}

template <int WPR>
__device__ __forceinline__ double row_sum(double v, double* red)
{
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1)
        v += __shfl_xor(v, o, kWave);
    if constexpr (WPR > 1) {
        const int wv = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0)
            red[wv] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < WPR; ++i)
            v += red[i];
    }
    return v;
}

template <int WPR>
__device__ __forceinline__ float row_max(float v, float* red)
{
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor(v, o, kWave));
    if constexpr (WPR > 1) {
        const int wv = threadIdx.x / kWave;
        if (threadIdx.x % kWave == 0)
            red[wv] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < WPR; ++i)
            v = fmaxf(v, red[i]);
    }
    return v;
}

// Rows of 8 to NC * WPR * 512 values, WPR waves (of the block's four) per row:
// lane i of a row's waves holds values 8i.. +8 of every chunk. The last values
// of a row whose length is no multiple of 8 are the chunk at d - 8, whose first
// ones another lane holds too: they are left out of the sum and written twice,
// with the same bits. All of a row's loads are unconditional and in flight
// together (lanes behind the row read its end). Every value is read before the
// first one is written, so y and the sum may take the place of x or the residual.
template <typename T, int NC, int WPR>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a)
{
    __shared__ double reds[2][WPR];
    __shared__ float redm[2][WPR];
    const int d = a.d;
    constexpr int kStep = WPR * kWave * 8;
    const int i0 = (threadIdx.x % (WPR * kWave)) * 8;
    const int64_t step = (int64_t)gridDim.x * (kWaves / WPR);
    int turn = 0;
    for (int64_t t = (int64_t)blockIdx.x * (kWaves / WPR) + threadIdx.x / (WPR * kWave); t < a.rows; t += step) {
        const T* x = (const T*)a.x + t * a.x_ld;
        float v[NC][8], w[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i)
            load8(x + min(i0 + i * kStep, d - 8), v[i]);
        if (a.r) {
            const T* r = (const T*)a.r + t * a.r_ld;
            float u[NC][8];
#pragma unroll
            for (int i = 0; i < NC; ++i)
                load8(r + min(i0 + i * kStep, d - 8), u[i]);
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] += u[i][j];
        }
#pragma unroll
        for (int i = 0; i < NC; ++i)
            weights8(a, min(i0 + i * kStep, d - 8), w[i]);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = i0 + i * kStep;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double z = min(c, d - 8) + j >= c ? (double)v[i][j] : 0.0;
                sum = fma(z, z, sum);
            }
        }
        const Scale sc = row_scale(row_sum<WPR>(sum, reds[turn]), a);
        if (a.r_out) {
            T* r = (T*)a.r_out + t * a.r_out_ld;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (i0 + i * kStep < d)
                    store8(r + min(i0 + i * kStep, d - 8), v[i]);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = scaled<T>(v[i][j], sc, w[i][j]);
        if (a.y) {
            T* y = (T*)a.y + t * d;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (i0 + i * kStep < d)
                    store8(y + min(i0 + i * kStep, d - 8), v[i]);
        }
        if (a.codes) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    m = fmaxf(m, finite_abs(v[i][j]));
            m = row_max<WPR>(m, redm[turn]);
            const int e = fp8_scale_exp(m);
            const float inv = ldexpf(1.0f, -e);  // exact
            uint8_t* q = a.codes + t * d;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (i0 + i * kStep < d)
                    *(Vec8u*)(q + min(i0 + i * kStep, d - 8)) = fp8x8(v[i], inv);
            if (i0 == 0)
                a.scales[t] = ldexpf(1.0f, e);
        }
        turn ^= 1;  // the next row's partial results go where no wave still reads this one's
    }
}

// Rows of any other length, a block each, read once more for every step.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_long_kernel(NormArgs a)
{
    __shared__ double reds[2][kWaves];
    __shared__ float redm[2][kWaves];
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
        const T* x = (const T*)a.x + t * a.x_ld;
        const T* r = a.r ? (const T*)a.r + t * a.r_ld : nullptr;
        auto value = [&](int c) { return load1(x + c) + (r ? load1(r + c) : 0.0f); };
        auto weight = [&](int c) { return a.w_bf16 ? load1((const uint16_t*)a.w + c) : load1((const float*)a.w + c); };
        double sum = 0.0;
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
            const double z = value(c);
            sum = fma(z, z, sum);
        }
        const Scale sc = row_scale(row_sum<kWaves>(sum, reds[turn]), a);
        float inv = 0.0f;
        if (a.codes) {
            float m = 0.0f;
            for (int c = threadIdx.x; c < a.d; c += kThreads)
                m = fmaxf(m, finite_abs(scaled<T>(value(c), sc, weight(c))));
            const int e = fp8_scale_exp(row_max<kWaves>(m, redm[turn]));
            inv = ldexpf(1.0f, -e);
            if (threadIdx.x == 0)
                a.scales[t] = ldexpf(1.0f, e);
        }
        // each value is read and written by one thread
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
            const float v = value(c), y = scaled<T>(v, sc, weight(c));
            if (a.r_out)
                store1((T*)a.r_out + t * a.r_out_ld + c, v);
            if (a.y)
                store1((T*)a.y + t * a.d + c, y);
            if (a.codes)
                a.codes[t * a.d + c] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(fp8_input(y, inv), 0.0f, 0, false);
        }
        turn ^= 1;
    }
}

template <typename T>
hipError_t launch(const NormArgs& a, hipStream_t s)
{
    auto go = [&](auto kern, int per_block) {
        const int64_t blocks = std::min<int64_t>((a.rows + per_block - 1) / per_block, 16384);
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    };
    if (a.d < 8 || a.d > 16384)
        go(norm_long_kernel<T>, 1);
    else if (a.d <= 512)
        go(norm_kernel<T, 1, 1>, 4);
    else if (a.d <= 1024)
        go(norm_kernel<T, 2, 1>, 4);
    else if (a.d <= 2048)
        go(norm_kernel<T, 1, 4>, 1);
    else if (a.d <= 4096)
        go(norm_kernel<T, 2, 4>, 1);
    else if (a.d <= 8192)
        go(norm_kernel<T, 4, 4>, 1);
    else
        go(norm_kernel<T, 8, 4>, 1);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s)
{
    return a.bf16 ? launch<uint16_t>(a, s) : launch<float>(a, s);
}

}  // namespace cmoe
