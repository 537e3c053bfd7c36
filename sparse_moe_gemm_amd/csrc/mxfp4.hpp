// mxfp4.hpp - 4-bit microscaled values (OCP MXFP4): device helpers shared by
// the quantizer and the GEMMs that multiply them.
//
// A block of 32 consecutive values of a row is kept as 32 E2M1 codes (sign,
// 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) and one E8M0 scale byte b, the power of two 2^(b - 127); b = 255
// makes all 32 values NaN. Code 2i of a row is in the low half of byte i.
#pragma once

#include "tiles.hpp"

namespace cmoe {

constexpr int kMxBlock = 32;          // values that share a scale
constexpr uint32_t kMxNan = 255;      // scale byte of a block with a NaN or an infinity

// Scale byte of a block from the bit pattern of its largest magnitude (the
// largest of the values' patterns without the sign, which orders finite
// values, infinity and NaN). The smallest exponent e >= -127 with
// amax <= 6 * 2^e: with amax = 1.m * 2^(E - 127), 6 = 1.5 * 2^2, so e is E - 129
// if 1.m <= 1.5 and E - 128 otherwise; subnormal maxima clamp to e = -127. A
// block of zeros takes e = 0.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits)
{
    if (amax_bits >= 0x7F800000u)
        return kMxNan;
    if (amax_bits == 0)
        return 127;
    const int b = (int)(amax_bits >> 23) - 2 + ((amax_bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    return (uint32_t)max(b, 0);
}

// 2^(127 - b), the exact inverse of the block's scale (b <= 253 for finite
// blocks, so it is a normal number).
__device__ __forceinline__ float mx_inv_scale(uint32_t b)
{
    return __uint_as_float((254u - b) << 23);
}

// Eight codes of v[0..7] * inv, value i in bits 4i .. 4i+3: nearest E2M1 value,
// ties to the even mantissa, the sign kept by zeros. v_cvt_scalef32_pk_fp4_f32
// rounds so on every f32 of magnitude at most 6 (a test compares all of them with
// the rule), and the products are exact wherever they are not far
// below the smallest code.
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8], float inv)
{
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * inv, v[1] * inv, 1.0f, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * inv, v[3] * inv, 1.0f, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * inv, v[5] * inv, 1.0f, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * inv, v[7] * inv, 1.0f, 3);
    return r;
}

// The scale byte as the conversions below take it: the f32 whose exponent
// field it is. Byte 0 gives the pattern 0, which they read as 2^-127, and byte
// 255 the pattern of an infinity, which makes every result NaN.
__device__ __forceinline__ float mx_scale(uint32_t b)
{
    return __uint_as_float(b << 23);
}

// Eight codes (one word) times the block's scale as bf16: exact, since an
// E2M1 value has two significant bits.
__device__ __forceinline__ bf16x8 mx8_to_bf16(uint32_t w, float sc)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3);
    return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// GEMM layout of 4-bit weights [E][N][K] (K a multiple of 128): block
// (e, nb, kb) of 1 KiB holds rows 32 nb .. +32 and k 64 kb .. +64; lane l's 16
// bytes at 16 l are the 32 codes of row 32 nb + l%32, k 64 kb + 32 (l/32) ..
// +32, one scale block. That is the operand order of
// v_mfma_scale_f32_32x32x64_f8f6f4 on 4-bit codes; turned into bf16, the
// lane's word s (8 codes, k + 8 s) is its fragment of a 16-wide MFMA k step,
// for which the activations are read in the same k order. The scale bytes
// stand apart, 1 KiB per 256 rows x 128 k (what a GEMM tile takes in one load
// per wave): byte mx_scale_at(...) is that of lane l's codes in block kb.
__host__ __device__ __forceinline__ int mx_scale_tiles(int N)
{
    return (N + 255) / 256;
}
// Start of the 1 KiB of expert e's 32-row blocks 8 (nb/8) .. +8 at k unit u = kb/2.
__host__ __device__ __forceinline__ int64_t mx_scale_group(int64_t e, int nb, int u, int N, int K)
{
    return ((e * mx_scale_tiles(N) + nb / 8) * (K / 128) + u) * 1024;
}
__host__ __device__ __forceinline__ int mx_scale_at(int nb, int kb, int l)
{
    return (nb % 8) * 128 + l * 2 + (kb & 1);
}

// Token rows in 4 bits for the tiled GEMM, by sorted position: every expert's
// rows start a new 32-row block, blocks are numbered through the experts, at
// most mx_row_blocks of them. Codes as the weights': block (b, kb) of 1 KiB at
// (b * K/64 + kb) * 1024; scale bytes of block b and k unit u: 128 bytes at
// (u * mx_row_blocks + b) * 128, lane l's two at 2 l.
__host__ __device__ __forceinline__ int mx_row_blocks(int A, int E)
{
    return A / 32 + (A < E ? A : E);
}

// From a tile table: blocks of the experts below this lane's four, and an
// expert's first block (e wave-uniform).
__device__ __forceinline__ int mx_blocks_below(const TileTable& t, int lane)
{
    int own = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        own += (t.cnt[q] + 31) / 32;
    int incl = own;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(incl, d, kWave);
        if (lane >= d)
            incl += o;
    }
    return incl - own;
}

__device__ __forceinline__ int mx_block_of(const TileTable& t, int below, int e)
{
    const int ln = e / 4;
    int b = __builtin_amdgcn_readlane(below, ln);
#pragma unroll
    for (int q = 0; q < 3; ++q)
        b += q < e % 4 ? (__builtin_amdgcn_readlane(t.cnt[q], ln) + 31) / 32 : 0;
    return __builtin_amdgcn_readfirstlane(b);
}

}  // namespace cmoe
