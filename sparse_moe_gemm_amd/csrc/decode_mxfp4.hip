// decode_mxfp4.hip - small-batch expert GEMMs on 4-bit microscaled weights.
//
// The weight-streaming path of decode_bf16.hip for MXFP4 weights (mxfp4.hpp):
// no LDS, no barriers; a wave takes work items (expert, kNB 32-row weight
// blocks, K slice) round robin and reads their codes once, straight into
// registers. It steps through K 128 at a time: per weight block two 1 KiB
// blocks of codes (16 bytes per lane each) and the scale word that holds both
// blocks' bytes. bf16 token rows meet the codes as bf16 (exact) on
// v_mfma_f32_32x32x16_bf16, 4-bit token rows (A4, gate/up) meet them on
// v_mfma_scale_f32_32x32x64_f8f6f4. Four weight blocks per item, since the
// activations' fragments of a bf16 step are twice a weight block's bytes: each
// feeds all four. fp32 slice partials, or H itself where a gate/up item covers
// all of K, as in decode_bf16.hip. Bound by HBM: 17/32 bytes per weight.
#include "mxfp4.hpp"

namespace cmoe {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kNB = 4;  // 32-row weight blocks per item

template <bool A4>
struct MxStep {
    Vec16 b[kNB][2];
    uint32_t bs[kNB];
    Vec16 a[A4 ? 2 : 8];
    uint32_t as;
};

template <bool GATE_UP, bool A4>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2))) void decode_mx_kernel(MxDecodeArgs g)
{
    if (g.gate_rows > 0 && max_expert_rows(g.offsets, g.E) > g.gate_rows)
        return;  // the tiled kernels take this call
    const int lane = threadIdx.x % kWave, half = lane >> 5;
    const int W = gridDim.x * (kThreads / kWave);
    const int w0 = blockIdx.x * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int N = GATE_UP ? 2 * g.f : g.d;
    const int K = GATE_UP ? g.d : g.f;
    const int NB = N / 32, KB = K / 64, KU = K / 128, KG = mx_scale_groups(K), S = g.split;
    const int NI = NB / kNB;
    const int items = g.E * NI * S;

    for (int it = w0; it < items; it += W) {
        const int s = it % S;
        const int rest = it / S;
        const int nb = (rest % NI) * kNB;
        const int e = rest / NI;
        const int seg0 = g.offsets[e];
        const int cnt = g.offsets[e + 1] - seg0;
        if (cnt <= 0)
            continue;
        const int u0 = (int)((int64_t)s * KU / S), u1 = (int)((int64_t)(s + 1) * KU / S);
        const int64_t blk = (int64_t)e * NB + nb;
        const Vec16* bp = (const Vec16*)g.b + blk * KB * kWave + lane;
        const uint32_t* sp = (const uint32_t*)g.b_scales + blk * KG * kWave + lane;

        for (int r0 = 0; r0 < cnt; r0 += 32) {
            const int r = min(r0 + (lane & 31), cnt - 1);
            const int64_t src = GATE_UP ? g.perm[seg0 + r] : seg0 + r;
            const Vec16* ap = (const Vec16*)((const uint8_t*)g.a + src * (A4 ? K / 2 : K * 2));
            const uint32_t* asp = A4 ? (const uint32_t*)(g.a_scales + src * (K / 32)) : nullptr;
            floatx16 acc[kNB];
#pragma unroll
            for (int n = 0; n < kNB; ++n)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    acc[n][q] = 0.f;
            // 128 k of the item, as loaded by step u (past the slice: its last
            // step again, not multiplied)
            auto load = [&](MxStep<A4>& t, int u) {
                u = min(u, u1 - 1);
#pragma unroll
                for (int n = 0; n < kNB; ++n) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        t.b[n][h] = __builtin_nontemporal_load(&bp[((int64_t)n * KB + 2 * u + h) * kWave]);
                    t.bs[n] = sp[((int64_t)n * KG + u / 2) * kWave];
                }
                if constexpr (A4) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        t.a[h] = ap[u * 4 + 2 * h + half];
                    t.as = asp[u];
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        t.a[q] = ap[u * 16 + (q / 4) * 8 + 4 * half + q % 4];
                }
            };
            auto multiply = [&](const MxStep<A4>& t, int u) {
                if constexpr (A4) {
                    const uint32_t sa = t.as >> (8 * half);
                    auto step = [&](auto h_const) {
                        constexpr int h = decltype(h_const)::value;
                        const Vec16 w = t.a[h];
                        const v8i fa{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
#pragma unroll
                        for (int n = 0; n < kNB; ++n) {
                            const Vec16 c = t.b[n][h];
                            const v8i fb{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
                            acc[n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                fa, fb, acc[n], 4, 4, 2 * h, (int)sa, h, (int)(t.bs[n] >> (16 * (u & 1))));
                        }
                    };
                    step(std::integral_constant<int, 0>{});
                    step(std::integral_constant<int, 1>{});
                } else {
#pragma unroll
                    for (int n = 0; n < kNB; ++n) {
                        const uint32_t sw = t.bs[n] >> (16 * (u & 1));
                        const float sc[2] = {mx_scale(sw & 255u), mx_scale((sw >> 8) & 255u)};
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            acc[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                as_bf16x8(t.a[q]), mx8_to_bf16(t.b[n][q / 4][q % 4], sc[q / 4]), acc[n], 0, 0, 0);
                    }
                }
            };
            MxStep<A4> t0, t1;
            load(t0, u0);
            for (int u = u0; u < u1; u += 2) {
                load(t1, u + 1);
                multiply(t0, u);
                load(t0, u + 2);
                if (u + 1 < u1)
                    multiply(t1, u + 1);
            }
            // Result lane: weight row lane%32 of a block, token rows
            // 8 (q/4) + 4 (lane/32) + q%4.
            if (GATE_UP && g.h != nullptr) {
#pragma unroll
                for (int n = 0; n < kNB; n += 2) {
                    uint16_t* hcol = g.h + (nb + n) * 16 + (lane & 31);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const int row = r0 + 8 * (q / 4) + 4 * half + (q % 4);
                        if (row < cnt)
                            hcol[(int64_t)(seg0 + row) * g.f] = f32_to_bf16_bits(silu(acc[n][q]) * acc[n + 1][q]);
                    }
                }
            } else {
                float* out = g.part + (int64_t)s * g.A * N + nb * 32 + (lane & 31);
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int row = r0 + 8 * (q / 4) + 4 * half + (q % 4);
                    if (row < cnt)
#pragma unroll
                        for (int n = 0; n < kNB; ++n)
                            out[(int64_t)(seg0 + row) * N + 32 * n] = acc[n][q];
                }
            }
        }
    }
}

}  // namespace

int decode_mx_split(int E, int N, int K, int waves)
{
    // as decode_split, with items of four weight blocks and 128-wide steps
    return decode_split(E, N / 2, K, 128, waves, 64);
}

hipError_t launch_decode_mx(const MxDecodeArgs& a, int gate_up, int cus, hipStream_t s)
{
    const dim3 grid(cus * 2), block(kThreads);
    if (!gate_up)
        hipLaunchKernelGGL((decode_mx_kernel<false, false>), grid, block, 0, s, a);
    else if (a.a_scales)
        hipLaunchKernelGGL((decode_mx_kernel<true, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((decode_mx_kernel<true, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace cmoe
