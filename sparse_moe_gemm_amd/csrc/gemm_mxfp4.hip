// gemm_mxfp4.hip - grouped expert GEMMs on 4-bit microscaled weights.
//
// The two expert GEMMs of gemm_bf16.hip for layers whose expert weights are
// MXFP4 (mxfp4.hpp): for every sorted position p of expert e
//   gate/up:  H[p][c]  = SiLU(sum_i X[perm[p]][i] Wg[e][c][i]) * (sum_i X[perm[p]][i] Wu[e][c][i])
//   down:     Ys_s[p][o] = sum_{c in K split s} H[p][c] Wd[e][o][c]     (fp32)
// with W the values the codes stand for. Two ways to multiply them:
//   A4 false: bf16 rows (x for gate/up, H for down). A lane's 32 codes become
//             four bf16 fragments in registers (exact) for
//             v_mfma_f32_32x32x16_bf16.
//   A4 true:  the token rows are MXFP4 too and gate/up runs on
//             v_mfma_scale_f32_32x32x64_f8f6f4, 4-bit codes on both sides, one
//             scale byte per lane: products of 4-bit values are multiples of
//             1/4 up to 36, whose sums within a block are exact.
// Both sum in fp32. H is stored as bf16 (the activation type and the down
// GEMM's MFMA operand, relative error 2^-8), expert outputs stay fp32 until the
// combine.
//
// A tile is BM sorted rows of one expert x 256 weight rows (x a K split); a
// persistent workgroup walks its tiles (tiles.hpp) and streams their K stages
// (64 k of bf16 rows, 128 k of 4-bit rows) through a ring of SLOTS LDS slots:
// while stage s is multiplied, the next SLOTS - 1 are on their way, across tile
// borders too, but for gate/up on bf16 rows: its next tile's row numbers come
// from perm when they are needed, and as vector memory returns in order, the
// wait for them is a wait for all stages in flight. One wait and one barrier per
// stage: after it every wave's loads of stage s are in LDS and every wave has
// read stage s - 1 to the end, so its slot can take stage s + SLOTS - 1. Weights are streamed straight into LDS in
// whole 1 KiB blocks, which keeps enough of them in flight to read HBM at 5.1 -
// 5.4 TB/s from experts of a few rows (32 tokens on 8 experts of 4096 x 14336:
// gate/up 499 MB in 90 us, down 249 MB in 47 us; streaming them into registers
// without LDS took 133 and 88 us).
// Waves form WAVES_M x 4; a wave multiplies WM = BM / WAVES_M rows with 64
// weight rows (one gate and one up block of 32, so SiLU(g)*u stays in its
// registers). The weight fragment is the MFMA's first operand: a result lane
// holds one token row and groups of four consecutive outputs.
//
// With many rows (8 experts, 4096 tokens, k = 2): down 0.96 TFLOP in 770 - 840 us
// (1.15 - 1.25 PFLOP/s, 61% MFMA busy at 1.86 GHz; random bf16 operands alone, no
// loads, run at 1.6 PFLOP/s under the power limit); gate/up on 4-bit rows 1.92
// TFLOP in 485 - 550 us (3.5 - 3.9 PFLOP/s; alone 6.3), bound by what the stages move:
// 35 KB into LDS and 96 KB out of it for 1024 MFMA cycles. A wave tile of 128 x
// 128 would read a third less but spills.
#include "lds_dma.hpp"
#include "mxfp4.hpp"
#include "tiles.hpp"

namespace cmoe {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kBN = 256;  // weight rows per tile

__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b)
{
    return (uint32_t)f32_to_bf16_bits(a) | ((uint32_t)f32_to_bf16_bits(b) << 16);
}

// fn(0), fn(1), ... with the numbers as types.
template <int... I, typename F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F fn)
{
    (fn(std::integral_constant<int, I>{}), ...);
}

// One K stage: the token rows (64 k of BM bf16 rows, 128 bytes each; or 128 k of
// 4-bit rows, which come blocked as the weights do), KBS 1 KiB weight blocks
// for each 32 weight rows, and the scales of the 128 k they belong to.
template <int BM, bool A4>
struct MxStage {
    static constexpr int KBS = A4 ? 2 : 1;
    Vec16 a[A4 ? BM / 32 * 2 * kWave : BM * 8];
    Vec16 b[(kBN / 32) * KBS * kWave];
    uint16_t bs[(kBN / 32) * kWave];
    uint16_t as[A4 ? BM / 32 * kWave : 8];
};

// Position of 16-byte chunk c of bf16 tile row r in the stage: the 16 rows that
// 16 lanes read at one chunk fall into 16 different 16-byte bank groups.
__device__ __forceinline__ int mx_swz(int r, int c)
{
    return c ^ ((r >> 1) & 7);
}

template <int BM, int WAVES_M, bool A4>
struct MxShape {
    using Stage = MxStage<BM, A4>;
    static constexpr int NW = WAVES_M * 4;
    static constexpr int WM = BM / WAVES_M;
    // Loads per wave and stage. Every wave issues as many (the waits count
    // them); where there are fewer loads than waves, waves share one and write
    // the same data to the same place.
    static constexpr int A_ALL = A4 ? BM / 16 : BM / 8, A_INS = A_ALL < NW ? 1 : A_ALL / NW;
    static constexpr int B_INS = (kBN / 32) * Stage::KBS / NW;
    static constexpr int AS_ALL = BM / kWave;  // A4
    static constexpr int NLD = A_INS + B_INS + 1 + (A4 ? 1 : 0);
    static_assert(B_INS >= 1, "every wave loads a share");
};

// Where the next stage to load comes from: a position in the stream of all K
// stages of this workgroup's tiles.
template <int A_INS>
struct MxCursor {
    Rsrc rb, rs;           // the tile's weight blocks and scale groups
    Rsrc ra, ras;          // A4: its token blocks and their scales
    uint32_t aoff[A_INS];  // bf16 rows: byte offsets of this lane's rows and chunk
    int kt, left;          // next stage along K, stages left in the tile
    int L;                 // the tile's launch index
};

// Workgroups on a compute unit: what its LDS and registers hold, since their
// barriers and loads then fall into each other's MFMAs. Three of four waves for
// bf16 rows in tiles of 32 and 64 (53 KB each), against two with one more slot
// each (67 and 70 KB), gate/up + down in us: 8 experts of 4096 x 14336 with 4
// rows on average 99 + 53 -> 96 + 52, 32 rows 128 + 65 -> 110 + 62; 128 of 2048 x
// 768 with 31 rows 53 + 38 -> 52 + 36; 64 of 4096 x 1408 with 31 rows 96 + 53 -> 91 +
// 53, most of them on two experts 106 + 69 -> 111 + 63. (Four of three slots for
// tiles of 32 rows: the same as three.)
template <int BM, int WAVES_M, bool A4>
__host__ __device__ constexpr int mx_groups()
{
    return WAVES_M > 1 ? 1 : BM <= 64 && !A4 ? 3 : 2;
}

template <int BM, int WAVES_M, int SLOTS, bool A4, bool GATE_UP>
__global__ __launch_bounds__(WAVES_M * 4 * kWave)
    __attribute__((amdgpu_waves_per_eu(WAVES_M * mx_groups<BM, WAVES_M, A4>(),
                                       WAVES_M * mx_groups<BM, WAVES_M, A4>()))) void mx_gemm_kernel(MxGemmArgs g)
{
    using Sh = MxShape<BM, WAVES_M, A4>;
    using Stage = typename Sh::Stage;
    constexpr int SM = GATE_UP ? 0 : 64;  // tile order as in the other GEMMs
    constexpr int MI = Sh::WM / 32;
    __shared__ Stage ring[SLOTS];

    const int N = GATE_UP ? 2 * g.f : g.d;
    const int K = GATE_UP ? g.d : g.f;
    const int NT = (N + kBN - 1) / kBN;
    const int KB = K / 64;
    const int KT = K / (A4 ? 128 : 64);
    const int S = GATE_UP ? 1 : g.split;
    const int lane = threadIdx.x % kWave;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wv / 4, wn = wv % 4;
    const int half = lane >> 5;

    TileTable tt;
    const int total = make_table<BM, SM>(g.offsets, g.E, lane, NT * S, tt);
    const int GRID = gridDim.x;
    if ((int)blockIdx.x >= total)
        return;

    const uint32_t Kbytes = (uint32_t)K * 2;
    const uint32_t a_rows = GATE_UP ? (uint32_t)(g.A_max / g.k) : (uint32_t)g.A_max;
    const Rsrc ra = buffer_rsrc(g.a, A4 ? 0u : a_rows * Kbytes);
    const int MB = mx_row_blocks(g.A_max, g.E);
    int blocks_below = 0;  // A4: 32-row blocks of the experts below this lane's four
    if constexpr (A4)
        blocks_below = mx_blocks_below(tt, lane);
    const uint32_t lane16 = (uint32_t)lane * 16u, lane4 = (uint32_t)lane * 4u;
    const uint32_t ring0 = lds_address(&ring[0]);

    auto row_of = [&](const Tile& t, int r) {
        const int p = t.row0 + min(r, t.rows - 1);  // past the segment: its last row again
        return (uint32_t)(GATE_UP ? g.perm[p] : p);
    };
    auto open = [&](MxCursor<Sh::A_INS>& c, int L) {
        const Tile t = decode<BM, SM>(tt, L, NT, S, g.group_n, KT);
        const int nb0 = t.n * (kBN / 32), nbs = N / 32 - nb0;  // row blocks from here to the expert's end
        const int64_t blk = (int64_t)t.e * (N / 32) + nb0;
        c.rb = buffer_rsrc((const uint8_t*)g.b + blk * KB * 1024, (uint32_t)min(nbs, kBN / 32) * (uint32_t)KB * 1024u);
        c.rs = buffer_rsrc(g.b_scales + mx_scale_group(t.e, nb0, 0, N, K), (uint32_t)(K / 128) * 1024u);
        if constexpr (A4) {
            const int first = mx_block_of(tt, blocks_below, t.e) + t.m * (BM / 32), n = (t.rows + 31) / 32;
            c.ra = buffer_rsrc((const uint8_t*)g.a + (int64_t)first * KB * 1024, (uint32_t)n * (uint32_t)KB * 1024u);
            c.ras = buffer_rsrc(g.a_scales + (int64_t)first * 128, ((uint32_t)KT * (uint32_t)MB - (uint32_t)first) * 128u);
        } else {
#pragma unroll
            for (int q = 0; q < Sh::A_INS; ++q) {
                const int r = (wv * Sh::A_INS + q) % Sh::A_ALL * 8 + lane / 8;
                c.aoff[q] = row_of(t, r) * Kbytes + (uint32_t)mx_swz(r, lane % 8) * 16u;
            }
        }
        c.kt = t.kt0;
        c.left = t.nkt;
        c.L = L;
    };
    // Load q (of NLD) of this wave's share of the cursor's stage into the slot
    // at LDS address base.
    auto piece = [&](const MxCursor<Sh::A_INS>& c, uint32_t base, auto q_const) {
        constexpr int q = decltype(q_const)::value;
        if constexpr (q < Sh::A_INS) {
            const int i = (wv * Sh::A_INS + q) % Sh::A_ALL;
            const uint32_t to = base + (uint32_t)offsetof(Stage, a) + (uint32_t)i * 1024u;
            if constexpr (A4)
                lds_load16(c.ra, lane16, ((uint32_t)(i / 2) * (uint32_t)KB + (uint32_t)(c.kt * 2 + i % 2)) * 1024u, to);
            else
                lds_load16(ra, c.aoff[q], (uint32_t)c.kt * 128u, to);
        } else if constexpr (q < Sh::A_INS + Sh::B_INS) {
            const int i = wv * Sh::B_INS + q - Sh::A_INS;  // row block i / KBS, k block i % KBS of the stage
            lds_load16(c.rb, lane16,
                       ((uint32_t)(i / Stage::KBS) * (uint32_t)KB + (uint32_t)(c.kt * Stage::KBS + i % Stage::KBS)) * 1024u,
                       base + (uint32_t)offsetof(Stage, b) + (uint32_t)i * 1024u);
        } else if constexpr (q == Sh::A_INS + Sh::B_INS) {
            lds_load4(c.rs, lane4, (uint32_t)(c.kt * Stage::KBS / 2) * 1024u + (uint32_t)(wv % 4) * 256u,
                      base + (uint32_t)offsetof(Stage, bs) + (uint32_t)(wv % 4) * 256u);
        } else {
            lds_load4(c.ras, lane4 + (uint32_t)(wv % Sh::AS_ALL) * 256u, (uint32_t)c.kt * (uint32_t)MB * 128u,
                      base + (uint32_t)offsetof(Stage, as) + (uint32_t)(wv % Sh::AS_ALL) * 256u);
        }
    };
    // Pieces Q0 .. Q1 of a stage.
    auto pieces = [&](const MxCursor<Sh::A_INS>& c, uint32_t base, auto q0_const, auto q1_const) {
        constexpr int Q0 = decltype(q0_const)::value, Q1 = decltype(q1_const)::value;
        each(std::make_integer_sequence<int, Q1 - Q0>{},
             [&](auto i) { piece(c, base, std::integral_constant<int, Q0 + decltype(i)::value>{}); });
    };
    // The cursor moves on; past the last tile it stays, and the last stage is
    // loaded again (read by no one), which keeps the loads in flight per stage
    // the same.
    auto advance = [&](MxCursor<Sh::A_INS>& c) {
        if (c.left > 1) {
            ++c.kt;
            --c.left;
        } else if (c.L + GRID < total) {
            open(c, c.L + GRID);
        }
    };
    auto slot_at = [&](int slot) { return ring0 + (uint32_t)slot * (uint32_t)sizeof(Stage); };

    MxCursor<Sh::A_INS> cur;
    open(cur, blockIdx.x);
#pragma unroll
    for (int q = 0; q < SLOTS - 1; ++q) {
        pieces(cur, slot_at(q), std::integral_constant<int, 0>{}, std::integral_constant<int, Sh::NLD>{});
        advance(cur);
    }
    int slot = 0;

    for (int L = blockIdx.x; L < total; L += GRID) {
        const Tile t = decode<BM, SM>(tt, L, NT, S, g.group_n, KT);
        floatx16 acc[2][MI];  // [gate/up or first/second 32 weight rows][32-row group]
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    acc[j][i][q] = 0.f;
        const int wrows = t.rows - wm * Sh::WM;
        const int RG = wrows <= 0 ? 0 : min((wrows + 31) / 32, MI);  // row groups with valid rows

        // All K stages with the first RGC row groups multiplied.
        auto stages = [&](auto rg_const) {
            constexpr int RGC = decltype(rg_const)::value;
            auto stage = [&](int j) {
                // Its own loads of the stage have landed, and its LDS reads of the
                // one before (the compiler may move the MFMAs that use them past
                // the barrier, and their waits with them, while the slot they
                // read is filled anew behind it).
                wait_vm<Sh::NLD * (SLOTS - 2)>();
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                const uint32_t fill = slot_at(slot == 0 ? SLOTS - 1 : slot - 1);
                const Stage& st = ring[slot];
                const int kb = (t.kt0 + j) * Stage::KBS;
                if constexpr (RGC == 0 || !A4)
                    pieces(cur, fill, std::integral_constant<int, 0>{}, std::integral_constant<int, Sh::NLD>{});
                if constexpr (RGC > 0 && A4) {
                    uint32_t sb[2], sa[RGC];
                    Vec16 wb[2][2], wa[2][RGC];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            wb[s][n] = st.b[((wn * 2 + n) * 2 + s) * kWave + lane];
                        if (s == 0) {
#pragma unroll
                            for (int n = 0; n < 2; ++n)
                                sb[n] = st.bs[(wn * 2 + n) * kWave + lane];
#pragma unroll
                            for (int i = 0; i < RGC; ++i)
                                sa[i] = st.as[(wm * MI + i) * kWave + lane];
                        }
#pragma unroll
                        for (int i = 0; i < RGC; ++i)
                            wa[s][i] = st.a[((wm * MI + i) * 2 + s) * kWave + lane];
                    }
                    auto step = [&](auto s_const) {
                        constexpr int s = decltype(s_const)::value;
                        auto wide = [](const Vec16& w) {
                            return v8i{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
                        };
                        auto row = [&](auto i_const) {
                            constexpr int i = decltype(i_const)::value;
                            if constexpr (i < RGC) {
                                // The next loads are spread over the MFMAs, in the order
                                // written: all issued first they hold every wave up at the
                                // load unit (8 x 14336, 4096 tokens: 590 -> 520 us; reading
                                // the fragments half a stage ahead as well gained nothing).
                                constexpr int m = s * RGC + i;
                                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                                for (int n = 0; n < 2; ++n)
                                    acc[n][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                        wide(wb[s][n]), wide(wa[s][i]), acc[n][i], 4, 4, s, (int)sb[n], s, (int)sa[i]);
                                __builtin_amdgcn_sched_barrier(0);
                                pieces(cur, fill, std::integral_constant<int, m * Sh::NLD / (2 * RGC)>{},
                                       std::integral_constant<int, (m + 1) * Sh::NLD / (2 * RGC)>{});
                            }
                        };
                        row(std::integral_constant<int, 0>{});
                        row(std::integral_constant<int, 1>{});
                        row(std::integral_constant<int, 2>{});
                        row(std::integral_constant<int, 3>{});
                    };
                    step(std::integral_constant<int, 0>{});
                    step(std::integral_constant<int, 1>{});
                    __builtin_amdgcn_sched_barrier(0);
                } else if constexpr (RGC > 0) {
                    Vec16 wb[2];
                    float sc[2];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        wb[n] = st.b[(wn * 2 + n) * kWave + lane];
                        sc[n] = mx_scale(((const uint8_t*)st.bs)[((wn * 2 + n) * kWave + lane) * 2 + (kb & 1)]);
                    }
                    auto step = [&](auto s_const) {
                        constexpr int s = decltype(s_const)::value;
                        bf16x8 fb[2], fa[RGC];
#pragma unroll
                        for (int i = 0; i < RGC; ++i) {
                            const int r = wm * Sh::WM + i * 32 + (lane & 31);
                            fa[i] = as_bf16x8(st.a[r * 8 + mx_swz(r, 4 * half + s)]);
                        }
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            fb[n] = mx8_to_bf16(wb[n][s], sc[n]);
#pragma unroll
                        for (int i = 0; i < RGC; ++i)
#pragma unroll
                            for (int n = 0; n < 2; ++n)
                                acc[n][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[n], fa[i], acc[n][i], 0, 0, 0);
                    };
                    step(std::integral_constant<int, 0>{});
                    step(std::integral_constant<int, 1>{});
                    step(std::integral_constant<int, 2>{});
                    step(std::integral_constant<int, 3>{});
                }
                slot = slot == SLOTS - 1 ? 0 : slot + 1;
            };
            // The cursor is SLOTS - 1 stages ahead: in this tile until the last
            // SLOTS stages (a loop without branches: behind one the compiler sinks
            // the MFMAs), then in the next.
            int j = 0;
            for (; j + SLOTS < t.nkt; ++j) {
                stage(j);
                ++cur.kt;
                --cur.left;
            }
            for (; j < t.nkt; ++j) {
                stage(j);
                advance(cur);
            }
        };
        if (RG == MI)
            stages(std::integral_constant<int, MI>{});
        else if (MI > 2 && RG == 3)
            stages(std::integral_constant<int, (MI > 2 ? 3 : MI)>{});
        else if (MI > 2 && RG == 2)
            stages(std::integral_constant<int, (MI > 2 ? 2 : MI)>{});
        else if (MI > 1 && RG == 1)
            stages(std::integral_constant<int, 1>{});
        else
            stages(std::integral_constant<int, 0>{});

        // Outputs. Result lane: token row lane%32 of a 32-row group, weight rows
        // 8 (q/4) + 4 (lane/32) + q%4.
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int row = wm * Sh::WM + i * 32 + (lane & 31);
            if (row >= t.rows)
                continue;
            const int64_t p = t.row0 + row;
            if constexpr (GATE_UP) {
                uint16_t* hp = (uint16_t*)g.out + p * g.f + (t.n * kBN + wn * 64) / 2 + 4 * half;
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    float h[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        h[q] = silu_rcp(acc[0][i][4 * q4 + q]) * acc[1][i][4 * q4 + q];
                    *(uint2*)(hp + 8 * q4) = make_uint2(bf16x2_bits(h[0], h[1]), bf16x2_bits(h[2], h[3]));
                }
            } else {
                const int col0 = t.n * kBN + wn * 64;
                float* yp = (float*)g.out + ((int64_t)t.s * g.A_max + p) * g.d + col0 + 4 * half;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    if (col0 + 32 * n >= N)  // a last tile of 128 weight rows
                        continue;
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4)
                        *(floatx4*)(yp + 32 * n + 8 * q4) = floatx4{acc[n][i][4 * q4], acc[n][i][4 * q4 + 1],
                                                                    acc[n][i][4 * q4 + 2], acc[n][i][4 * q4 + 3]};
                }
            }
        }
    }
    wait_vm<0>();  // the loads past the last tile
}

template <int BM, int WAVES_M, int SLOTS, bool A4, bool GATE_UP>
hipError_t launch_shape(const MxGemmArgs& a, hipStream_t s)
{
    const int NT = ((GATE_UP ? 2 * a.f : a.d) + kBN - 1) / kBN;
    const int64_t tiles = ((int64_t)a.A_max / BM + a.E) * NT * (GATE_UP ? 1 : a.split);  // at most
    const int grid = (int)std::min<int64_t>(tiles, mx_groups<BM, WAVES_M, A4>() * a.cus);
    hipLaunchKernelGGL((mx_gemm_kernel<BM, WAVES_M, SLOTS, A4, GATE_UP>), dim3(grid), dim3(WAVES_M * 4 * kWave), 0, s,
                       a);
    return hipGetLastError();
}

// Rows per tile from the mean rows per expert (the routing is on the device).
// The choice would be better for the number of tiles as well: few large experts
// (112 n-tiles each) still gain by tiles of 64 rows at 64 rows on average, where
// many small ones lose, and the rule takes 128 for both.
// A tile costs its weights' stages whatever rows it holds, and its multiplied
// row groups; an expert with a few rows more than the tile pays for two.
// Gate/up + down in us with tiles of 64 / 128 rows, bf16 rows: 8 experts of
// 4096 x 14336 with 45 rows on average 126 + 74 / 143 + 70, 64 rows 158 + 90 / 166 +
// 102, 98 rows 201 + 111 / 207 + 103; 128 of 2048 x 768 with 44 rows 60 + 44 / 66 +
// 47, 64 rows 95 + 56 / 73 + 53; 64 of 4096 x 1408 with 47 rows 108 + 72 / 109 + 70,
// 62 rows 126 + 79 / 119 + 77. 32 / 64 rows, gate/up: 128 of 2048 x 768 with 10
// rows 44 / 44, 31 rows 61 / 52; 8 of 4096 x 14336 with 32 rows 137 / 110. (256
// rows: 1024 on average 1478 against 1496, but down 834 against 803.) 4-bit rows
// (gate/up, 64 / 128 / 256): 8 x 4096 x 14336 with
// 8 rows 92 / 92 / 92, 83 rows 145 / 111 / 113, 175 rows 222 / 161 / 143, 1024
// rows 735 / 586 / 571; 128 x 2048 x 768 with 128 rows 91 / 71 / 61; 64 x 4096 x
// 1408 with two experts taking most rows, mean 10: 45 / 46 / 54, mean 31: 86 /
// 79 / 81, mean 128: 143 / 133 / 142.
int mx_tile_rows(int A, int E, bool a4)
{
    const int64_t mean = ((int64_t)A + E - 1) / E;
    if (a4)
        return mean <= 20 ? 64 : mean <= 100 ? 128 : 256;
    return mean <= 20 ? 32 : mean <= 50 ? 64 : 128;
}

}  // namespace

int mx_down_split(int A, int E, int d, int f, int cus)
{
    // K splits of the down GEMM: up to four, until there are three tiles per
    // compute unit (two or three run there at a time), while each part keeps 1024 k.
    // Measured with one / two / four (down GEMM and combine, us): 8 experts of
    // 4096 x 14336, 32 tokens - / 58 / 59, 333 tokens - / 103 / 96, 2047 tokens
    // 470 / 454 / 483, 4096 tokens 842 / 859 / -; 128 experts of 2048 x 768 lose
    // by every split (16 tokens 22 / 24).
    const int rows = mx_tile_rows(A, E, false);
    const int64_t mt = std::max<int64_t>(((int64_t)A + rows - 1) / rows, std::min(A, E));
    const int64_t tiles = mt * ((d + kBN - 1) / kBN);
    int s = 1;
    while (s < kMxMaxSplit && tiles * s < 3 * (int64_t)cus && f / (2 * s) >= 1024)
        s *= 2;
    return s;
}

int64_t mx_split_rows(int cus)
{
    return (int64_t)128 * 3 * cus;  // then tiles of 128 rows make three per compute unit
}

hipError_t launch_gate_up_mx(const MxGemmArgs& a, hipStream_t s)
{
    if (a.a_scales) {
        const int rows = mx_tile_rows(a.A_max, a.E, true);
        return rows == 64    ? launch_shape<64, 1, 3, true, true>(a, s)
               : rows == 128 ? launch_shape<128, 1, 3, true, true>(a, s)
                             : launch_shape<256, 2, 3, true, true>(a, s);
    }
    const int rows = mx_tile_rows(a.A_max, a.E, false);
    return rows == 32   ? launch_shape<32, 1, 4, false, true>(a, s)
           : rows == 64 ? launch_shape<64, 1, 3, false, true>(a, s)
                        : launch_shape<128, 1, 3, false, true>(a, s);
}

hipError_t launch_down_mx(const MxGemmArgs& a, hipStream_t s)
{
    const int rows = mx_tile_rows(a.A_max, a.E, false);
    return rows == 32   ? launch_shape<32, 1, 4, false, false>(a, s)
           : rows == 64 ? launch_shape<64, 1, 3, false, false>(a, s)
                        : launch_shape<128, 1, 3, false, false>(a, s);
}

}  // namespace cmoe
