// Products of rows in 4-bit floating point with a scale a block, for sm_103a:
//   C[i][j] = rowA[i] rowB[j] sum_b sA[i][b] sB[j][b] sum_{p in b} a[i][p] b[j][p] + bias[j]
// with A (M tokens) and B (N channels) as sgemm_quantize_fp4 writes them.  The tensor
// cores multiply the codes and apply the blocks' scales themselves (tcgen05.mma
// .kind::mxf4nvf4 with block scaling): products and their sums in FP32.
//
//  * fp4_tile_kernel -- 128 channels x NT = 16, 32, 64 or 128 tokens a CTA, for few
//    tokens: bound by the weights' way from HBM.  The channels are the MMA's M, so that
//    a weight tile is used whole however few the tokens.  Up to 8 CTAs of a cluster
//    share a tile's K range; their sums meet in distributed shared memory and are
//    added in the order of the ranks, each CTA a slice of the tokens.  In a graph 1 x 4096 x
//    4096 4.0 us (NV; launch, tensor memory and first loads are 2.5 of them), 64 x 8192 x 8192
//    9.9 (MX; 5.4 at HBM's rate, 128 of the SMs busy, 1 of exchange).
//  * fp4_pair_kernel -- 256 channels x 256 tokens on a CTA pair (cta_group::2),
//    persistent, for many tokens: each CTA holds 128 of the channels and 128 of the
//    tokens.  The epilogue's eight warps take the whole accumulator into registers
//    and leave it to the next tile's MMAs before they write C.  8192^3: 161 us in short runs
//    (NV, 6.8 PFLOP/s; MX 174), 182 to 187 when repeated until the power limit shows.  What bounds
//    it: with a quarter of the MMAs 151 us, without the operands' loads 133 (2.5 GB cross from
//    L2 to the SMs, 16.5 TB/s), without the writes of C 147 (the accumulator's way into
//    registers, 1 us a tile, in which no MMA runs).
//  * fp4_generic_kernel -- CUDA cores, any alignment, where the rows can neither be
//    read as stored nor be copied.
//
// Operand tiles are 256 k deep, 128 bytes a row (128-byte swizzle); the scales of 128
// rows are 512 contiguous bytes for every four blocks, fetched by TMA and copied to
// tensor memory (tcgen05.cp) by the lane that issues the MMAs, into columns of the
// stage's own: nothing is overwritten before the MMAs that read it have finished.
// Accumulators hold channels in lanes and tokens in columns, so a warp writes 32
// consecutive elements of a row of C at a time.
// Every wait is bounded, as in the library's other tensor-core kernels.
#include "device_common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "rows.cuh"
#include "sgemm.h"
#include "tcgen05.cuh"

namespace sg {
namespace {

constexpr int kStageK = 256, kRowBytes = kStageK / 2;  // a stage: one 128-byte row of 4-bit elements
constexpr int kTileCh = 128;                            // channels of a CTA
constexpr int kChBytes = kTileCh * kRowBytes;
constexpr int kSmemLimit = 232448;
template <int FORMAT>
constexpr int kStageWords = kStageK / (4 * fp4_block(FORMAT));  // words of four scales a row and stage

// Instruction descriptor of the block-scaled 4-bit MMAs: bits 4-5 / 29-30 which byte of
// a scale word B / A starts at, 7-9 and 10-11 E2M1 operands (1), 17-22 N >> 3, 23 the
// scales' type (1 E8M0, 0 E4M3), 27-28 M >> 7; both operands K-major, K = 64.
__host__ __device__ constexpr uint32_t idesc_fp4(int format, int M, int N, int sf_byte) {
    return (static_cast<uint32_t>(sf_byte) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           ((format == SGEMM_FP4_MX ? 1u : 0u) << 23) | (static_cast<uint32_t>(M >> 7) << 27) |
           (static_cast<uint32_t>(sf_byte) << 29);
}

template <int FORMAT, int GROUP>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
#define SG_MMA(G, V)                                                                                             \
    asm volatile(                                                                                                \
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                                        \
        "tcgen05.mma.cta_group::" G ".kind::mxf4nvf4.block_scale.scale_vec::" V " [%0], %1, %2, %3, [%5], [%6], p;\n\t}" \
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)                                  \
        : "memory")
    if (GROUP == 1) {
        if (FORMAT == SGEMM_FP4_MX) SG_MMA("1", "2X");
        else SG_MMA("1", "4X");
    } else {
        if (FORMAT == SGEMM_FP4_MX) SG_MMA("2", "2X");
        else SG_MMA("2", "4X");
    }
#undef SG_MMA
}

// 512 bytes of scales (32 x 16 bytes) to four columns of tensor memory, the same in
// each of its four groups of 32 lanes.
template <int GROUP>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    if (GROUP == 1) asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// MMAs of one stage, after the copies of its scales.  CH_COLS, TOK_COLS: tensor-memory
// columns of a word of the channels' and of the tokens' scales.
template <int FORMAT, int GROUP, int TOK_TILES, int N>
__device__ __forceinline__ void stage_mmas(uint32_t d, uint32_t sf, uint64_t ch, uint64_t tok, uint64_t ch_s, uint64_t tok_s,
                                           int k_left, bool first) {
    constexpr int W = kStageWords<FORMAT>;
    // (words of the stage behind the row's last: whatever lies there, never multiplied)
#pragma unroll
    for (int w = 0; w < W; ++w) {
        copy_scales<GROUP>(sf + 4 * w, ch_s + w * (512 / 16));
#pragma unroll
        for (int t = 0; t < TOK_TILES; ++t)
            copy_scales<GROUP>(sf + 4 * W + 4 * (w * TOK_TILES + t), tok_s + (t * W + w) * (512 / 16));
    }
#pragma unroll
    for (int kk = 0; kk < kStageK / 64; ++kk) {
        if (kk * 64 >= k_left) break;
        const int w = FORMAT == SGEMM_FP4_MX ? kk / 2 : kk;
        const uint32_t id = idesc_fp4(FORMAT, 128 * GROUP, N, FORMAT == SGEMM_FP4_MX ? 2 * (kk & 1) : 0);
        mma_fp4<FORMAT, GROUP>(d, ch + kk * 2, tok + kk * 2, id, sf + 4 * w, sf + 4 * W + 4 * TOK_TILES * w,
                               first && kk == 0 ? 0u : 1u);
    }
}

__device__ __forceinline__ uint64_t scale_desc(const void *p) { return tc::smem_desc(smem_u32(p), 0, 128, 0); }
__device__ __forceinline__ uint64_t tile_desc(const void *p) { return tc::smem_desc(smem_u32(p), 16, 1024, tc::kLayoutSwizzle128); }

// The result's types.
template <class F>
__device__ __forceinline__ void with_type(int type, F f) {
    if (type == SGEMM_IN_F32) f(ElF32{});
    else if (type == SGEMM_IN_BF16) f(ElBF16{});
    else f(ElF16{});
}

// A place in a ring of stages and the parity of its current round.
struct Ring {
    int s = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step(int stages) {
        if (++s == stages) {
            s = 0;
            round ^= 1u;
        }
    }
};

__device__ __forceinline__ void tma_load_words(void *dst, const CUtensorMap *map, uint64_t *bar, int y) {
    tma_load_2d(dst, map, bar, 0, y);
}

// ---- few tokens: one CTA, or a cluster that splits K --------------------------------
constexpr int kMostStages = 6, kTileThreads = 192;
struct TileShared {
    uint64_t full[kMostStages], empty[kMostStages], done;
    uint32_t tmem_base;
    int abort;
};

template <int FORMAT, int NT>
struct TileCfg {
    static constexpr int kTokBytes = NT * kRowBytes, kScaleBytes = kStageWords<FORMAT> * 512;
    static constexpr int kStage = kChBytes + kTokBytes + 2 * kScaleBytes;
    static constexpr int kScaleCols = 8 * kStageWords<FORMAT>;  // of a stage: channels, tokens
    // two CTAs an SM
    static constexpr int kRoom = 233472 / 2 - 1024 - 1024 - static_cast<int>(sizeof(TileShared));
    static constexpr int kFit = kRoom / kStage < kMostStages ? kRoom / kStage : kMostStages;
    static constexpr int kStages = kFit;
    static constexpr uint32_t kCols = 256;
    static constexpr int kSmem = 1024 + kStages * kStage + static_cast<int>(sizeof(TileShared));
    static constexpr int kD = kStages * kScaleCols;  // first column of the accumulator
    static_assert(kD + (NT < 32 ? 32 : NT) <= static_cast<int>(kCols) && kStages >= 3, "tensor memory");
    static_assert(kStages * kStage >= NT * kTileCh * 4, "the exchange");
};

// Scales of up to 32 tokens from `first` on, one a lane: the warp's lanes hand them
// round (loaded token by token, each load waited for the store before it: an epilogue of
// 256 x 256 took 8 us).
__device__ __forceinline__ float token_scale(const Fp4Args &a, int first, int lane) {
    return !a.rowA ? 1.f : first + lane < a.M ? __ldcg(a.rowA + first + lane) : 0.f;
}

// `cols` sums of channel n to the rows first .. of C, with the scales and the bias; `sa`
// of lane FROM + j is the scale of sum j's token.
template <class El, int COLS, int FROM>
__device__ __forceinline__ void write_columns(const Fp4Args &a, int n, int first, int cols, const float (&acc)[COLS], float sb,
                                              float bias, float sa) {
    typename El::T *c = static_cast<typename El::T *>(a.C) + static_cast<long long>(first) * a.ldc + n;
    if (n >= a.N) cols = 0;
#pragma unroll
    for (int j = 0; j < COLS; ++j, c += a.ldc) {
        const float v = fmaf(acc[j] * sb, __shfl_sync(0xffffffffu, sa, FROM + j), bias);
        if (j < cols) *c = El::down(v);
    }
}

template <int FORMAT, int NT, int KS>
__global__ void __launch_bounds__(kTileThreads, 2)
fp4_tile_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA,
                const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmSA, const Fp4Args a) {
    using Cf = TileCfg<FORMAT, NT>;
    constexpr int S = Cf::kStages, W = kStageWords<FORMAT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    TileShared *sh = reinterpret_cast<TileShared *>(base + S * Cf::kStage);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = KS > 1 ? static_cast<int>(cluster_ctarank()) : 0, unit = static_cast<int>(blockIdx.x) / KS;
    const int tok_tiles = (a.M + NT - 1) / NT;
    const int ch0 = unit / tok_tiles * kTileCh, t0 = unit % tok_tiles * NT;
    const int kt = (a.K + kStageK - 1) / kStageK;
    const int k_first = static_cast<int>(static_cast<long long>(rank) * kt / KS);
    const int k_last = static_cast<int>(static_cast<long long>(rank + 1) * kt / KS);

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        mbar_init(&sh->done, 1);
        sh->abort = 0;
        fence_barrier_init();
    }
    if (warp == 5) {
        tc::tmem_alloc(&sh->tmem_base, Cf::kCols);
        tc::tmem_relinquish();
    }
    if (tid == 128) {
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmSB);
        prefetch_tensormap(&tmSA);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
    volatile int *abort_flag = &sh->abort;
    griddep_wait();
    griddep_launch_dependents();

    bool ok = true;
    if (warp == 4) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            Ring r;
            int issued = 0;
            for (int i = k_first; i < k_last; ++i, r.step(S), ++issued) {
                if (!mbar_wait(&sh->empty[r.s], r.round ^ 1u, a.status) || *abort_flag) {
                    *abort_flag = 1;
                    break;
                }
                uint8_t *st = base + r.s * Cf::kStage;
                mbar_arrive_expect_tx(&sh->full[r.s], Cf::kStage);
                tma_load_2d(st, &tmB, &sh->full[r.s], i * kRowBytes, ch0);
                tma_load_words(st + kChBytes + Cf::kTokBytes, &tmSB, &sh->full[r.s], ch0 / 128 * a.words + i * W);
                tma_load_2d(st + kChBytes, &tmA, &sh->full[r.s], i * kRowBytes, t0);
                tma_load_words(st + kChBytes + Cf::kTokBytes + Cf::kScaleBytes, &tmSA, &sh->full[r.s], t0 / 128 * a.words + i * W);
            }
            if (*abort_flag)  // no copy outlives the CTA
                for (int t = max(0, issued - S); t < issued; ++t) mbar_wait(&sh->full[t % S], (t / S) & 1, a.status);
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------ MMA issuer
        Ring r;
        for (int i = k_first; i < k_last; ++i, r.step(S)) {
            ok = mbar_wait(&sh->full[r.s], r.round, a.status) && !*abort_flag;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                *abort_flag = 1;
                break;
            }
            tc::fence_after_sync();
            if (tc::elect_one()) {
                const uint8_t *st = base + r.s * Cf::kStage;
                stage_mmas<FORMAT, 1, 1, NT>(tmem + Cf::kD, tmem + r.s * Cf::kScaleCols, tile_desc(st), tile_desc(st + kChBytes),
                                             scale_desc(st + kChBytes + Cf::kTokBytes),
                                             scale_desc(st + kChBytes + Cf::kTokBytes + Cf::kScaleBytes), a.K - i * kStageK,
                                             i == k_first);
                tc::commit(&sh->empty[r.s]);
            }
            __syncwarp();
        }
        if (tc::elect_one()) {
            tc::commit(&sh->done);
            if (!ok) mbar_wait(&sh->done, 0, a.status);  // no teardown under a running MMA
        }
        __syncwarp();
    } else if (warp < 4) {
        ok = mbar_wait(&sh->done, 0, a.status) && !*abort_flag;
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_after_sync();
    }
    const int n = ch0 + warp * 32 + lane;  // (the epilogue's warps)
    const uint32_t src = tmem + Cf::kD + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float sb = 1.f, bias = 0.f;
    if (warp < 4 && n < a.N) {
        if (a.rowB) sb = __ldcg(a.rowB + n);
        if (a.bias) bias = __ldcg(a.bias + n);
    }
    if (KS == 1) {
        if (warp < 4 && ok) {
#pragma unroll 1
            for (int c = 0; c < NT && t0 + c < a.M; c += 16) {
                const float sa = token_scale(a, t0 + c, lane & 15);
                float v[16];
                tc::tmem_ld16(src + c, v);
                with_type(a.out_type, [&](auto el) {
                    write_columns<decltype(el), 16, 0>(a, n, t0 + c, a.M - t0 - c, v, sb, bias, sa);
                });
            }
        }
    } else {
        // Rank r adds up the tokens [r * kPer, (r + 1) * kPer): every CTA's part of them
        // goes to its shared memory, over the stages that no one needs any longer.
        constexpr int kPer = NT / KS;
        const float sa = token_scale(a, t0 + rank * kPer, lane);  // (at most 64 tokens: lanes 0 to 31, and the second half below)
        const float sa2 = kPer > 32 ? token_scale(a, t0 + rank * kPer + 32, lane) : 0.f;
        cluster_sync();
        if (warp < 4 && ok) {
            const uint32_t here = smem_u32(base) + static_cast<uint32_t>((rank * kPer * kTileCh + warp * 32 + lane) * 4);
#pragma unroll
            for (int c = 0; c < NT; c += 16) {
                float v[16];
                tc::tmem_ld16(src + c, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t at = tc::map_shared_rank(here, static_cast<uint32_t>((c + j) / kPer)) +
                                        static_cast<uint32_t>((c + j) % kPer * kTileCh * 4);
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v[j]) : "memory");
                }
            }
        }
        // a CTA that gave up has left its part out: nothing is written by any of them
        if (!ok || *abort_flag) {
            if (lane == 0)
                for (int q = 0; q < KS; ++q)
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_addr(&sh->abort, static_cast<uint32_t>(q))), "r"(1) : "memory");
        }
        cluster_sync();
        if (warp < 4 && !*abort_flag) {
            const float *mine = reinterpret_cast<const float *>(base) + warp * 32 + lane;
            constexpr int kGo = kPer < 16 ? kPer : 16;
            const int t = t0 + rank * kPer;
#pragma unroll
            for (int j0 = 0; j0 < kPer; j0 += kGo) {
                if (t + j0 >= a.M) break;
                float v[kGo];
#pragma unroll
                for (int j = 0; j < kGo; ++j) {
                    v[j] = 0.f;
#pragma unroll
                    for (int q = 0; q < KS; ++q) v[j] += mine[(q * kPer + j0 + j) * kTileCh];
                }
                with_type(a.out_type, [&](auto el) {
                    // (token j0 + j: lane (j0 + j) % 32 of one scale or the other)
                    if (j0 % 32 == 0) write_columns<decltype(el), kGo, 0>(a, n, t + j0, a.M - t - j0, v, sb, bias, j0 < 32 ? sa : sa2);
                    else write_columns<decltype(el), kGo, 32 - kGo>(a, n, t + j0, a.M - t - j0, v, sb, bias, j0 < 32 ? sa : sa2);
                });
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 5) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, Cf::kCols);
    }
}

// ---- many tokens: CTA pairs ----------------------------------------------------------
constexpr int kPairThreads = 320, kPairTok = 256, kPairCh = 256;
struct PairShared {
    uint64_t full[kMostStages], empty[kMostStages], dfull, dempty, drained;
    uint32_t tmem_base;
    int abort;
};

template <int FORMAT>
struct PairCfg {
    static constexpr int kTokBytes = 128 * kRowBytes, kScaleBytes = kStageWords<FORMAT> * 512;
    static constexpr int kStage = kChBytes + kTokBytes + 3 * kScaleBytes;  // scales: own channels, all tokens
    static constexpr int kScaleCols = 12 * kStageWords<FORMAT>;
    static constexpr int kStages = 5;
    static constexpr uint32_t kCols = 512;
    static constexpr int kSmem = 1024 + kStages * kStage + static_cast<int>(sizeof(PairShared));
    static constexpr int kD = kStages * kScaleCols;
    static_assert(kD + kPairTok <= static_cast<int>(kCols) && kSmem <= kSmemLimit, "a CTA's memory");
};

// Tile order: groups of 8 channel tiles, whose tokens' tiles are then in L2 together.
__device__ __forceinline__ void pair_tile(int u, int ch_tiles, int tok_tiles, int &ch, int &tok) {
    constexpr int kGroup = 8;
    const int per = kGroup * tok_tiles, g = u / per, first = g * kGroup, wide = min(ch_tiles - first, kGroup), r = u - g * per;
    ch = first + r % wide;
    tok = r / wide;
}

template <int FORMAT>
__global__ void __launch_bounds__(kPairThreads, 1)
fp4_pair_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA,
                const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmSA, const Fp4Args a) {
    using Cf = PairCfg<FORMAT>;
    constexpr int S = Cf::kStages, W = kStageWords<FORMAT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // the same in both CTAs
    PairShared *sh = reinterpret_cast<PairShared *>(base + S * Cf::kStage);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());  // 0: issues the MMAs
    const int ch_tiles = (a.N + kPairCh - 1) / kPairCh, tok_tiles = (a.M + kPairTok - 1) / kPairTok;
    const int units = ch_tiles * tok_tiles, first_unit = static_cast<int>(blockIdx.x) >> 1, unit_step = static_cast<int>(gridDim.x) >> 1;
    const int kt = (a.K + kStageK - 1) / kStageK;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        mbar_init(&sh->dfull, 1);
        mbar_init(&sh->dempty, 16);
        mbar_init(&sh->drained, 1);
        sh->abort = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tc::tmem_alloc_pair(&sh->tmem_base, Cf::kCols);
        tc::tmem_relinquish_pair();
    }
    if (tid == 256) {
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmSB);
        prefetch_tensormap(&tmSA);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync_all();  // both CTAs' barriers are initialised before any cross-CTA arrive
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
    volatile int *abort_flag = &sh->abort;
    griddep_wait();
    griddep_launch_dependents();
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity, a.status)) return true;
        *abort_flag = 1;
        return false;
    };

    if (warp == 8) {
        // ------------------------------------------------ TMA producer (each CTA; both count on the even one's barrier)
        if (lane == 0) {
            const uint32_t full = tc::map_shared_rank(smem_u32(&sh->full[0]), 0);
            Ring r;
            bool ok = true;
            for (int u = first_unit; u < units && ok; u += unit_step) {
                int ch, tok;
                pair_tile(u, ch_tiles, tok_tiles, ch, tok);
                const int ch0 = ch * kPairCh + rank * 128, t0 = tok * kPairTok;
                for (int i = 0; i < kt; ++i, r.step(S)) {
                    if (!wait(&sh->empty[r.s], r.round ^ 1u)) { ok = false; break; }
                    uint8_t *st = base + r.s * Cf::kStage;
                    uint8_t *sc = st + kChBytes + Cf::kTokBytes;
                    const uint32_t bar = full + r.s * 8;
                    if (rank == 0) mbar_arrive_expect_tx(&sh->full[r.s], 2 * Cf::kStage);
                    tc::tma_load_2d_pair(st, &tmB, bar, i * kRowBytes, ch0);
                    tc::tma_load_2d_pair(st + kChBytes, &tmA, bar, i * kRowBytes, t0 + rank * 128);
                    tc::tma_load_2d_pair(sc, &tmSB, bar, 0, ch0 / 128 * a.words + i * W);
                    tc::tma_load_2d_pair(sc + Cf::kScaleBytes, &tmSA, bar, 0, t0 / 128 * a.words + i * W);
                    tc::tma_load_2d_pair(sc + 2 * Cf::kScaleBytes, &tmSA, bar, 0, (t0 / 128 + 1) * a.words + i * W);
                }
            }
            // No copy outlives its CTA: the MMAs that read the last ones have finished
            // (a stage that was never loaded stands at its first round).
            for (int s = 0; s < S; ++s, r.step(S)) mbar_wait(&sh->empty[r.s], r.round ^ 1u, a.status);
        }
        __syncwarp();
    } else if (warp == 9 && rank == 0) {
        // ------------------------------------------------ MMA issuer (even CTA)
        Ring r;
        uint32_t dround = 0;
        bool ok = true;
        for (int u = first_unit; u < units && ok; u += unit_step, dround ^= 1u) {
            ok = __all_sync(0xffffffffu, wait(&sh->dempty, dround ^ 1u));
            if (!ok) break;
            for (int i = 0; i < kt; ++i, r.step(S)) {
                ok = __all_sync(0xffffffffu, wait(&sh->full[r.s], r.round));
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint8_t *st = base + r.s * Cf::kStage, *sc = st + kChBytes + Cf::kTokBytes;
                    stage_mmas<FORMAT, 2, 2, kPairTok>(tmem + Cf::kD, tmem + r.s * Cf::kScaleCols, tile_desc(st), tile_desc(st + kChBytes),
                                                       scale_desc(sc), scale_desc(sc + Cf::kScaleBytes), a.K - i * kStageK, i == 0);
                    tc::commit_pair(&sh->empty[r.s], 0x3);
                    if (i + 1 == kt) tc::commit_pair(&sh->dfull, 0x3);
                }
                __syncwarp();
            }
        }
        if (!ok && tc::elect_one()) {  // no teardown under a running MMA
            tc::commit_pair(&sh->drained, 0x1);
            mbar_wait(&sh->drained, 0, a.status);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ------------------------------------------------ accumulators to C: warps 4 to 7 the second half of the tokens
        constexpr int kCols = kPairTok / 2;
        const int half = warp / 4, in_tile = (warp % 4) * 32 + lane;
        const uint32_t src = tmem + Cf::kD + half * kCols + (static_cast<uint32_t>(warp % 4 * 32) << 16);
        const uint32_t dempty = tc::map_shared_rank(smem_u32(&sh->dempty), 0);
        uint32_t round = 0;
        for (int u = first_unit; u < units; u += unit_step, round ^= 1u) {
            int ch, tok;
            pair_tile(u, ch_tiles, tok_tiles, ch, tok);
            const int n = ch * kPairCh + rank * 128 + in_tile, t0 = tok * kPairTok + half * kCols;
            float sb = 1.f, bias = 0.f;
            if (n < a.N) {
                if (a.rowB) sb = __ldcg(a.rowB + n);
                if (a.bias) bias = __ldcg(a.bias + n);
            }
            float sa[kCols / 32];
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) sa[c] = token_scale(a, t0 + c * 32, lane);
            if (!__all_sync(0xffffffffu, wait(&sh->dfull, round))) break;
            tc::fence_after_sync();
            uint32_t v[kCols / 16][16];
#pragma unroll
            for (int c = 0; c < kCols / 16; ++c) tc::tmem_ld16_begin(src + c * 16, v[c]);
#pragma unroll
            for (int c = 0; c < kCols / 16; ++c) tc::tmem_ld_wait(v[c]);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_remote(dempty);
            with_type(a.out_type, [&](auto el) {
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    float f[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[2 * c + j / 16][j % 16]);
                    if (t0 + c * 32 < a.M) write_columns<decltype(el), 32, 0>(a, n, t0 + c * 32, a.M - t0 - c * 32, f, sb, bias, sa[c]);
                }
            });
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync_all();  // the peer is done with this CTA's barriers and tensor memory
    if (warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(tmem, Cf::kCols);
    }
}

// ---- any layout: CUDA cores ----------------------------------------------------------
constexpr int kGTile = 64, kGK = 32;

// An element of format MX may pass FP32's range with its scale (2^126 and 2^127) where its products do
// not: both operands are taken at a quarter, which is exact, and the sum 16 times (exact, as are the
// products, but for sums that would be subnormal: those are off by 2^-145 a term at most).
template <int FORMAT>
__global__ void __launch_bounds__(256) fp4_generic_kernel(const Fp4Args a) {
    constexpr float kLess = FORMAT == SGEMM_FP4_MX ? 0.25f : 1.f;
    __shared__ float at[kGK][kGTile + 4], bt[kGK][kGTile + 4];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16, n0 = blockIdx.x * kGTile;
    for (long long m0 = static_cast<long long>(blockIdx.y) * kGTile; m0 < a.M; m0 += static_cast<long long>(gridDim.y) * kGTile) {
        float acc[4][4] = {};
        for (int k0 = 0; k0 < a.K; k0 += kGK) {
            // 64 rows of 32 elements of each operand: 8 elements (4 bytes) a thread
            const int r = tid / 4, p0 = k0 + tid % 4 * 8;
            auto fetch = [&](float (*to)[kGTile + 4], const uint8_t *q, long long ld, const uint8_t *s, long long row, int rows) {
                uint32_t code = 0, scale = 0;
                if (row < rows && p0 < a.K) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (p0 + 2 * j < a.K) code |= static_cast<uint32_t>(__ldcg(q + row * ld + p0 / 2 + j)) << (8 * j);
                    const int b = p0 / fp4_block(FORMAT);
                    scale = __ldcg(s + fp4_scale_word(row, b / 4, a.words) + (b & 3));
                }
                uint32_t h[4];
                from_e2m1x8(code, h);
                const float f = fp4_scale<FORMAT>(scale) * kLess;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    to[tid % 4 * 8 + e][r] = __half2float(__ushort_as_half(static_cast<uint16_t>(h[e / 2] >> (16 * (e & 1))))) * f;
            };
            fetch(at, a.A, a.lda, a.SA, m0 + r, a.M);
            fetch(bt, a.B, a.ldb, a.SB, static_cast<long long>(n0) + r, a.N);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kGK; ++k) {
                float x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = at[k][ty * 4 + j];
                    y[j] = bt[k][tx * 4 + j];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
            }
            __syncthreads();
        }
        with_type(a.out_type, [&](auto el) {
            using El = decltype(el);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long m = m0 + ty * 4 + i;
                if (m >= a.M) break;
                const float sa = a.rowA ? __ldcg(a.rowA + m) : 1.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = n0 + tx * 4 + j;
                    if (n >= a.N) break;
                    const float sb = a.rowB ? __ldcg(a.rowB + n) : 1.f;
                    static_cast<typename El::T *>(a.C)[m * a.ldc + n] = El::down(fmaf(acc[i][j] * (1.f / (kLess * kLess)) * sb, sa, a.bias ? __ldcg(a.bias + n) : 0.f));
                }
            }
        });
    }
}

template <int FORMAT, int NT, int KS>
cudaError_t launch_split(const Fp4Args &a, const Fp4Maps &m, int smem, cudaStream_t stream) {
    const unsigned units = static_cast<unsigned>((a.N + kTileCh - 1) / kTileCh) * static_cast<unsigned>((a.M + NT - 1) / NT);
    return launch_dependent(fp4_tile_kernel<FORMAT, NT, KS>, dim3(units * KS), dim3(kTileThreads), smem > 0 ? smem : TileCfg<FORMAT, NT>::kSmem,
                            stream, KS, m.B, m.A, m.SB, m.SA, a);
}

template <int FORMAT, int NT>
cudaError_t launch_tile(const Fp4Args &a, const Fp4Maps &m, int smem, cudaStream_t stream) {
    switch (a.ksplit) {
        case 1: return launch_split<FORMAT, NT, 1>(a, m, smem, stream);
        case 2: return launch_split<FORMAT, NT, 2>(a, m, smem, stream);
        case 4: return launch_split<FORMAT, NT, 4>(a, m, smem, stream);
        default: return launch_split<FORMAT, NT, 8>(a, m, smem, stream);
    }
}

template <int FORMAT>
cudaError_t launch_format(const Fp4Args &a, const Fp4Maps &m, int num_sms, int smem, cudaStream_t stream) {
    switch (a.nt) {
        case 16: return launch_tile<FORMAT, 16>(a, m, smem, stream);
        case 32: return launch_tile<FORMAT, 32>(a, m, smem, stream);
        case 64: return launch_tile<FORMAT, 64>(a, m, smem, stream);
        case 128: return launch_tile<FORMAT, 128>(a, m, smem, stream);
        default: {
            const long long units = static_cast<long long>((a.N + kPairCh - 1) / kPairCh) * ((a.M + kPairTok - 1) / kPairTok);
            const long long pairs = units < num_sms / 2 ? units : num_sms / 2;
            return launch_dependent(fp4_pair_kernel<FORMAT>, dim3(static_cast<unsigned>(2 * pairs)), dim3(kPairThreads), smem > 0 ? smem : PairCfg<FORMAT>::kSmem,
                                    stream, 2, m.B, m.A, m.SB, m.SA, a);
        }
    }
}

template <int FORMAT, int NT>
cudaError_t prepare_tile() {
    cudaError_t e = cudaSuccess;
    for (auto *k : {fp4_tile_kernel<FORMAT, NT, 1>, fp4_tile_kernel<FORMAT, NT, 2>, fp4_tile_kernel<FORMAT, NT, 4>, fp4_tile_kernel<FORMAT, NT, 8>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, TileCfg<FORMAT, NT>::kSmem);
    return e;
}

template <int FORMAT>
cudaError_t prepare_format() {
    cudaError_t e = cudaFuncSetAttribute(fp4_pair_kernel<FORMAT>, cudaFuncAttributeMaxDynamicSharedMemorySize, PairCfg<FORMAT>::kSmem);
    for (cudaError_t r : {prepare_tile<FORMAT, 16>(), prepare_tile<FORMAT, 32>(), prepare_tile<FORMAT, 64>(), prepare_tile<FORMAT, 128>()})
        if (e == cudaSuccess) e = r;
    return e;
}

}  // namespace

cudaError_t fp4_prepare() {
    const cudaError_t e = prepare_format<SGEMM_FP4_MX>();
    return e != cudaSuccess ? e : prepare_format<SGEMM_FP4_NV>();
}

cudaError_t launch_fp4_tc(const Fp4Args &a, const Fp4Maps &m, int num_sms, int smem_override, cudaStream_t stream) {
    return a.format == SGEMM_FP4_MX ? launch_format<SGEMM_FP4_MX>(a, m, num_sms, smem_override, stream)
                                    : launch_format<SGEMM_FP4_NV>(a, m, num_sms, smem_override, stream);
}

cudaError_t launch_fp4_generic(const Fp4Args &a, cudaStream_t stream) {
    const int y = (a.M + kGTile - 1) / kGTile;
    const dim3 grid((a.N + kGTile - 1) / kGTile, y < 65535 ? y : 65535);
    return launch_dependent(a.format == SGEMM_FP4_MX ? fp4_generic_kernel<SGEMM_FP4_MX> : fp4_generic_kernel<SGEMM_FP4_NV>, grid, dim3(256), 0, stream, 1, a);
}

}  // namespace sg
