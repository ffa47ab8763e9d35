// 8-bit integer products for sm_103a:
//
//   C[i][j] = (sum_p A[i][p] * B_e[j][p]) * scaleB[e][j] * scaleA[i] + bias[e][j]
//
// with A (tokens x K) and B_e (channels x K) in int8, one scale a token and one
// a channel, C in FP32, BF16 or FP16; e is the expert that owns row i (one
// expert owns every row in the dense call).  The sum is exact in 32-bit
// integers; float(sum) * scaleB * scaleA (+ bias) is rounded to the output type
// once.
//
// The tensor cores of sm_103a have no 8-bit integer MMA (.kind::i8 is not
// assembled for it) and the CUDA cores' and mma.sync's integer rates are far
// below the 16-bit rate of tcgen05.  An int8 is exact in FP16, a product of two
// in FP32, and a sum of 1024 such products has magnitude <= 2^24, so it is an
// integer that FP32 holds exactly: the kernel multiplies with .kind::f16, FP32
// accumulators in tensor memory, and moves them into int32 registers every
// 1024 k.  Sums of integers do not depend on their order, so every split of K
// gives the same bits.
//
//  * int8_tc_kernel -- D[channel][token] = B * A^T with the channels as the
//    MMA's M (128 rows) and a tile of NT tokens as its N, so that few tokens
//    cost a narrow tile and not a padded one.  B crosses HBM and shared memory
//    as int8 (half the bytes of 16-bit operands; it is what a decode step is
//    bound by) and becomes FP16 only on its way into tensor memory, where the
//    MMA reads it as its A operand: shared memory sees one 8-bit write and one
//    8-bit read of it.  The tokens' rows are converted to FP16 once, by
//    int8_to_f16_kernel, and read by TMA.
//      warp 0     TMA producer: a ring of stages of 128 k (B: 128 x 128 bytes,
//                 tokens: two swizzled boxes of 64 k x NT)
//      warp 1     one lane issues the MMAs; owns the tensor memory
//      warp 2     sums up the experts' token tiles once, at the start
//      warps 4-11 two warpgroups convert half of each stage: a thread reads 64
//                 bytes of its channel (16 at a time, conflict-free through the
//                 swizzle), turns byte b into the FP16 bits 0x6400 + (b ^ 0x80)
//                 = 1152 + b, subtracts 1152 (exact), and stores 32 columns of
//                 tensor memory.  (Alternate stages would not do: a warp that
//                 skips a phase of a stage's barrier cannot tell by its parity
//                 whether the phase before has ended when the ring is odd.)
//      warps 12.. one or two warpgroups drain the accumulators (two of NT
//                 columns each, so that the next 1024 k start at once) and
//                 write C: a warp's lanes are 32 consecutive channels of a token
//    Tensor memory: 2 x NT accumulator columns and 4 stages of 64 columns of B.
//    Persistent over (expert, token tile, channel tile) units, token tiles
//    innermost within groups of 16 so that concurrent CTAs share B's tiles in L2.
//    With few tiles the 2, 4 or 8 CTAs of a cluster share a tile's K range;
//    each sends the others their columns' int32 partial sums through
//    distributed shared memory (tiles of up to 64 tokens, one epilogue warpgroup).
//  * int8_generic_kernel -- any layout and alignment, dp4a on the CUDA cores.
//  * int8_to_f16_kernel, int8_relayout_kernel -- the tokens' rows as FP16, and B
//    as the TMA can read it (stored K x N, or not on 16-byte boundaries).
// Every wait is bounded; on a timeout the kernel records it, waits (bounded)
// for its own copies and MMAs in flight, frees the tensor memory and returns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "internal.h"
#include "sgemm.h"
#include "tcgen05.cuh"

namespace sg {
namespace {

// ---- epilogue arithmetic, common to both kernels --------------------------------
__device__ __forceinline__ float int8_value(int sum, float sb, float sa, float bias) {
    return fmaf(__int2float_rn(sum) * sb, sa, bias);
}

// Two values of the output type from one conversion, and the store of one or
// the other.
struct OutF32 {
    using T = float;
    using Two = float2;
    static __device__ __forceinline__ Two two(float a, float b) { return make_float2(a, b); }
    static __device__ __forceinline__ T lo(Two v) { return v.x; }
    static __device__ __forceinline__ T hi(Two v) { return v.y; }
};
struct OutBF16 {
    using T = __nv_bfloat16;
    using Two = __nv_bfloat162;
    static __device__ __forceinline__ Two two(float a, float b) { return __floats2bfloat162_rn(a, b); }
    static __device__ __forceinline__ T lo(Two v) { return __low2bfloat16(v); }
    static __device__ __forceinline__ T hi(Two v) { return __high2bfloat16(v); }
};
struct OutF16 {
    using T = __half;
    using Two = __half2;
    static __device__ __forceinline__ Two two(float a, float b) { return __floats2half2_rn(a, b); }
    static __device__ __forceinline__ T lo(Two v) { return __low2half(v); }
    static __device__ __forceinline__ T hi(Two v) { return __high2half(v); }
};

// Call f with the output type's traits.
template <class F>
__device__ __forceinline__ void with_out_type(int type, F &&f) {
    if (type == SGEMM_IN_BF16) f(OutBF16{});
    else if (type == SGEMM_IN_F16) f(OutF16{});
    else f(OutF32{});
}

// A thread's COLS sums (one channel, COLS tokens) to C: C points at the first
// token's element of the channel, `live` tokens exist (live <= 0: none, and a
// channel that does not exist has none).  sa: lane l holds the scales of tokens
// l, l + 32, ..  The whole warp takes part.  A warp whose tokens and channels all
// exist, as in every tile but those at the edges, runs without predicates: the
// code is unrolled over the registers that hold the sums, and its size counts
// (it is fetched anew for every tile).
template <class Out, int COLS>
__device__ __forceinline__ void write_columns(typename Out::T *C, long long ldc, int live, const int (&acc)[COLS],
                                              const float (&sa)[(COLS + 31) / 32], float sb, float bias) {
    if (__all_sync(0xffffffffu, live >= COLS)) {
#pragma unroll
        for (int j = 0; j < COLS; j += 2) {
            const float s0 = __shfl_sync(0xffffffffu, sa[j / 32], j % 32);
            const float s1 = __shfl_sync(0xffffffffu, sa[j / 32], j % 32 + 1);
            const typename Out::Two v =
                Out::two(int8_value(acc[j], sb, s0, bias), int8_value(acc[j + 1], sb, s1, bias));
            C[0] = Out::lo(v);
            C[ldc] = Out::hi(v);
            C += 2 * ldc;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < COLS; j += 2) {
        const float s0 = __shfl_sync(0xffffffffu, sa[j / 32], j % 32);
        const float s1 = __shfl_sync(0xffffffffu, sa[j / 32], j % 32 + 1);
        const typename Out::Two v = Out::two(int8_value(acc[j], sb, s0, bias), int8_value(acc[j + 1], sb, s1, bias));
        if (j < live) C[0] = Out::lo(v);
        if (j + 1 < live) C[ldc] = Out::hi(v);
        C += 2 * ldc;
    }
}

// offsets[e], kept within the rows there are (whatever the array holds).
__device__ __forceinline__ int bound_of(const Int8Args &a, int e) {
    if (!a.offsets) return e == 0 ? 0 : a.total_rows;
    return min(max(__ldg(a.offsets + e), 0), a.total_rows);
}

// ---- generic kernel -----------------------------------------------------------
// 64 x 64 tile of C, 64 k a step as 16 packed words a row, 4 x 4 sums a thread.
constexpr int kGTile = 64, kGWords = 16;

__global__ void __launch_bounds__(256) int8_generic_kernel(const Int8Args a) {
    __shared__ int As[kGWords][kGTile + 1], Bs[kGWords][kGTile + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int n0 = blockIdx.x * kGTile;
    for (int e = blockIdx.z; e < a.experts; e += gridDim.z) {
        const int8_t *B = a.B + e * a.strideB;
        const int lo = max(bound_of(a, e), a.row0), hi = min(bound_of(a, e + 1), a.row0 + a.rows);
        for (int m0 = lo + static_cast<int>(blockIdx.y) * kGTile; m0 < hi; m0 += static_cast<int>(gridDim.y) * kGTile) {
            int acc[4][4] = {};
            for (int k0 = 0; k0 < a.K; k0 += 4 * kGWords) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = tid + r * 256, w = at % kGWords, i = at / kGWords;
                    unsigned av = 0, bv = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int k = k0 + 4 * w + b;
                        if (k >= a.K) break;
                        if (m0 + i < hi)
                            av |= static_cast<unsigned>(static_cast<uint8_t>(a.A[static_cast<long long>(m0 + i) * a.lda + k])) << (8 * b);
                        if (n0 + i < a.N)
                            bv |= static_cast<unsigned>(static_cast<uint8_t>(
                                      a.transB ? B[static_cast<long long>(n0 + i) * a.ldb + k]
                                               : B[static_cast<long long>(k) * a.ldb + n0 + i])) << (8 * b);
                    }
                    As[w][i] = static_cast<int>(av);
                    Bs[w][i] = static_cast<int>(bv);
                }
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kGWords; ++w) {
                    int x[4], y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = As[w][ty + 16 * i];
                        y[i] = Bs[w][tx + 16 * i];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(x[i], y[j], acc[i][j]);
                }
                __syncthreads();
            }
            with_out_type(a.out_type, [&](auto out) {
                using Out = decltype(out);
                auto *C = static_cast<typename Out::T *>(a.C);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = m0 + ty + 16 * i;
                    if (row >= hi) continue;
                    const float sa = __ldg(a.scaleA + row);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int ch = n0 + tx + 16 * j;
                        if (ch >= a.N) continue;
                        const long long at = static_cast<long long>(e) * a.N + ch;
                        const float v =
                            int8_value(acc[i][j], __ldg(a.scaleB + at), sa, a.bias ? __ldg(a.bias + at) : 0.f);
                        C[static_cast<long long>(row) * a.ldc + ch] = Out::lo(Out::two(v, 0.f));
                    }
                }
            });
        }
    }
}

// ---- operand copies -------------------------------------------------------------
// Four int8 (a word) as two pairs of FP16: 0x6400 + u is the FP16 value 1024 + u,
// u = b + 128 the biased byte; minus 1152 gives b, exactly.
__device__ __forceinline__ void int8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t p = __byte_perm(u, 0x64646464u, 0x4140), q = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&p), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&q), off);
    lo = *reinterpret_cast<const uint32_t *>(&a);
    hi = *reinterpret_cast<const uint32_t *>(&b);
}

// Bytes p[0..15] of a row of which `n` remain (zeros beyond).
__device__ __forceinline__ uint4 load_int8x16(const int8_t *p, int n, bool vec) {
    if (vec && n >= 16) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) w[i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(p[i])) << (8 * (i % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 k a thread; ldd is a multiple of 64, so its rows divide into whole threads.
// peaks[block]: the largest sum of |a| over the 512 k (of one row, or the end of
// one and the start of the next) that a warp of the block converts at a time.
__global__ void __launch_bounds__(256)
int8_to_f16_kernel(const int8_t *__restrict__ A, long long lda, int rows, int K, uint4 *__restrict__ dst, int ldd,
                   int vec, int *__restrict__ peaks) {
    __shared__ int part[8];
    griddep_wait();
    griddep_launch_dependents();
    const int per_row = ldd / 16;
    const long long total = static_cast<long long>(rows) * per_row;
    int top = 0;
    for (long long i0 = blockIdx.x * 256ll; i0 < total; i0 += gridDim.x * 256ll) {
        const long long i = i0 + threadIdx.x;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i < total) {
            const long long row = div_floor(i, per_row);
            const int k = static_cast<int>(i - row * per_row) * 16;
            if (k < K) v = load_int8x16(A + row * lda + k, K - k, vec);
            uint4 o0, o1;
            int8x4_to_f16(v.x, o0.x, o0.y);
            int8x4_to_f16(v.y, o0.z, o0.w);
            int8x4_to_f16(v.z, o1.x, o1.y);
            int8x4_to_f16(v.w, o1.z, o1.w);
            dst[2 * i] = o0;
            dst[2 * i + 1] = o1;
        }
        unsigned sum = 0;  // |-128| is the byte 128 to an unsigned dot product
        sum = __dp4a(__vabs4(v.x), 0x01010101u, sum);
        sum = __dp4a(__vabs4(v.y), 0x01010101u, sum);
        sum = __dp4a(__vabs4(v.z), 0x01010101u, sum);
        sum = __dp4a(__vabs4(v.w), 0x01010101u, sum);
        top = max(top, static_cast<int>(__reduce_add_sync(0xffffffffu, sum)));
    }
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) top = max(top, part[w]);
        peaks[blockIdx.x] = top;
    }
}

// B stored N x K, rows copied onto 16-byte boundaries: 16 k a thread.
__global__ void __launch_bounds__(256)
int8_realign_kernel(const int8_t *__restrict__ B, long long ldb, long long strideB, int N, int K,
                    int8_t *__restrict__ dst, int ldd) {
    griddep_wait();
    griddep_launch_dependents();
    const int per_row = ldd / 16;
    const int8_t *src = B + blockIdx.y * strideB;
    int8_t *d = dst + static_cast<long long>(blockIdx.y) * N * ldd;
    const long long total = static_cast<long long>(N) * per_row;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const long long row = div_floor(i, per_row);
        const int k = static_cast<int>(i - row * per_row) * 16;
        reinterpret_cast<uint4 *>(d)[i] = load_int8x16(src + row * ldb + k, K - k, false);
    }
}

// B stored K x N -> N x ldd: a tile of 128 k x 64 channels through shared memory
// (rows of 65 bytes: the 8 lanes that gather 16 k each of one channel fall in
// distinct banks).
constexpr int kTK = 128, kTN = 64;

__global__ void __launch_bounds__(256)
int8_transpose_kernel(const int8_t *__restrict__ B, long long ldb, long long strideB, int N, int K,
                      int8_t *__restrict__ dst, int ldd) {
    __shared__ uint8_t tile[kTK][kTN + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int8_t *src = B + blockIdx.z * strideB;
    int8_t *d = dst + static_cast<long long>(blockIdx.z) * N * ldd;
    const int k0 = blockIdx.x * kTK;
    for (int n0 = blockIdx.y * kTN; n0 < N; n0 += gridDim.y * kTN) {
        uint8_t v[kTK * kTN / 256];
#pragma unroll
        for (int r = 0; r < kTK * kTN / 256; ++r) {
            const int at = threadIdx.x + r * 256, k = at / kTN, n = at % kTN;
            v[r] = (k0 + k < K && n0 + n < N) ? static_cast<uint8_t>(src[static_cast<long long>(k0 + k) * ldb + n0 + n]) : 0;
        }
#pragma unroll
        for (int r = 0; r < kTK * kTN / 256; ++r) {
            const int at = threadIdx.x + r * 256;
            tile[at / kTN][at % kTN] = v[r];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kTN * (kTK / 16) / 256; ++r) {
            const int at = threadIdx.x + r * 256, kg = at % (kTK / 16), n = at / (kTK / 16);
            if (n0 + n < N && k0 + kg * 16 < ldd) {
                uint32_t w[4] = {};
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i / 4] |= static_cast<uint32_t>(tile[kg * 16 + i][n]) << (8 * (i % 4));
                *reinterpret_cast<uint4 *>(d + static_cast<long long>(n0 + n) * ldd + k0 + kg * 16) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncthreads();
    }
}

// ---- tensor-core kernel -----------------------------------------------------------
constexpr int kBBytes = kI8TileN * kI8StageK;  // 16 KiB of B a stage
constexpr int kAStages = 4, kACols = kI8StageK / 2;  // stages of B in tensor memory, 32-bit columns each
constexpr int kChunk = 8;                       // stages (1024 k) whose sums fit an accumulator whatever the data
constexpr int kConvWGs = 2;                     // warpgroups that convert B, alternate stages
constexpr uint32_t kI8TmemCols = 512;
constexpr int kMaxStages = 10;
constexpr int kSmemLimit = 232448;

struct I8Shared {
    uint64_t bfull[kMaxStages];   // B (DIRECT: and the tokens' int8) of the stage has landed
    uint64_t bempty[kMaxStages];  // a warpgroup's four warps (DIRECT: and four more) have read it
    uint64_t xfull[kMaxStages];   // the tokens of the stage stand in shared memory
    uint64_t xempty[kMaxStages];  // the MMAs have read them
    uint64_t afull[kAStages];     // the stage's B stands in tensor memory (four warps)
    uint64_t aempty[kAStages];    // the MMAs that read it have finished
    uint64_t dfull[2];            // an accumulator holds up to 1024 k
    uint64_t dempty[2];           // it has been read
    uint64_t drained;             // abort only: every MMA issued has finished
    uint32_t tmem_base;
    int abort;
    int units;                    // units of this launch
    int chunk;                    // stages between drains of an accumulator
    int bound[kMaxExperts + 1];   // first row of each expert, nondecreasing
    int tiles[kMaxExperts + 1];   // token tiles of the experts before
};

// DIRECT: the tokens' int8 rows come with B's stages and are expanded to FP16
// here, by four warps; else they are read as FP16 by TMA.
template <int NT, bool SPLIT, bool DIRECT>
struct I8Cfg {
    static constexpr int kXBytes = NT * kI8StageK * 2;
    static constexpr int kXchg = SPLIT ? kI8TileN * NT * 4 : 0;  // partial sums from the cluster's CTAs
    static constexpr int kFree = kSmemLimit - 1024 - static_cast<int>(sizeof(I8Shared)) - kXchg;
    static constexpr int kStage = kBBytes + (DIRECT ? NT * kI8StageK : 0);
    // Rings: up to 32 KiB of FP16 tokens (at least two stages, three where TMA
    // fetches them from L2), and the stages of B in what is left.  An even
    // number of B's stages, so that a converting warpgroup sees every phase of
    // the stages it reads: the parity of a phase tells it from the one before
    // only.
    static constexpr int kXStages = !DIRECT ? 3 : 32768 / kXBytes < 4 ? 32768 / kXBytes : 4;
    static constexpr int kBFit = (kFree - kXStages * kXBytes) / kStage / 2 * 2;
    static constexpr int kBStages = kBFit < kMaxStages ? kBFit : kMaxStages;
    static constexpr int kRing = kBStages * kStage + kXStages * kXBytes;
    static constexpr int kSmem = 1024 + kRing + kXchg + static_cast<int>(sizeof(I8Shared));
    static constexpr int kEpiWGs = NT > 64 ? 2 : 1;
    static constexpr int kCols = NT / kEpiWGs;  // accumulator columns a thread drains
    static constexpr int kWarpX = 4, kWarpConv = kWarpX + (DIRECT ? 4 : 0), kWarpEpi = kWarpConv + 4 * kConvWGs;
    static constexpr int kThreads = 32 * (kWarpEpi + 4 * kEpiWGs);
    static constexpr int kPieces = NT / 16;              // 16-byte pieces of a stage's tokens a thread expands
    static_assert(2 * NT + kAStages * kACols <= static_cast<int>(kI8TmemCols), "tensor memory");
    static_assert(kBStages >= 4 && kBStages % kConvWGs == 0 && kXStages >= 2 && kXStages <= kMaxStages, "rings");
    static_assert(!SPLIT || (kEpiWGs == 1 && NT / 2 <= 32), "a lane holds a token scale");
    static_assert(kAStages % kConvWGs == 0 && kSmem <= kSmemLimit, "shared memory");
};

// acc[j] += column j of an accumulator (integers): the load of the next 16
// columns is in flight while 16 are converted.
template <int COLS>
__device__ __forceinline__ void drain(uint32_t tmem, int (&acc)[COLS]) {
    uint32_t v[2][16];
    tc::tmem_ld16_begin(tmem, v[0]);
    tc::tmem_ld_wait(v[0]);
#pragma unroll
    for (int c = 0; c < COLS / 16; ++c) {
        if (c + 1 < COLS / 16) tc::tmem_ld16_begin(tmem + (c + 1) * 16, v[(c + 1) & 1]);
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[c * 16 + j] += __float2int_rn(__uint_as_float(v[c & 1][j]));
        if (c + 1 < COLS / 16) tc::tmem_ld_wait(v[(c + 1) & 1]);
    }
}

struct I8Unit {
    int e, ch0, t0, tend;
};

// Unit u of tiles of NT tokens x CH channels: the expert by bisection of the
// tile counts; within the expert groups of 2048 tokens or 16 tiles, channel
// tiles outer and token tiles inner.
template <int NT, int CH, class Shared>
__device__ __forceinline__ I8Unit unit_of(const Shared *sh, const Int8Args &a, int ch_tiles, int u) {
    int lo = 0, hi = a.experts;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (sh->tiles[mid] * ch_tiles <= u) lo = mid; else hi = mid;
    }
    constexpr int kGroup = 2048 / NT < 16 ? 2048 / NT : 16;
    const int mine = sh->tiles[lo + 1] - sh->tiles[lo];
    const int l = u - sh->tiles[lo] * ch_tiles;
    const int grp = l / (kGroup * ch_tiles), first = grp * kGroup;
    const int rows = min(mine - first, kGroup);
    const int r = l - grp * kGroup * ch_tiles;
    I8Unit q;
    q.e = lo;
    q.ch0 = r / rows * CH;
    q.t0 = max(sh->bound[lo], a.row0) + (first + r % rows) * NT;
    q.tend = min(sh->bound[lo + 1], a.row0 + a.rows);
    return q;
}

// One warp: the experts' first rows and the sums of their token tiles.
template <class Shared>
__device__ __forceinline__ void sum_tiles(Shared *sh, const Int8Args &a, int nt, int ch_tiles, int lane) {
    int top = 0, sum = 0;
    for (int e0 = 0; e0 <= a.experts; e0 += 32) {
        const int e = e0 + lane;
        int b = e <= a.experts ? bound_of(a, e) : 0;
        b = max(b, top);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, b, d);
            if (lane >= d) b = max(b, up);
        }
        if (e <= a.experts) sh->bound[e] = b;
        top = __shfl_sync(0xffffffffu, b, 31);
    }
    __syncwarp();
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
        const int e = e0 + lane;
        int n = 0;
        if (e < a.experts) {
            const int lo = max(sh->bound[e], a.row0), hi = min(sh->bound[e + 1], a.row0 + a.rows);
            n = hi > lo ? (hi - lo + nt - 1) / nt : 0;
        }
        int s = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += up;
        }
        if (e < a.experts) sh->tiles[e] = sum + s - n;
        sum += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) {
        sh->tiles[a.experts] = sum;
        sh->units = sum * ch_tiles;
    }
}

// Stages between drains, from the tokens' own size.  int8_to_f16_kernel leaves in
// peaks the largest sum of |a| over any 512 consecutive k that one of its warps
// saw; a run of c * 512 k touches at most c + 1 of those windows and |b| <= 128,
// so no partial sum over it exceeds 128 * (c + 1) * peak, and up to 2^24 FP32
// holds it exactly.  Real activations stay well below 127 on average (a normal
// distribution quantized to its largest value: 4096 k and more), which leaves
// an eighth to a quarter of the drains; data at the extremes gets 1024 k.  An
// even number, for the pair kernel's two stages at a time.  One warp.
__device__ __forceinline__ int chunk_of(const Int8Args &a, int lane) {
    int top = 1;
    for (int i = lane; i < a.n_peaks; i += 32) top = max(top, __ldcg(a.peaks + i));
    top = __reduce_max_sync(0xffffffffu, top);
    return max(((1 << 17) / top - 1) * (512 / kI8StageK) & ~1, kChunk);
}

template <int NT, bool SPLIT, bool DIRECT>
__global__ void __launch_bounds__(I8Cfg<NT, SPLIT, DIRECT>::kThreads, 1)
int8_tc_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA, const Int8Args a) {
    using Cf = I8Cfg<NT, SPLIT, DIRECT>;
    constexpr int SB = Cf::kBStages, SX = Cf::kXStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    uint8_t *ring_b = smem_raw + pad, *ring_x = ring_b + SB * Cf::kStage;
    int *xchg = reinterpret_cast<int *>(ring_b + Cf::kRing);
    I8Shared *sh = reinterpret_cast<I8Shared *>(ring_b + Cf::kRing + Cf::kXchg);
    // warp number and tensor-memory address through a shuffle: uniform to the compiler too
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int splits = SPLIT ? a.ksplit : 1;
    const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    const int first_unit = SPLIT ? static_cast<int>(blockIdx.x) / splits : static_cast<int>(blockIdx.x);
    const int unit_step = SPLIT ? static_cast<int>(gridDim.x) / splits : static_cast<int>(gridDim.x);
    const int ch_tiles = (a.N + kI8TileN - 1) / kI8TileN;
    const int kt = (a.K + kI8StageK - 1) / kI8StageK;
    // this CTA's stages of every unit
    const int kb = SPLIT ? rank * kt / splits : 0, ke = SPLIT ? (rank + 1) * kt / splits : kt;

    if (tid == 0) {
        for (int s = 0; s < SB; ++s) {
            mbar_init(&sh->bfull[s], 1);
            mbar_init(&sh->bempty[s], DIRECT ? 8 : 4);
        }
        for (int s = 0; s < SX; ++s) {
            mbar_init(&sh->xfull[s], DIRECT ? 4 : 1);
            mbar_init(&sh->xempty[s], 1);
        }
        for (int s = 0; s < kAStages; ++s) {
            mbar_init(&sh->afull[s], 4);
            mbar_init(&sh->aempty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh->dfull[s], 1);
            mbar_init(&sh->dempty[s], 4 * Cf::kEpiWGs);
        }
        mbar_init(&sh->drained, 1);
        sh->abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmA);
    }
    if (warp == 1) {
        tc::tmem_alloc(&sh->tmem_base, kI8TmemCols);
        tc::tmem_relinquish();
    }
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 2) sum_tiles(sh, a, NT, ch_tiles, lane);
    if (!DIRECT && warp == 3) {
        const int c = chunk_of(a, lane);
        if (lane == 0) sh->chunk = c;
    }
    tc::fence_before_sync();
    __syncthreads();
    if (SPLIT) cluster_sync();  // every CTA runs before another writes into it
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
    const uint32_t tmem_a = tmem + 2 * NT;
    volatile int *abort_flag = &sh->abort;
    const int units = sh->units, chunk_stages = DIRECT ? kChunk : sh->chunk;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity, a.status)) return true;
        *abort_flag = 1;
        return false;
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int it = 0;
        bool ok = true;
        for (int u = first_unit; u < units; u += unit_step) {
            if (lane == 0 && ok) {
                const I8Unit q = unit_of<NT, kI8TileN>(sh, a, ch_tiles, u);
                for (int i = kb; i < ke; ++i, ++it) {
                    const int s = it % SB;
                    if (it >= SB && !wait(&sh->bempty[s], (it / SB - 1) & 1)) { ok = false; break; }
                    uint8_t *st = ring_b + s * Cf::kStage;
                    mbar_arrive_expect_tx(&sh->bfull[s], Cf::kStage);
                    tma_load_3d(st, &tmB, &sh->bfull[s], i * kI8StageK, q.ch0, q.e);
                    if (DIRECT) tma_load_2d(st + kBBytes, &tmA, &sh->bfull[s], i * kI8StageK, q.t0 - a.row0);
                }
            }
            __syncwarp();
            if (SPLIT) {
                cluster_sync();
                if (u + unit_step < units) cluster_sync();
            }
        }
        if (lane == 0)  // no copy outlives the CTA
            for (int t = max(0, it - SB); t < it; ++t) mbar_wait(&sh->bfull[t % SB], (t / SB) & 1, a.status);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        // The whole warp walks the stages and waits; one elected lane issues.
        constexpr uint32_t idesc = tc::idesc_f16_kmajor(kI8TileN, NT);
        const uint64_t xdesc = tc::smem_desc(smem_u32(ring_x), 16, 1024, tc::kLayoutSwizzle128);
        int it = 0, chunk = 0;
        bool ok = true;
        for (int u = first_unit; u < units; u += unit_step) {
            int run = 0;  // stages in the accumulator so far
            for (int i = kb; i < ke && ok; ++i, ++it) {
                const int x = it % SX, t = it % kAStages, d = chunk & 1;
                const bool start = run == 0, end = i + 1 == ke || run + 1 == chunk_stages;
                ok = (!start || chunk < 2 || wait(&sh->dempty[d], (chunk / 2 - 1) & 1)) &&
                     wait(&sh->xfull[x], (it / SX) & 1) && wait(&sh->afull[t], (it / kAStages) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint64_t b = xdesc + static_cast<uint64_t>(x * (Cf::kXBytes / 16));
#pragma unroll
                    for (int kk = 0; kk < kI8StageK / 16; ++kk)
                        tc::mma_f16_ta(tmem + d * NT, tmem_a + t * kACols + kk * 8,
                                       b + ((kk / 4) * NT * 128 + (kk % 4) * 32) / 16, idesc,
                                       (start && kk == 0) ? 0u : 1u);
                    tc::commit(&sh->xempty[x]);
                    tc::commit(&sh->aempty[t]);
                    if (end) tc::commit(&sh->dfull[d]);
                }
                __syncwarp();
                run = end ? 0 : run + 1;
                if (end) ++chunk;
            }
            if (SPLIT) {
                __syncwarp();
                cluster_sync();
                if (u + unit_step < units) cluster_sync();
            }
        }
        if (!ok && tc::elect_one()) {  // no teardown under a running MMA
            tc::commit(&sh->drained);
            mbar_wait(&sh->drained, 0, a.status);
        }
        __syncwarp();
    } else if (!DIRECT && warp == 2) {
        // ------------------------------------------------ TMA producer of the tokens
        int it = 0;
        bool ok = true;
        for (int u = first_unit; u < units; u += unit_step) {
            if (lane == 0 && ok) {
                const I8Unit q = unit_of<NT, kI8TileN>(sh, a, ch_tiles, u);
                for (int i = kb; i < ke; ++i, ++it) {
                    const int x = it % SX;
                    if (it >= SX && !wait(&sh->xempty[x], (it / SX - 1) & 1)) { ok = false; break; }
                    uint8_t *st = ring_x + x * Cf::kXBytes;
                    mbar_arrive_expect_tx(&sh->xfull[x], Cf::kXBytes);
                    tma_load_2d(st, &tmA, &sh->xfull[x], i * kI8StageK, q.t0 - a.row0);
                    tma_load_2d(st + NT * 128, &tmA, &sh->xfull[x], i * kI8StageK + 64, q.t0 - a.row0);
                }
            }
            __syncwarp();
            if (SPLIT) {
                cluster_sync();
                if (u + unit_step < units) cluster_sync();
            }
        }
        if (lane == 0)
            for (int t = max(0, it - SX); t < it; ++t) mbar_wait(&sh->xfull[t % SX], (t / SX) & 1, a.status);
        __syncwarp();
    } else if (DIRECT && warp >= Cf::kWarpX && warp < Cf::kWarpConv) {
        // ------------------------------------------------ the tokens' rows to FP16
        const int me = tid - 32 * Cf::kWarpX;
        const int kc = me % 8;  // 16 k of a row; rows me / 8, me / 8 + 16, ..
        int it = 0;
        bool ok = true;
        for (int u = first_unit; u < units; u += unit_step) {
            for (int i = kb; i < ke && ok; ++i, ++it) {
                const int s = it % SB, x = it % SX;
                ok = wait(&sh->bfull[s], (it / SB) & 1) && (it < SX || wait(&sh->xempty[x], (it / SX - 1) & 1));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint8_t *src = ring_b + s * Cf::kStage + kBBytes;
                uint8_t *st = ring_x + x * Cf::kXBytes + (kc / 4) * NT * 128;
                uint4 v[Cf::kPieces];
#pragma unroll
                for (int j = 0; j < Cf::kPieces; ++j) {
                    const int row = me / 8 + 16 * j;
                    v[j] = *reinterpret_cast<const uint4 *>(src + row * 128 + ((kc ^ (row & 7)) * 16));
                }
#pragma unroll
                for (int j = 0; j < Cf::kPieces; ++j) {
                    const int row = me / 8 + 16 * j, c = (kc % 4) * 2;
                    uint4 o0, o1;
                    int8x4_to_f16(v[j].x, o0.x, o0.y);
                    int8x4_to_f16(v[j].y, o0.z, o0.w);
                    int8x4_to_f16(v[j].z, o1.x, o1.y);
                    int8x4_to_f16(v[j].w, o1.z, o1.w);
                    *reinterpret_cast<uint4 *>(st + row * 128 + ((c ^ (row & 7)) * 16)) = o0;
                    *reinterpret_cast<uint4 *>(st + row * 128 + (((c + 1) ^ (row & 7)) * 16)) = o1;
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh->bempty[s]);
                    mbar_arrive(&sh->xfull[x]);
                }
            }
            if (SPLIT) {
                __syncwarp();
                cluster_sync();
                if (u + unit_step < units) cluster_sync();
            }
        }
    } else if (warp >= Cf::kWarpConv && warp < Cf::kWarpEpi) {
        // ------------------------------------------------ B to FP16, into tensor memory
        const int wg = (warp - Cf::kWarpConv) / 4;
        const int row = (warp % 4) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        int it = 0, stored = -1;  // stored: the stage in tensor memory whose stores have not been waited for
        bool ok = true;
        auto flush = [&]() {
            if (stored < 0) return;
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->afull[stored]);
            stored = -1;
        };
        for (int u = first_unit; u < units; u += unit_step) {
            for (int i = kb; i < ke && ok; ++i, ++it) {
                if (it % kConvWGs != wg) continue;
                const int s = it % SB, t = it % kAStages;
                // the stage before is handed on while this one is read, unless
                // this one has yet to land
                if (!__all_sync(0xffffffffu, mbar_try_wait(&sh->bfull[s], (it / SB) & 1))) {
                    flush();
                    ok = __all_sync(0xffffffffu, wait(&sh->bfull[s], (it / SB) & 1));
                    if (!ok) break;
                }
                const uint8_t *src = ring_b + s * Cf::kStage + row * kI8StageK;
                uint4 w[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) w[c] = *reinterpret_cast<const uint4 *>(src + ((c ^ (row & 7)) * 16));
                flush();
                ok = it < kAStages || wait(&sh->aempty[t], (it / kAStages - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        int8x4_to_f16(w[h * 4 + c].x, o[c * 8 + 0], o[c * 8 + 1]);
                        int8x4_to_f16(w[h * 4 + c].y, o[c * 8 + 2], o[c * 8 + 3]);
                        int8x4_to_f16(w[h * 4 + c].z, o[c * 8 + 4], o[c * 8 + 5]);
                        int8x4_to_f16(w[h * 4 + c].w, o[c * 8 + 6], o[c * 8 + 7]);
                    }
                    tc::tmem_st32(tmem_a + t * kACols + h * 32 + lanes, o);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->bempty[s]);
                stored = t;
            }
            flush();
            if (SPLIT) {
                __syncwarp();
                cluster_sync();
                if (u + unit_step < units) cluster_sync();
            }
        }
    } else if (warp >= Cf::kWarpEpi) {
        // ------------------------------------------------ accumulators to C
        const int wg = (warp - Cf::kWarpEpi) / 4;
        const int ch = (warp % 4) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        int chunk = 0;
        bool ok = true;
        for (int u = first_unit; u < units; u += unit_step) {
            const I8Unit q = unit_of<NT, kI8TileN>(sh, a, ch_tiles, u);
            // What the epilogue needs of global memory, asked for before the sums
            // are ready: the channel's scale and bias, and lane l's share of the
            // token scales (handed round by shuffles).
            const int n = q.ch0 + ch;
            const long long at = static_cast<long long>(q.e) * a.N + n;
            const float sb = n < a.N ? __ldg(a.scaleB + at) : 0.f;
            const float bias = n < a.N && a.bias ? __ldg(a.bias + at) : 0.f;
            const int per = SPLIT ? NT / splits : Cf::kCols;  // this CTA's (warpgroup's) columns of the result
            const int shift = 31 - __clz(per);
            const int first = q.t0 + (SPLIT ? rank * per : wg * Cf::kCols);
            float sa[(Cf::kCols + 31) / 32];
#pragma unroll
            for (int c = 0; c < (Cf::kCols + 31) / 32; ++c)
                sa[c] = c * 32 + lane < per && first + c * 32 + lane < q.tend ? __ldg(a.scaleA + first + c * 32 + lane) : 0.f;
            int acc[Cf::kCols];
#pragma unroll
            for (int j = 0; j < Cf::kCols; ++j) acc[j] = 0;
            for (int i = kb; i < ke && ok; i += chunk_stages, ++chunk) {
                const int d = chunk & 1;
                ok = __all_sync(0xffffffffu, wait(&sh->dfull[d], (chunk / 2) & 1));
                if (!ok) break;
                tc::fence_after_sync();
                drain(tmem + d * NT + wg * Cf::kCols + lanes, acc);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->dempty[d]);
            }
            if (!SPLIT) {
                if (ok)
                    with_out_type(a.out_type, [&](auto out) {
                        using Out = decltype(out);
                        write_columns<Out>(static_cast<typename Out::T *>(a.C) + static_cast<long long>(first) * a.ldc + n,
                                           a.ldc, n < a.N ? q.tend - first : 0, acc, sa, sb, bias);
                    });
            } else {
                // column j belongs to CTA j / per of the cluster
                if (ok) {
                    // (splits and per are powers of two)
                    const uint32_t mine = smem_u32(xchg + rank * per * kI8TileN + ch);
                    uint32_t to = 0;
#pragma unroll
                    for (int j = 0; j < Cf::kCols; ++j) {
                        if ((j & (per - 1)) == 0)
                            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(mine), "r"(j >> shift));
                        asm volatile("st.shared::cluster.u32 [%0], %1;"
                                     ::"r"(to + (j & (per - 1)) * kI8TileN * 4), "r"(acc[j]) : "memory");
                    }
                }
                __syncwarp();
                cluster_sync();
                if (ok)
                    with_out_type(a.out_type, [&](auto out) {
                        using Out = decltype(out);
                        auto *C = static_cast<typename Out::T *>(a.C) + static_cast<long long>(first) * a.ldc + n;
                        for (int c0 = 0; c0 < per; c0 += 8) {
                            int sum[8] = {};
                            for (int r = 0; r < splits; ++r)
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    if (c0 + c < per) sum[c] += xchg[(r * per + c0 + c) * kI8TileN + ch];
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const float s = __shfl_sync(0xffffffffu, sa[0], (c0 + c) & 31);
                                if (c0 + c < per && first + c0 + c < q.tend && n < a.N)
                                    C[static_cast<long long>(c0 + c) * a.ldc] =
                                        Out::lo(Out::two(int8_value(sum[c], sb, s, bias), 0.f));
                            }
                        }
                    });
                __syncwarp();
                if (u + unit_step < units) cluster_sync();
            }
        }
    } else {
        for (int u = first_unit; SPLIT && u < units; u += unit_step) {
            cluster_sync();
            if (u + unit_step < units) cluster_sync();
        }
    }
    // ---------------------------------------------------- teardown
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kI8TmemCols);
    }
}

// ---- CTA pairs: 256 channels x 256 tokens -------------------------------------------
constexpr int kPairN = 256, kPairT = 256;        // channels and tokens of a pair's tile
constexpr int kPairXBytes = 128 * kI8StageK * 2;  // this CTA's half of the tokens, FP16: 32 KiB a stage
constexpr int kPairBStages = 5, kPairXStages = 4;
constexpr int kPairThreads = 512;

struct PairShared {
    uint64_t bfull[kPairBStages], bempty[kPairBStages];
    uint64_t xfull[kPairXStages];   // (even CTA) both CTAs' tokens of the stage have landed
    uint64_t xempty[kPairXStages];  // the MMAs have read them (both CTAs are told)
    uint64_t afull[kAStages];       // (even CTA) B stands in both CTAs' tensor memory
    uint64_t aempty[kAStages];
    uint64_t dfull[2];              // a half accumulator holds up to 1024 k
    uint64_t dempty[2];             // (even CTA) both CTAs have read it
    uint64_t drained;
    uint32_t tmem_base;
    int abort;
    int units, chunk;
    int bound[kMaxExperts + 1];
    int tiles[kMaxExperts + 1];
};
constexpr int kPairSmem = 1024 + kPairBStages * kBBytes + kPairXStages * kPairXBytes + static_cast<int>(sizeof(PairShared));
static_assert(kPairSmem <= kSmemLimit, "shared memory");

// Registers a thread of each warpgroup: control, conversion, two epilogue
// warpgroups (128 sums a thread).  Their sum stays below 4 x 128, what the
// block is launched with.
constexpr int kRegsControl = 56, kRegsConvert = 96, kRegsEpilogue = 176;
static_assert(kRegsControl + kRegsConvert + 2 * kRegsEpilogue <= 4 * 128, "register split");
template <int R>
__device__ __forceinline__ void regs_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

__global__ void __launch_bounds__(kPairThreads, 1)
int8_tc_pair_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA, const Int8Args a) {
    constexpr int SB = kPairBStages, SX = kPairXStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;  // the same in both CTAs
    uint8_t *ring_x = smem_raw + pad, *ring_b = ring_x + SX * kPairXBytes;
    PairShared *sh = reinterpret_cast<PairShared *>(ring_b + SB * kBBytes);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());  // 0: issues the MMAs
    const int first_unit = static_cast<int>(blockIdx.x) >> 1, unit_step = static_cast<int>(gridDim.x) >> 1;
    const int ch_tiles = (a.N + kPairN - 1) / kPairN;
    const int kt = (a.K + kI8StageK - 1) / kI8StageK;

    if (tid == 0) {
        for (int s = 0; s < SB; ++s) {
            mbar_init(&sh->bfull[s], 1);
            mbar_init(&sh->bempty[s], 4);
        }
        for (int s = 0; s < SX; ++s) {
            mbar_init(&sh->xfull[s], 1);
            mbar_init(&sh->xempty[s], 1);
        }
        for (int s = 0; s < kAStages; ++s) {
            mbar_init(&sh->afull[s], 8);
            mbar_init(&sh->aempty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh->dfull[s], 1);
            mbar_init(&sh->dempty[s], 8);
        }
        mbar_init(&sh->drained, 1);
        sh->abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmA);
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(&sh->tmem_base, kI8TmemCols);
        tc::tmem_relinquish_pair();
    }
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 2) sum_tiles(sh, a, kPairT, ch_tiles, lane);
    if (warp == 3) {
        const int c = chunk_of(a, lane);
        if (lane == 0) sh->chunk = c;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync_all();  // both CTAs' barriers are initialised before any cross-CTA arrive
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
    const uint32_t tmem_a = tmem + kPairT;
    volatile int *abort_flag = &sh->abort;
    const int units = sh->units, chunk_stages = sh->chunk;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity, a.status)) return true;
        *abort_flag = 1;
        return false;
    };

    if (warp < 4) {
        regs_fewer<kRegsControl>();
        if (warp == 0) {
            // -------------------------------------------- TMA producer of B
            int it = 0;
            bool ok = true;
            if (lane == 0) {
                for (int u = first_unit; u < units && ok; u += unit_step) {
                    const I8Unit q = unit_of<kPairT, kPairN>(sh, a, ch_tiles, u);
                    for (int i = 0; i < kt; ++i, ++it) {
                        const int s = it % SB;
                        if (it >= SB && !wait(&sh->bempty[s], (it / SB - 1) & 1)) { ok = false; break; }
                        mbar_arrive_expect_tx(&sh->bfull[s], kBBytes);
                        tma_load_3d(ring_b + s * kBBytes, &tmB, &sh->bfull[s], i * kI8StageK, q.ch0 + rank * kI8TileN, q.e);
                    }
                }
                for (int t = max(0, it - SB); t < it; ++t) mbar_wait(&sh->bfull[t % SB], (t / SB) & 1, a.status);
            }
            __syncwarp();
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------- MMA issuer (even CTA)
            constexpr uint32_t idesc = tc::idesc_f16_kmajor(2 * kI8TileN, kPairT / 2);
            const uint64_t xdesc = tc::smem_desc(smem_u32(ring_x), 16, 1024, tc::kLayoutSwizzle128);
            int it = 0, chunk = 0;
            bool ok = true;
            for (int u = first_unit; u < units && ok; u += unit_step) {
                // Two stages at a time: both for half 0 of the accumulators, then
                // both for half 1, so that at the end of 1024 k either half has the
                // time of 16 MMAs (1024 cycles) to be drained in while the other
                // is added to.
                int run = 0;  // stages in the accumulators so far
                for (int i = 0; i < kt; i += 2) {
                    const int two = i + 1 < kt ? 2 : 1;
                    const bool start = run == 0, end = i + two == kt || run + two == chunk_stages;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ok = ok && (!start || chunk == 0 || wait(&sh->dempty[h], (chunk - 1) & 1));
                        for (int j = 0; j < two; ++j) {
                            const int x = (it + j) % SX, t = (it + j) % kAStages;
                            if (h == 0)
                                ok = ok && wait(&sh->xfull[x], ((it + j) / SX) & 1) &&
                                     wait(&sh->afull[t], ((it + j) / kAStages) & 1);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            tc::fence_after_sync();
                            if (tc::elect_one()) {
                                const uint64_t b =
                                    xdesc + static_cast<uint64_t>(x * (kPairXBytes / 16) + h * (64 * 128 / 16));
#pragma unroll
                                for (int kk = 0; kk < kI8StageK / 16; ++kk)
                                    tc::mma_f16_ta_pair(tmem + h * (kPairT / 2), tmem_a + t * kACols + kk * 8,
                                                        b + ((kk / 4) * 16384 + (kk % 4) * 32) / 16, idesc,
                                                        (start && j == 0 && kk == 0) ? 0u : 1u);
                                if (h == 1) {
                                    tc::commit_pair(&sh->xempty[x], 0x3);
                                    tc::commit_pair(&sh->aempty[t], 0x3);
                                }
                                if (end && j + 1 == two) tc::commit_pair(&sh->dfull[h], 0x3);
                            }
                            __syncwarp();
                        }
                    }
                    if (!ok) break;
                    it += two;
                    run = end ? 0 : run + two;
                    if (end) ++chunk;
                }
            }
            if (!ok && tc::elect_one()) {  // no teardown under a running MMA
                tc::commit_pair(&sh->drained, 0x1);
                mbar_wait(&sh->drained, 0, a.status);
            }
            __syncwarp();
        } else if (warp == 2) {
            // -------------------------------------------- TMA producer of the tokens
            // Half h of the accumulators covers tokens t0 + 128 h ..+127, 64 from
            // each CTA: this CTA's rows 64 h .. 64 h + 63 of a stage.  Both CTAs'
            // bytes count on the even CTA's barrier.
            int it = 0;
            bool ok = true;
            if (lane == 0) {
                const uint32_t xfull = tc::map_shared_rank(smem_u32(&sh->xfull[0]), 0);
                for (int u = first_unit; u < units && ok; u += unit_step) {
                    const I8Unit q = unit_of<kPairT, kPairN>(sh, a, ch_tiles, u);
                    const int row = q.t0 - a.row0 + rank * 64;
                    for (int i = 0; i < kt; ++i, ++it) {
                        const int x = it % SX;
                        if (it >= SX && !wait(&sh->xempty[x], (it / SX - 1) & 1)) { ok = false; break; }
                        uint8_t *st = ring_x + x * kPairXBytes;
                        if (rank == 0) mbar_arrive_expect_tx(&sh->xfull[x], 2 * kPairXBytes);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                tc::tma_load_2d_pair(st + k * 16384 + h * 8192, &tmA, xfull + x * 8,
                                                     i * kI8StageK + k * 64, row + h * 128);
                    }
                }
                // no copy outlives its CTA: the MMAs that read the last ones have finished
                for (int t = max(0, it - SX); t < it; ++t) mbar_wait(&sh->xempty[t % SX], (t / SX) & 1, a.status);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        // ------------------------------------------------ B to FP16, into tensor memory
        regs_fewer<kRegsConvert>();
        const int row = (warp % 4) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        const uint32_t afull = tc::map_shared_rank(smem_u32(&sh->afull[0]), 0);
        int it = 0, stored = -1;
        bool ok = true;
        auto flush = [&]() {
            if (stored < 0) return;
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_remote(afull + stored * 8);
            stored = -1;
        };
        for (int u = first_unit; u < units && ok; u += unit_step) {
            for (int i = 0; i < kt; ++i, ++it) {
                const int s = it % SB, t = it % kAStages;
                if (!__all_sync(0xffffffffu, mbar_try_wait(&sh->bfull[s], (it / SB) & 1))) {
                    flush();
                    ok = __all_sync(0xffffffffu, wait(&sh->bfull[s], (it / SB) & 1));
                    if (!ok) break;
                }
                const uint8_t *src = ring_b + s * kBBytes + row * kI8StageK;
                uint4 w[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) w[c] = *reinterpret_cast<const uint4 *>(src + ((c ^ (row & 7)) * 16));
                flush();
                ok = it < kAStages || wait(&sh->aempty[t], (it / kAStages - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        int8x4_to_f16(w[h * 4 + c].x, o[c * 8 + 0], o[c * 8 + 1]);
                        int8x4_to_f16(w[h * 4 + c].y, o[c * 8 + 2], o[c * 8 + 3]);
                        int8x4_to_f16(w[h * 4 + c].z, o[c * 8 + 4], o[c * 8 + 5]);
                        int8x4_to_f16(w[h * 4 + c].w, o[c * 8 + 6], o[c * 8 + 7]);
                    }
                    tc::tmem_st32(tmem_a + t * kACols + h * 32 + lanes, o);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->bempty[s]);
                stored = t;
            }
            flush();
        }
    } else {
        // ------------------------------------------------ accumulators to C: warpgroup h reads half h
        regs_more<kRegsEpilogue>();
        constexpr int kCols = kPairT / 2;
        const int h = (warp - 8) / 4;
        const int ch = (warp % 4) * 32 + lane;
        const uint32_t src = tmem + h * kCols + (static_cast<uint32_t>(warp % 4 * 32) << 16);
        const uint32_t dempty = tc::map_shared_rank(smem_u32(&sh->dempty[h]), 0);
        int chunk = 0;
        bool ok = true;
        for (int u = first_unit; u < units && ok; u += unit_step) {
            const I8Unit q = unit_of<kPairT, kPairN>(sh, a, ch_tiles, u);
            const int n = q.ch0 + rank * kI8TileN + ch;
            const long long at = static_cast<long long>(q.e) * a.N + n;
            const float sb = n < a.N ? __ldg(a.scaleB + at) : 0.f;
            const float bias = n < a.N && a.bias ? __ldg(a.bias + at) : 0.f;
            const int first = q.t0 + h * kCols;
            float sa[kCols / 32];
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c)
                sa[c] = first + c * 32 + lane < q.tend ? __ldg(a.scaleA + first + c * 32 + lane) : 0.f;
            int acc[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0;
            for (int i = 0; i < kt; i += chunk_stages, ++chunk) {
                ok = __all_sync(0xffffffffu, wait(&sh->dfull[h], chunk & 1));
                if (!ok) break;
                tc::fence_after_sync();
                drain(src, acc);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_remote(dempty);
            }
            if (ok)
                with_out_type(a.out_type, [&](auto out) {
                    using Out = decltype(out);
                    write_columns<Out>(static_cast<typename Out::T *>(a.C) + static_cast<long long>(first) * a.ldc + n,
                                       a.ldc, n < a.N ? q.tend - first : 0, acc, sa, sb, bias);
                });
        }
    }
    // ---------------------------------------------------- teardown
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync_all();  // the peer is done with this CTA's barriers and tensor memory
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(tmem, kI8TmemCols);
    }
}

template <int NT, bool SPLIT, bool DIRECT>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(int8_tc_kernel<NT, SPLIT, DIRECT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                I8Cfg<NT, SPLIT, DIRECT>::kSmem);
}

template <int NT, bool SPLIT, bool DIRECT>
cudaError_t launch_one(const Int8Args &a, const CUtensorMap &tmB, const CUtensorMap &tmA, int num_sms,
                       int smem_override, cudaStream_t stream) {
    using Cf = I8Cfg<NT, SPLIT, DIRECT>;
    const int ch_tiles = (a.N + kI8TileN - 1) / kI8TileN, splits = SPLIT ? a.ksplit : 1;
    // at most this many units (the experts' row counts are on the device)
    const long long tiles = a.experts == 1 ? (a.rows + NT - 1) / NT
                                           : static_cast<long long>(a.rows) / NT + (a.experts < a.rows ? a.experts : a.rows);
    const long long units = tiles * ch_tiles, most = num_sms / splits;
    return launch_dependent(int8_tc_kernel<NT, SPLIT, DIRECT>,
                            dim3(static_cast<unsigned>(splits * (units < most ? units : most))), dim3(Cf::kThreads),
                            smem_override > 0 ? smem_override : Cf::kSmem, stream, splits, tmB, tmA, a);
}

cudaError_t launch_pair(const Int8Args &a, const CUtensorMap &tmB, const CUtensorMap &tmA, int num_sms,
                        int smem_override, cudaStream_t stream) {
    const int ch_tiles = (a.N + kPairN - 1) / kPairN;
    const long long tiles = a.experts == 1
                                ? (a.rows + kPairT - 1) / kPairT
                                : static_cast<long long>(a.rows) / kPairT + (a.experts < a.rows ? a.experts : a.rows);
    const long long units = tiles * ch_tiles, most = num_sms / 2;
    return launch_dependent(int8_tc_pair_kernel, dim3(static_cast<unsigned>(2 * (units < most ? units : most))),
                            dim3(kPairThreads), smem_override > 0 ? smem_override : kPairSmem, stream, 2, tmB, tmA, a);
}

template <int NT>
cudaError_t launch_direct(const Int8Args &a, const CUtensorMap &tmB, const CUtensorMap &tmA, int num_sms,
                          int smem_override, cudaStream_t stream) {
    return a.ksplit > 1 ? launch_one<NT, true, true>(a, tmB, tmA, num_sms, smem_override, stream)
                        : launch_one<NT, false, true>(a, tmB, tmA, num_sms, smem_override, stream);
}

}  // namespace

cudaError_t int8_prepare() {
    cudaError_t e = cudaSuccess;
    for (cudaError_t r : {prepare_one<16, false, true>(), prepare_one<32, false, true>(),
                          prepare_one<64, false, true>(), prepare_one<16, true, true>(),
                          prepare_one<32, true, true>(), prepare_one<64, true, true>(),
                          prepare_one<128, false, false>(),
                          cudaFuncSetAttribute(int8_tc_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kPairSmem)})
        if (e == cudaSuccess) e = r;
    return e;
}

cudaError_t launch_int8_tc(const Int8Args &a, const CUtensorMap &tmB, const CUtensorMap &tmA, int num_sms,
                           int smem_override, cudaStream_t stream) {
    switch (a.nt) {
        case 16: return launch_direct<16>(a, tmB, tmA, num_sms, smem_override, stream);
        case 32: return launch_direct<32>(a, tmB, tmA, num_sms, smem_override, stream);
        case 64: return launch_direct<64>(a, tmB, tmA, num_sms, smem_override, stream);
        case 256: return launch_pair(a, tmB, tmA, num_sms, smem_override, stream);
        default: return launch_one<128, false, false>(a, tmB, tmA, num_sms, smem_override, stream);
    }
}

cudaError_t launch_int8_generic(const Int8Args &a, cudaStream_t stream) {
    const int y = (a.rows + kGTile - 1) / kGTile;
    const dim3 grid((a.N + kGTile - 1) / kGTile, y < 65535 ? y : 65535, a.experts);
    return launch_dependent(int8_generic_kernel, grid, dim3(256), 0, stream, 1, a);
}

cudaError_t launch_int8_to_f16(const int8_t *A, long long lda, int rows, int K, void *dst, int ldd, int *peaks,
                               int *n_peaks, cudaStream_t stream) {
    const int vec = reinterpret_cast<uintptr_t>(A) % 16 == 0 && lda % 16 == 0;
    const long long blocks = (static_cast<long long>(rows) * (ldd / 16) + 255) / 256;
    *n_peaks = static_cast<int>(blocks < kI8Peaks ? blocks : kI8Peaks);
    return launch_dependent(int8_to_f16_kernel, dim3(*n_peaks), dim3(256), 0, stream, 1, A, lda, rows, K,
                            static_cast<uint4 *>(dst), ldd, vec, peaks);
}

cudaError_t launch_int8_relayout(const int8_t *B, long long ldb, long long strideB, int trans, int experts, int N,
                                 int K, int8_t *dst, int ldd, cudaStream_t stream) {
    if (trans) {
        const long long blocks = (static_cast<long long>(N) * (ldd / 16) + 255) / 256;
        return launch_dependent(int8_realign_kernel,
                                dim3(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)), experts),
                                dim3(256), 0, stream, 1, B, ldb, strideB, N, K, dst, ldd);
    }
    const int y = (N + kTN - 1) / kTN;
    return launch_dependent(int8_transpose_kernel, dim3((ldd + kTK - 1) / kTK, y < 65535 ? y : 65535, experts),
                            dim3(256), 0, stream, 1, B, ldb, strideB, N, K, dst, ldd);
}

}  // namespace sg
