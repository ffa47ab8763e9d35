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
// integer that FP32 holds exactly: the kernels multiply with .kind::f16, FP32
// accumulators in tensor memory, and move them into int32 registers at least
// that often.  Sums of integers do not depend on their order, so every tile and
// every split of K gives the same bits.
//
// Both tensor-core kernels compute D[channel][token] = B * A^T, the channels as
// the MMA's M and a tile of tokens as its N, so that few tokens cost a narrow tile
// and not a padded one.  B crosses HBM, L2 and shared memory as int8 (half the
// bytes of 16-bit operands; a decode step is bound by them) and becomes FP16
// only on its way into tensor memory, where the MMA reads it as its A operand:
// a converting thread reads its channel's 128 bytes of a stage (16 at a time,
// conflict-free through the TMA's swizzle), makes of byte b the FP16 bits
// 0x6400 + (b ^ 0x80) = 1152 + b, subtracts 1152 (exact: 5 instructions for 4
// bytes) and stores 64 columns of its lane.  A stage's stores are waited for
// while the next one is read.  Both are persistent over (expert, token tile,
// channel tile) units, token tiles innermost within groups so that concurrent
// CTAs share B's tiles in L2; the MMAs are issued by an elected lane of a warp
// whose addresses are uniform (from one lane of a divergent warp, with its
// descriptors moved to uniform registers one by one, an MMA takes about 150
// cycles to issue: 8192^3 1138 us instead of 783).
//
//  * int8_tc_kernel -- up to 64 tokens a tile, 128 channels, two CTAs an SM, the
//    tokens' int8 rows expanded here too:
//      warp 0     TMA producer: stages of 128 k, B 128 x 128 bytes and the tokens
//      warp 1     MMA issuer; owns the tensor memory (two accumulators of NT
//                 columns, drained in turn, and two stages of B)
//      warps 2-3  the stage's tokens to FP16 in the MMA's layout
//      warps 4-7  B to FP16 in tensor memory
//      warps 8-11 accumulators to C: a warp's lanes are 32 consecutive channels of
//                 a token; its scales are asked for before the sums are ready
//    With few tiles the 2, 4 or 8 CTAs of a cluster share a tile's K range and
//    send one another their columns' int32 partial sums through distributed
//    shared memory.  Bound by HBM once B is large (32 experts x 4096 x 4096 and
//    128 rows: 86 us, 6.3 TB/s), by the chain of latencies before (16 x 4096 x 4096:
//    6.4 us from one call's end to the next's, 3.9 of them from the first load to
//    the last sum; 64 x 8192 x 8192: 20 us, 12.5 of them at 5.3 TB/s).
//    Prefetching further stages into L2 made both slower.
//  * int8_tc_pair_kernel -- 256 channels x 128 or 256 tokens on a CTA pair
//    (cta_group::2), the tokens as FP16 from int8_copies_kernel: at this size
//    expanding them in the kernel would take all of the shared memory's
//    bandwidth.  Accumulators of 256 columns leave no room for a second set, so
//    they are worked on as halves of the tokens, two stages of one and two of the
//    other in turn, and each half is drained while the other is added to; data
//    whose tokens are not at the extremes needs a drain every 4096 k or so only
//    (chunk_of).  Warpgroups: control (B and token producers, MMA issuer),
//    conversion, and two that take 128 columns a thread (setmaxnreg).
//    Signals that only guard tensor memory go to the other CTA without a release
//    at cluster scope, which costs its thread 1500 cycles (8192^3 1184 us instead
//    of 693).  8192^3: 581 us in short runs, 1890 TFLOP/s, as much as the
//    measured rate of cuBLAS in BF16, and 635 us (1730) when repeated until the
//    power limit shows; 31 us of it are the tokens' conversion.  Of a stage of
//    1130 cycles the MMAs take 1024; without the conversion and all loads it
//    would be 1070.
//  * int8_few_kernel -- up to 8 tokens on the CUDA cores, B on any alignment (below).
//  * int8_generic_kernel -- any layout and alignment, dp4a on the CUDA cores.
//  * int8_copies_kernel -- the tokens' rows as FP16 or on 16-byte boundaries, and B
//    as the TMA can read it (stored K x N, or not on 16-byte boundaries).
// Every wait is bounded; on a timeout the kernel records it, waits (bounded)
// for its own copies and MMAs in flight, frees the tensor memory and returns.
// No load is a read-only-cache load (ld.global.nc): what is read may have been
// written by the kernel before, whose end the launch overlaps.  Other loads are in
// order after the wait for that kernel.  16-byte pieces of rows and what a thread alone
// reads go past L1 (ld.global.cg); words and bytes whose sectors neighbouring threads
// read too do not (B 8191 x 8191 stored K x N, 16 tokens 61 us instead of 69; one token x
// 8190 x 8190 on the CUDA cores 17.0 instead of 20.1).
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "internal.h"
#include "sgemm.h"
#include "tcgen05.cuh"

namespace sg {
namespace {

// ---- epilogue arithmetic, common to both kernels --------------------------------
__device__ __forceinline__ float int8_value(float sum, float sb, float sa, float bias) {
    return fmaf(sum * sb, sa, bias);
}
__device__ __forceinline__ float int8_value(int sum, float sb, float sa, float bias) {
    return int8_value(__int2float_rn(sum), sb, sa, bias);
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
// FLOATS: the sums are the bits of FP32 values.
template <class Out, bool FLOATS, int COLS>
__device__ __forceinline__ void write_columns(typename Out::T *C, long long ldc, int live, const int (&acc)[COLS],
                                              const float (&sa)[(COLS + 31) / 32], float sb, float bias) {
    auto value = [&](int sum, float s) {
        return FLOATS ? int8_value(__int_as_float(sum), sb, s, bias) : int8_value(sum, sb, s, bias);
    };
    if (__all_sync(0xffffffffu, live >= COLS)) {
#pragma unroll
        for (int j = 0; j < COLS; j += 2) {
            const float s0 = __shfl_sync(0xffffffffu, sa[j / 32], j % 32);
            const float s1 = __shfl_sync(0xffffffffu, sa[j / 32], j % 32 + 1);
            const typename Out::Two v = Out::two(value(acc[j], s0), value(acc[j + 1], s1));
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
        const typename Out::Two v = Out::two(value(acc[j], s0), value(acc[j + 1], s1));
        if (j < live) C[0] = Out::lo(v);
        if (j + 1 < live) C[ldc] = Out::hi(v);
        C += 2 * ldc;
    }
}

// offsets[e], kept within the rows there are (whatever the array holds).
__device__ __forceinline__ int bound_of(const Int8Args &a, int e) {
    if (!a.offsets) return e == 0 ? 0 : a.total_rows;
    return min(max(__ldcg(a.offsets + e), 0), a.total_rows);
}

// ---- loads on any alignment -----------------------------------------------------
// The bytes of a matrix: [lo, hi).  Rows that do not start on 16-byte boundaries
// are read in aligned pieces that reach over a row's ends, which is what most of
// the loads below rest on; a piece that reaches over the matrix's own ends is read
// byte by byte.
struct Bytes {
    const int8_t *lo, *hi;
};
__device__ __forceinline__ Bytes matrix_of(const int8_t *p, long long rows, long long ld, int K) {
    return Bytes{p, p + (rows - 1) * ld + K};
}

// Four bytes on any alignment in two steps, so that a thread's loads are all in
// flight before the first is used: the two words that they lie in (`some`: where the
// bytes exist at all), then the bytes -- read one by one at the matrix's own ends,
// where a word would reach over them.
struct Word {
    uint32_t lo, hi, off;
    bool whole;
};
__device__ __forceinline__ Word ask_word(const int8_t *p, bool some, const Bytes &all) {
    Word w;
    w.off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u);
    const int8_t *q = p - w.off;
    w.whole = some && q >= all.lo && q + (w.off ? 8 : 4) <= all.hi;
    w.lo = w.whole ? reinterpret_cast<const uint32_t *>(q)[0] : 0u;
    w.hi = w.whole && w.off ? reinterpret_cast<const uint32_t *>(q)[1] : 0u;
    return w;
}
__device__ __forceinline__ uint32_t take_word(const Word &w, const int8_t *p, bool some, const Bytes &all) {
    uint32_t v = __funnelshift_r(w.lo, w.hi, 8 * w.off);
    if (some && !w.whole)
        for (int i = 0; i < 4; ++i)
            if (p + i < all.hi) v |= static_cast<uint32_t>(static_cast<uint8_t>(p[i])) << (8 * i);
    return v;
}

// ---- generic kernel -----------------------------------------------------------
// 64 x 64 tile of C, 64 k a step as 16 packed words a row, 4 x 4 sums a thread.  Bound
// by the latency of a step's loads, which are all in flight at once: 64 tokens x 1000 x
// 1000 26 us (with a branch around each load 46), x 8192 x 8192 182 (344), stored K x N
// 328 (413).
constexpr int kGTile = 64, kGWords = 16;

// The largest of offsets[0 .. e], kept within the rows there are: expert e's first
// row where the array is out of order too (its last row: that of e + 1).  The whole
// block takes part.
__device__ __forceinline__ int highest_bound(const Int8Args &a, int e) {
    if (!a.offsets) return bound_of(a, e);
    __shared__ int part[8];
    int top = 0;
    for (int i = threadIdx.x; i <= e; i += 256) top = max(top, bound_of(a, i));
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();  // the call before has been read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) top = max(top, part[w]);
    return top;
}

__global__ void __launch_bounds__(256) int8_generic_kernel(const Int8Args a) {
    __shared__ int As[kGWords][kGTile + 1], Bs[kGWords][kGTile + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int n0 = blockIdx.x * kGTile;
    const Bytes all_a = matrix_of(a.A, a.total_rows, a.lda, a.K);
    for (int e = blockIdx.z; e < a.experts; e += gridDim.z) {
        const int8_t *B = a.B + e * a.strideB;
        const Bytes all_b = a.transB ? matrix_of(B, a.N, a.ldb, a.K) : matrix_of(B, a.K, a.ldb, a.N);
        const int first = highest_bound(a, e), last = max(first, bound_of(a, e + 1));
        const int lo = max(first, a.row0), hi = min(last, a.row0 + a.rows);
        for (int m0 = lo + static_cast<int>(blockIdx.y) * kGTile; m0 < hi; m0 += static_cast<int>(gridDim.y) * kGTile) {
            int acc[4][4] = {};
            for (int k0 = 0; k0 < a.K; k0 += 4 * kGWords) {
                Word wa[4], wb[4];
                uint32_t kn[4] = {};  // B stored K x N: four rows' bytes
                auto each = [&](auto f) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = tid + r * 256, w = at % kGWords, i = at / kGWords, k = k0 + 4 * w;
                        f(r, w, i, k, a.A + static_cast<long long>(m0 + i) * a.lda + k, k < a.K && m0 + i < hi,
                          B + static_cast<long long>(n0 + i) * a.ldb + k, k < a.K && n0 + i < a.N);
                    }
                };
                each([&](int r, int, int i, int k, const int8_t *pa, bool some_a, const int8_t *pb, bool some_b) {
                    wa[r] = ask_word(pa, some_a, all_a);
                    if (a.transB) {
                        wb[r] = ask_word(pb, some_b, all_b);
                    } else {
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (k + b < a.K && some_b)
                                kn[r] |= static_cast<uint32_t>(static_cast<uint8_t>(
                                             B[static_cast<long long>(k + b) * a.ldb + n0 + i])) << (8 * b);
                    }
                });
                each([&](int r, int w, int i, int k, const int8_t *pa, bool some_a, const int8_t *pb, bool some_b) {
                    // (A's bytes from K on are zeros, so that B's may be any)
                    uint32_t av = take_word(wa[r], pa, some_a, all_a);
                    if (a.K - k < 4) av &= k < a.K ? (1u << (8 * (a.K - k))) - 1u : 0u;
                    As[w][i] = static_cast<int>(av);
                    Bs[w][i] = static_cast<int>(a.transB ? take_word(wb[r], pb, some_b, all_b) : kn[r]);
                });
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
                    const float sa = __ldcg(a.scaleA + row);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int ch = n0 + tx + 16 * j;
                        if (ch >= a.N) continue;
                        const long long at = static_cast<long long>(e) * a.N + ch;
                        const float v =
                            int8_value(acc[i][j], __ldcg(a.scaleB + at), sa, a.bias ? __ldcg(a.bias + at) : 0.f);
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

// Bytes of v from the `left`-th on made zeros.
__device__ __forceinline__ uint4 zeros_from(uint4 v, int left) {
    auto keep = [&](uint32_t w, int n) { return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u); };
    return make_uint4(keep(v.x, left), keep(v.y, left - 4), keep(v.z, left - 8), keep(v.w, left - 12));
}

// Bytes k..k+15 of a row of K (zeros from K on): 16 bytes at once where `vec` says
// that rows start on 16-byte boundaries, otherwise five words and a shift.
__device__ __forceinline__ uint4 load_int8x16(const int8_t *row, int k, int K, bool vec, const Bytes &all) {
    const int8_t *p = row + k;
    if (vec && k + 16 <= K) return __ldcg(reinterpret_cast<const uint4 *>(p));
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u);
    uint32_t w[5] = {};
    if (p - off >= all.lo && p - off + 20 <= all.hi) {
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p - off);
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = __ldca(q + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * off);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (k + i < K) w[i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(__ldca(p + i))) << (8 * (i % 4));
    }
    return zeros_from(make_uint4(w[0], w[1], w[2], w[3]), K - k);
}

// Rows on any alignment, a warp at a time: lane l reads the aligned 16 bytes in
// which bytes k .. k + 15 of the row begin (ALIGNED: that is those bytes), and
// takes their end from lane l + 1, which reads the next ones; so 31 lanes get 16
// bytes each.  A chunk that a row's first or last byte is in is read whole (bytes
// between the matrix's rows with it, of whatever value), except at the matrix's
// own ends [lo, hi), where it is put together from words, the one that an end is in
// byte by byte, with zeros outside.
// (Byte by byte at every row's ends, a load waits for them there: one token x 700 x
// 700 4.1 us instead of 3.5.)
template <bool ALIGNED>
__device__ __forceinline__ uint4 load_chunk(const int8_t *row, int k, int K, const Bytes &all) {
    const int off = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u);
    const int first = k - off;  // of the row, the chunk's first byte
    if (first >= K) return make_uint4(0, 0, 0, 0);
    const int8_t *p = row + first;
    if (p >= all.lo && p + 16 <= all.hi) return __ldcg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int8_t *q = p + 4 * i;
        const bool whole = q >= all.lo && q + 4 <= all.hi;
        w[i] = whole ? __ldca(reinterpret_cast<const uint32_t *>(q)) : 0u;
        if (!whole && q + 4 > all.lo && q < all.hi)  // a word that an end is in
            for (int b = 0; b < 4; ++b)
                if (q + b >= all.lo && q + b < all.hi) w[i] |= static_cast<uint32_t>(static_cast<uint8_t>(__ldca(q + b))) << (8 * b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// The 16 bytes that begin in this lane's chunk (lane 31: not its own).
__device__ __forceinline__ uint4 join_next(const uint4 &v, const int8_t *row) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
    uint32_t w[8] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = off & 8u ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = off & 4u ? w[i + 1] : w[i];
    const uint32_t bits = 8 * (off & 3u);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// The tokens' rows as FP16, 16 k a thread; ldd is a multiple of 64, so its rows
// divide into whole threads.  *peak: the largest sum of |a| over the 512 k (of
// one row, or the end of one and the start of the next) that a warp of the block
// converts at a time.
__device__ __forceinline__ void rows_to_f16(const Int8Copies &c, int block, int blocks, int *peak) {
    __shared__ int part[8];
    uint4 *dst = static_cast<uint4 *>(c.a_dst);
    const Bytes all = matrix_of(c.A, c.a_rows, c.lda, c.K);
    const int per_row = c.a_ld / 16;
    const long long total = static_cast<long long>(c.a_rows) * per_row;
    int top = 0;
    for (long long i0 = block * 256ll; i0 < total; i0 += blocks * 256ll) {
        const long long i = i0 + threadIdx.x;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i < total) {
            const long long row = div_floor(i, per_row);
            const int k = static_cast<int>(i - row * per_row) * 16;
            if (k < c.K) v = load_int8x16(c.A + row * c.lda, k, c.K, c.a_vec, all);
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
        *peak = top;
    }
}

// Rows of int8 copied onto 16-byte boundaries (ldd a multiple of 16; columns
// K..ldd-1 hold anything: no tensor map reaches them), 31 pieces of a row a warp and
// load, four loads at a time; row r of matrix m is m * rows + r of dst.
constexpr int kRealignRuns = 4;
__device__ __forceinline__ void realign(const int8_t *src, long long ld, long long stride, int matrices, int rows, int K,
                                        int8_t *dst, int ldd, int block, int blocks) {
    const int pieces = ldd / 16, tasks = (pieces + 31 * kRealignRuns - 1) / (31 * kRealignRuns), lane = threadIdx.x & 31;
    const long long total = static_cast<long long>(matrices) * rows * tasks;
    for (long long i = block * 8ll + (threadIdx.x >> 5); i < total; i += blocks * 8ll) {
        const long long row = div_floor(i, tasks), m = matrices > 1 ? div_floor(row, rows) : 0;
        const int piece = static_cast<int>(i - row * tasks) * (31 * kRealignRuns) + lane;
        const int8_t *s = src + m * stride + (row - m * rows) * ld;
        const Bytes all = matrix_of(src + m * stride, rows, ld, K);
        uint4 v[kRealignRuns];
#pragma unroll
        for (int r = 0; r < kRealignRuns; ++r) v[r] = load_chunk<false>(s, (piece + 31 * r) * 16, K, all);
#pragma unroll
        for (int r = 0; r < kRealignRuns; ++r) {
            const uint4 o = join_next(v[r], s);
            if (lane < 31 && piece + 31 * r < pieces) reinterpret_cast<uint4 *>(dst + row * ldd)[piece + 31 * r] = o;
        }
    }
}
// Blocks for it: a warp a task.
long long realign_blocks(long long rows, int ldd) {
    return (rows * ((ldd / 16 + 31 * kRealignRuns - 1) / (31 * kRealignRuns)) + 7) / 8;
}

// B stored K x N -> N x ldd: a tile of 128 k x 64 channels.  A thread reads four
// channels of four rows, turns the 4 x 4 bytes round and stores four words, four
// k of a channel each, in shared memory rows of 33 words: the writes of a warp
// (8 x 4 channels, 4 k words) and its reads (4 channels, 16 k of each of 8
// threads) fall in 32 distinct banks.
constexpr int kTK = 128, kTN = 64;

template <bool WORDS>
__device__ __forceinline__ void transpose(const Int8Copies &c, int block, int blocks) {
    __shared__ uint32_t tile[kTN][kTK / 4 + 1];
    const int tiles_k = (c.b_ld + kTK - 1) / kTK, tiles_n = (c.N + kTN - 1) / kTN;
    const long long total = static_cast<long long>(c.experts) * tiles_k * tiles_n;
    for (long long t = block; t < total; t += blocks) {
        const long long e = div_floor(t, tiles_k * static_cast<long long>(tiles_n));
        const int r = static_cast<int>(t - e * tiles_k * tiles_n);
        const int n0 = r % tiles_n * kTN, k0 = r / tiles_n * kTK;
        const int8_t *src = c.B + e * c.strideB;
        int8_t *d = c.b_dst + e * c.N * c.b_ld;
        // All words are asked for before any is used; of a misaligned four bytes the
        // two words that they lie in, read whole.  What is beyond the row goes to
        // channels that do not exist; only at the matrix's own ends (rows on word
        // boundaries: at theirs) the bytes are read one by one.  (Byte by byte at every
        // row's ends: 40 x 133 x 266 7.9 us instead of 6.1, 1000 x 1500 x 777 15.1
        // instead of 14.4.)
        const Bytes all = matrix_of(src, c.K, c.ldb, c.N);
        uint32_t w[2][4];
        uint32_t next[2][4];
        bool ends = false;
        auto each = [&](auto f) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = threadIdx.x + h * 256, n = n0 + (at % 8 + at / 256 % 2 * 8) * 4, k = k0 + at / 8 % 32 * 4;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int8_t *p = src + static_cast<long long>(k + j) * c.ldb + n;
                    const uint32_t off = WORDS ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u);
                    const bool some = k + j < c.K && n < c.N;
                    const bool whole =
                        some && (WORDS ? n + 4 <= c.N : p - off >= all.lo && p - off + (off ? 8 : 4) <= all.hi);
                    f(h, j, n, p, off, some, whole);
                }
            }
        };
        auto bytes = [&](const int8_t *p, int n) {
            uint32_t v = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (n + b < c.N) v |= static_cast<uint32_t>(static_cast<uint8_t>(__ldca(p + b))) << (8 * b);
            return v;
        };
        each([&](int h, int j, int n, const int8_t *p, uint32_t off, bool some, bool whole) {
            const uint32_t *q = reinterpret_cast<const uint32_t *>(p - off);
            w[h][j] = whole ? (WORDS ? __ldcg(q) : __ldca(q)) : WORDS && some ? bytes(p, n) : 0u;
            next[h][j] = !WORDS && whole && off ? __ldca(q + 1) : 0u;
            ends |= !WORDS && some && !whole;
        });
        if (!WORDS)
            each([&](int h, int j, int, const int8_t *, uint32_t off, bool, bool) {
                w[h][j] = __funnelshift_r(w[h][j], next[h][j], 8 * off);
            });
        if (ends)
            each([&](int h, int j, int n, const int8_t *p, uint32_t, bool some, bool whole) {
                if (some && !whole) w[h][j] = bytes(p, n);
            });
        __syncthreads();  // the tile before has been read
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = threadIdx.x + h * 256, n4 = at % 8 + at / 256 % 2 * 8, k4 = at / 8 % 32;
            const uint32_t a = __byte_perm(w[h][0], w[h][1], 0x5140), b = __byte_perm(w[h][2], w[h][3], 0x5140);
            const uint32_t x = __byte_perm(w[h][0], w[h][1], 0x7362), y = __byte_perm(w[h][2], w[h][3], 0x7362);
            tile[n4 * 4 + 0][k4] = __byte_perm(a, b, 0x5410);
            tile[n4 * 4 + 1][k4] = __byte_perm(a, b, 0x7632);
            tile[n4 * 4 + 2][k4] = __byte_perm(x, y, 0x5410);
            tile[n4 * 4 + 3][k4] = __byte_perm(x, y, 0x7632);
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = threadIdx.x + h * 256, kg = at % 8, n = at / 8;
            if (n0 + n < c.N && k0 + kg * 16 < c.b_ld)
                *reinterpret_cast<uint4 *>(d + static_cast<long long>(n0 + n) * c.b_ld + k0 + kg * 16) =
                    make_uint4(tile[n][kg * 4], tile[n][kg * 4 + 1], tile[n][kg * 4 + 2], tile[n][kg * 4 + 3]);
        }
    }
}

// Both operands' copies in one launch: blocks [0, b_blocks) copy B, the rest A.
// WORDS: B's rows start on word boundaries (fewer registers, five CTAs an SM instead
// of four: B 8192 x 8192 stored K x N, 16 tokens 48 us instead of 52).
template <bool WORDS>
__global__ void __launch_bounds__(256, WORDS ? 5 : 4) int8_copies_kernel(const Int8Copies c) {
    griddep_wait();
    griddep_launch_dependents();
    const int block = static_cast<int>(blockIdx.x);
    if (block < c.b_blocks) {
        if (c.b_trans) realign(c.B, c.ldb, c.strideB, c.experts, c.N, c.K, c.b_dst, c.b_ld, block, c.b_blocks);
        else transpose<WORDS>(c, block, c.b_blocks);
    } else if (c.peaks) {
        rows_to_f16(c, block - c.b_blocks, c.a_blocks, c.peaks + block - c.b_blocks);
    } else {
        realign(c.A, c.lda, 0, 1, c.a_rows, c.K, static_cast<int8_t *>(c.a_dst), c.a_ld, block - c.b_blocks, c.a_blocks);
    }
}

// ---- few tokens: the CUDA cores -----------------------------------------------------
// Up to 8 tokens: a warp takes two channels, its lanes 16 k each of a step, dp4a
// against the tokens' rows in shared memory; warps of a CTA may share a channel's
// K range (`split`).  One launch, no copies (B on any alignment), no cluster: a
// step of one or a few tokens is made of the launch and one latency of HBM, and
// for so few sums dp4a's rate does not show.  One token x 4096 x 4096 4.9 us (on the
// tensor cores 6.8), x 8192 x 8192 13.5 (14.8; 5.0 TB/s), x 8190 x 8190 17.0 (36.7, with
// B's copy); 4 tokens 6.8, 18.4, 24.5; 8 tokens 11.3 or more: choose_few in
// sgemm_ops_api.cu says which kernel runs.
constexpr int kFewThreads = 256;

constexpr int kFewC = 2, kFewAhead = 2;  // channels a warp; steps whose loads are in flight

// Four CTAs an SM (64 registers a thread) where the sums leave room for it: more
// warps hide more than more loads a warp do (one token x 4096 x 4096: 4.8 us; four
// steps ahead at two CTAs 6.2; 8 tokens spill at four).
template <int MT, bool VEC>
__global__ void __launch_bounds__(kFewThreads, MT <= 4 ? 4 : 2) int8_few_kernel(const Int8Args a, int split, int a_vec) {
    constexpr int C = kFewC, AHEAD = kFewAhead;
    constexpr int L = VEC ? 32 : 31;  // pieces of 16 k a step (join_next)
    extern __shared__ uint4 rows[];   // [token][16 k], zeros beyond K (where B's bytes may be any) and the last token
    __shared__ int part[kFewThreads / 32][MT * C];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pieces = (a.K + 15) / 16, steps = (pieces + L - 1) / L;
    const int group = warp / split, member = warp % split, groups = kFewThreads / 32 / split;
    const int n0 = (static_cast<int>(blockIdx.x) * groups + group) * C;
    const int8_t *b[C];
#pragma unroll
    for (int c = 0; c < C; ++c) b[c] = a.B + static_cast<long long>(n0 + c < a.N ? n0 + c : a.N - 1) * a.ldb;
    // the first steps of B into L2 while the kernel before this one ends
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) {
        const int k = ((s * split + member) * L + lane) * 16;
        if (k < a.K)
#pragma unroll
            for (int c = 0; c < C; ++c) asm volatile("prefetch.global.L2 [%0];" ::"l"(b[c] + k));
    }
    griddep_wait();
    griddep_launch_dependents();

    const Bytes all = matrix_of(a.B, a.N, a.ldb, a.K), all_a = matrix_of(a.A, a.rows, a.lda, a.K);
    int sum[MT][C] = {};
    uint4 raw[AHEAD][C];
    auto fetch = [&](int s0) {
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) {
            const int k = (((s0 + s) * split + member) * L + lane) * 16;
#pragma unroll
            for (int c = 0; c < C; ++c) raw[s][c] = load_chunk<VEC>(b[c], k, a.K, all);
        }
    };
    fetch(0);
    for (int i = threadIdx.x; i < MT * pieces; i += kFewThreads) {
        const int t = i / pieces, k = (i - t * pieces) * 16;
        rows[i] = t < a.rows ? load_int8x16(a.A + static_cast<long long>(t) * a.lda, k, a.K, a_vec, all_a) : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int mine = (steps - member + split - 1) / split;  // this warp's steps
    for (int s0 = 0; s0 < mine; s0 += AHEAD) {
        uint4 w[AHEAD][C];
#pragma unroll
        for (int s = 0; s < AHEAD; ++s)
#pragma unroll
            for (int c = 0; c < C; ++c) w[s][c] = VEC ? raw[s][c] : join_next(raw[s][c], b[c]);
        if (s0 + AHEAD < mine) fetch(s0 + AHEAD);
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) {
            const int piece = ((s0 + s) * split + member) * L + lane;
            if (piece < pieces && (VEC || lane < L)) {
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const uint4 x = rows[t * pieces + piece];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        sum[t][c] = __dp4a(static_cast<int>(x.x), static_cast<int>(w[s][c].x), sum[t][c]);
                        sum[t][c] = __dp4a(static_cast<int>(x.y), static_cast<int>(w[s][c].y), sum[t][c]);
                        sum[t][c] = __dp4a(static_cast<int>(x.z), static_cast<int>(w[s][c].z), sum[t][c]);
                        sum[t][c] = __dp4a(static_cast<int>(x.w), static_cast<int>(w[s][c].w), sum[t][c]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int all = __reduce_add_sync(0xffffffffu, sum[t][c]);
            if (lane == t * C + c) part[warp][lane] = all;
        }
    __syncthreads();
    // one thread a token and channel: consecutive channels of a token together
    for (int i = threadIdx.x; i < MT * groups * C; i += kFewThreads) {
        const int t = i / (groups * C), ch = i % (groups * C);
        const int n = static_cast<int>(blockIdx.x) * groups * C + ch;
        if (t >= a.rows || n >= a.N) continue;
        int total = 0;
        for (int m = 0; m < split; ++m) total += part[ch / C * split + m][t * C + ch % C];
        const float v = int8_value(total, __ldcg(a.scaleB + n), __ldcg(a.scaleA + t), a.bias ? __ldcg(a.bias + n) : 0.f);
        with_out_type(a.out_type, [&](auto out) {
            using Out = decltype(out);
            static_cast<typename Out::T *>(a.C)[static_cast<long long>(t) * a.ldc + n] = Out::lo(Out::two(v, 0.f));
        });
    }
}

// ---- tensor-core kernels -----------------------------------------------------------
constexpr int kBBytes = kI8TileN * kI8StageK;  // 16 KiB of B a stage
constexpr int kACols = kI8StageK / 2;          // 32-bit columns of tensor memory that hold a stage of B
constexpr int kChunk = 8;                      // stages (1024 k) whose sums fit an accumulator whatever the data
constexpr int kSmemLimit = 232448;             // dynamic shared memory of a CTA that has the SM to itself

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

template <int R>
__device__ __forceinline__ void regs_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

// sum + f for an integer f of magnitude <= 2^24, by the FP32 and integer pipes:
// adding M = 1.5 * 2^23 leaves a value below 2^22 rounded to an integer in the low
// bits, so h = f / 4096 + M holds round(f / 4096), r = f - 4096 * (h - M) the rest
// (exact, at most 2048), and the bits of h, shifted, and of r + M add up to f but
// for a constant (arithmetic modulo 2^32).
__device__ __forceinline__ int add_integer(int sum, float f) {
    constexpr float kM = 12582912.f;
    constexpr unsigned kBits = 0x4b400000u, kConst = (kBits << 12) + kBits;
    const float h = fmaf(f, 1.f / 4096.f, kM);
    const float r = __fadd_rn(fmaf(__fadd_rn(h, -kM), -4096.f, f), kM);
    return static_cast<int>(static_cast<unsigned>(sum) + ((__float_as_uint(h) << 12) + __float_as_uint(r)) - kConst);
}

// How an accumulator is taken over: its integers added to sums of which they are
// a part, or kept as the FP32 values that they are where one holds all of K.
enum class Take { kAdd, kOnly };

// acc[j] += column j of an accumulator (kOnly: acc[j] = its bits): the load of
// the next 16 columns is in flight while 16 are converted.  The conversion
// instruction runs at an eighth of the rate of an addition (128 columns in two
// warpgroups: 2300 cycles), so 9 of 16 columns go round it.
template <Take TAKE, int COLS>
__device__ __forceinline__ void drain(uint32_t tmem, int (&acc)[COLS]) {
    uint32_t v[2][16];
    tc::tmem_ld16_begin(tmem, v[0]);
    tc::tmem_ld_wait(v[0]);
#pragma unroll
    for (int c = 0; c < COLS / 16; ++c) {
        if (c + 1 < COLS / 16) tc::tmem_ld16_begin(tmem + (c + 1) * 16, v[(c + 1) & 1]);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            int &sum = acc[c * 16 + j];
            const float f = __uint_as_float(v[c & 1][j]);
            if (TAKE == Take::kOnly) sum = static_cast<int>(v[c & 1][j]);
            else if (j % 2 == 1 && j < 15) sum += __float2int_rn(f);
            else sum = add_integer(sum, f);
        }
        if (c + 1 < COLS / 16) tc::tmem_ld_wait(v[(c + 1) & 1]);
    }
}

struct I8Unit {
    int e, ch0, t0, tend;
};

// The largest e with before[e] * each <= u.
__device__ __forceinline__ int owner_of(const int *before, int experts, int each, int u) {
    int lo = 0, hi = experts;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (before[mid] * each <= u) lo = mid; else hi = mid;
    }
    return lo;
}

// Unit u of tiles of NT tokens x CH channels: the expert by bisection of the
// tile counts; within the expert groups of 2048 tokens or 16 tiles, channel
// tiles outer and token tiles inner.  TAILS: then the experts' last tiles of up to
// NT / 2 tokens, which take half the time: in this order the CTAs that get one
// tile more than others get a short one.
template <int NT, int CH, bool TAILS>
__device__ __forceinline__ I8Unit unit_of(const int *bound, const int *tiles, const int *tails, const Int8Args &a,
                                          int ch_tiles, int u) {
    I8Unit q;
    int tile;
    const int whole = tiles[a.experts] * ch_tiles;
    if (!TAILS || u < whole) {
        constexpr int kGroup = 2048 / NT < 16 ? 2048 / NT : 16;
        q.e = owner_of(tiles, a.experts, ch_tiles, u);
        const int mine = tiles[q.e + 1] - tiles[q.e];
        const int l = u - tiles[q.e] * ch_tiles;
        const int grp = l / (kGroup * ch_tiles), first = grp * kGroup;
        const int rows = min(mine - first, kGroup);
        const int r = l - grp * kGroup * ch_tiles;
        q.ch0 = r / rows * CH;
        tile = first + r % rows;
    } else {
        q.e = owner_of(tails, a.experts, ch_tiles, u - whole);
        q.ch0 = (u - whole - tails[q.e] * ch_tiles) * CH;
        tile = tiles[q.e + 1] - tiles[q.e];
    }
    q.t0 = max(bound[q.e], a.row0) + tile * NT;
    q.tend = min(bound[q.e + 1], a.row0 + a.rows);
    return q;
}

// One warp: bound[e], the experts' first rows (nondecreasing), and tiles[e], the
// token tiles of the experts before e (experts + 1 of each); returns all of them.
// TAILS: tiles[] counts the tiles of more than nt / 2 tokens, tails[] the rest (an
// expert has one at most), and the tiles of tails[] come after all of tiles[].
template <bool TAILS>
__device__ __forceinline__ int sum_tiles(int *bound, int *tiles, int *tails, const Int8Args &a, int nt, int lane) {
    int top = 0, sum = 0, tail_sum = 0;
    for (int e0 = 0; e0 <= a.experts; e0 += 32) {
        const int e = e0 + lane;
        int b = e <= a.experts ? bound_of(a, e) : 0;
        b = max(b, top);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, b, d);
            if (lane >= d) b = max(b, up);
        }
        if (e <= a.experts) bound[e] = b;
        top = __shfl_sync(0xffffffffu, b, 31);
    }
    __syncwarp();
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
        const int e = e0 + lane;
        int n = 0, tail = 0;
        if (e < a.experts) {
            const int rows = max(min(bound[e + 1], a.row0 + a.rows) - max(bound[e], a.row0), 0);
            n = (rows + (TAILS ? nt / 2 : nt) - 1) / nt;
            tail = TAILS && rows > n * nt ? 1 : 0;
        }
        int s = n, t = tail;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, s, d), upt = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) {
                s += up;
                t += upt;
            }
        }
        if (e < a.experts) {
            tiles[e] = sum + s - n;
            if (TAILS) tails[e] = tail_sum + t - tail;
        }
        sum += __shfl_sync(0xffffffffu, s, 31);
        tail_sum += __shfl_sync(0xffffffffu, t, 31);
    }
    if (lane == 0) {
        tiles[a.experts] = sum;
        if (TAILS) tails[a.experts] = tail_sum;
    }
    return sum + tail_sum;
}

// Stages between drains, from the tokens' own size.  rows_to_f16 leaves in
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

// 128 k of this thread's channel (128 bytes) as FP16 into 64 columns of its lane
// of tensor memory (whole warp; the stores are still to be waited for).
__device__ __forceinline__ void expand_to_tmem(const uint4 (&w)[8], uint32_t taddr) {
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
        tc::tmem_st32(taddr + h * 32, o);
    }
}

// ---- up to 64 tokens a tile: 128 channels x NT tokens, two CTAs an SM -----------------
// Four warpgroup-sized parts in 12 warps, so that two CTAs share an SM: each
// hides the other's waits, and the next call's CTAs set themselves up while
// the last ones of this call finish.
constexpr int kMaxStages = 6, kXStages = 2, kAStages = 2;
constexpr int kDirectThreads = 384;
constexpr uint32_t kDirectTmemCols = 256;
// Two CTAs an SM: half of its 228 KiB less 1 KiB each that the system reserves.
constexpr int kHalfSmem = 233472 / 2 - 1024;

struct DirectShared {
    uint64_t full[kMaxStages];    // B and the tokens' int8 of the stage have landed
    uint64_t empty[kMaxStages];   // four warps have read B, two the tokens
    uint64_t xfull[kXStages];     // the stage's tokens stand in shared memory as FP16 (two warps)
    uint64_t xempty[kXStages];    // the MMAs have read them
    uint64_t afull[kAStages];     // the stage's B stands in tensor memory (four warps)
    uint64_t aempty[kAStages];    // the MMAs have read it
    uint64_t dfull[2];            // an accumulator holds up to 1024 k
    uint64_t dempty[2];           // it has been read (four warps)
    uint64_t xchg_read;           // the cluster's partial sums have been read (four warps)
    uint64_t drained;             // abort only: every MMA issued has finished
    uint32_t tmem_base;
    int abort;
    int units;                    // units of this launch
    // then bound[experts + 1], tiles[experts + 1]
};

// Partial sums of a channel that cross the cluster together.
template <int V>
struct ExchangeVec;
template <>
struct ExchangeVec<2> {
    using T = int2;
    static __device__ __forceinline__ void rest(int2, int (&)[2]) {}
};
template <>
struct ExchangeVec<4> {
    using T = int4;
    static __device__ __forceinline__ void rest(int4 v, int (&sum)[4]) {
        sum[2] += v.z;
        sum[3] += v.w;
    }
};

template <int NT, bool SPLIT>
struct DirectCfg {
    static constexpr int kStage = kBBytes + NT * kI8StageK;
    static constexpr int kXBytes = NT * kI8StageK * 2;
    // The partial sums from the cluster's CTAs: in place of the FP16 tokens, which
    // are done with by then, except in the narrowest tile, whose 8 KiB fit beside.
    static constexpr int kXchgBytes = SPLIT ? kI8TileN * NT * 4 : 0;
    static constexpr bool kXchgOwn = NT == 16;
    static constexpr int kFixed = 1024 + kXStages * kXBytes + (kXchgOwn ? kXchgBytes : 0) + static_cast<int>(sizeof(DirectShared));
    static constexpr int kFit = (kHalfSmem - kFixed - 64) / kStage;
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    static constexpr int smem(int experts) { return kFixed + kStages * kStage + 2 * 4 * (experts + 1); }
    // Registers (80 a thread at launch): a thread of the widest tile's epilogue
    // holds 64 sums.
    static constexpr bool kRegs = NT == 64;
    static constexpr int kRegsControl = 56, kRegsEpilogue = 104;
    static_assert(kXchgOwn || kXchgBytes <= kXStages * kXBytes, "partial sums");
    static_assert(2 * NT + kAStages * kACols <= static_cast<int>(kDirectTmemCols), "tensor memory");
    static_assert(kStages >= 3, "shared memory");
    static_assert(!kRegs || kRegsControl + 80 + kRegsEpilogue <= 3 * 80, "register split");
    static_assert(!SPLIT || NT / 2 <= 32, "a lane holds a token scale");
};

template <int NT, bool SPLIT>
__global__ void __launch_bounds__(kDirectThreads, 2)
int8_tc_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA, const Int8Args a) {
    using Cf = DirectCfg<NT, SPLIT>;
    constexpr int S = Cf::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;  // the same in every CTA
    uint8_t *ring = smem_raw + pad, *ring_x = ring + S * Cf::kStage;
    uint8_t *after = ring_x + kXStages * Cf::kXBytes;
    int *xchg = reinterpret_cast<int *>(Cf::kXchgOwn ? after : ring_x);
    DirectShared *sh = reinterpret_cast<DirectShared *>(after + (Cf::kXchgOwn ? Cf::kXchgBytes : 0));
    int *bound = reinterpret_cast<int *>(sh + 1), *tiles = bound + a.experts + 1;
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
        for (int s = 0; s < S; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 4 + 2);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh->xfull[s], 2);
            mbar_init(&sh->xempty[s], 1);
            mbar_init(&sh->afull[s], 4);
            mbar_init(&sh->aempty[s], 1);
            mbar_init(&sh->dfull[s], 1);
            mbar_init(&sh->dempty[s], 4);
        }
        mbar_init(&sh->xchg_read, 4);
        mbar_init(&sh->drained, 1);
        sh->abort = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmA);
    }
    if (warp == 1) {
        tc::tmem_alloc(&sh->tmem_base, kDirectTmemCols);
        tc::tmem_relinquish();
    }
    // One expert's tiles do not depend on device memory.  Its first stages of B
    // are fetched into L2 ahead of the wait for the kernel before this one (a
    // prefetch returns no data, so it does not matter whether that kernel has
    // yet to write them).
    if (!a.offsets && warp == 2) {
        const int n = sum_tiles<false>(bound, tiles, nullptr, a, NT, lane);
        if (lane == 0) sh->units = n * ch_tiles;
        __syncwarp();
        if (first_unit < n * ch_tiles) {
            const I8Unit q = unit_of<NT, kI8TileN, false>(bound, tiles, nullptr, a, ch_tiles, first_unit);
            if (lane < S && kb + lane < ke) tma_prefetch_3d(&tmB, (kb + lane) * kI8StageK, q.ch0, q.e);
        }
    }
    griddep_wait();
    griddep_launch_dependents();
    if (a.offsets && warp == 2) {
        const int n = sum_tiles<false>(bound, tiles, nullptr, a, NT, lane);
        if (lane == 0) sh->units = n * ch_tiles;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
    const uint32_t tmem_a = tmem + 2 * NT;
    volatile int *abort_flag = &sh->abort;
    const int units = sh->units;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity, a.status)) return true;
        *abort_flag = 1;
        return false;
    };
    // Every thread of the cluster passes two barriers a unit: every CTA is ready
    // for the others' partial sums; all partial sums have been sent.
    auto pass_exchange = [&]() {
        if (SPLIT) {
            __syncwarp();
            cluster_sync();
            cluster_sync();
        }
    };

    if (warp < 4) {
        if (Cf::kRegs) regs_fewer<Cf::kRegsControl>();
        if (warp == 0) {
            // -------------------------------------------- TMA producer
            Ring r;
            int issued = 0;
            bool ok = true;
            for (int u = first_unit; u < units; u += unit_step) {
                if (lane == 0 && ok) {
                    const I8Unit q = unit_of<NT, kI8TileN, false>(bound, tiles, nullptr, a, ch_tiles, u);
                    for (int i = kb; i < ke; ++i, r.step(S), ++issued) {
                        if (!wait(&sh->empty[r.s], r.round ^ 1u)) { ok = false; break; }
                        uint8_t *st = ring + r.s * Cf::kStage;
                        mbar_arrive_expect_tx(&sh->full[r.s], Cf::kStage);
                        tma_load_3d(st, &tmB, &sh->full[r.s], i * kI8StageK, q.ch0, q.e);
                        tma_load_2d(st + kBBytes, &tmA, &sh->full[r.s], i * kI8StageK, q.t0 - a.row0);
                    }
                }
                pass_exchange();
            }
            if (lane == 0)  // no copy outlives the CTA
                for (int t = max(0, issued - S); t < issued; ++t) mbar_wait(&sh->full[t % S], (t / S) & 1, a.status);
            __syncwarp();
        } else if (warp == 1) {
            // -------------------------------------------- MMA issuer
            // The whole warp walks the stages and waits; one elected lane issues.
            constexpr uint32_t idesc = tc::idesc_f16_kmajor(kI8TileN, NT);
            const uint64_t xdesc = tc::smem_desc(smem_u32(ring_x), 16, 1024, tc::kLayoutSwizzle128);
            Ring x, t, d;  // stages of tokens and of B in tensor memory, accumulators
            bool ok = true;
            for (int u = first_unit; u < units; u += unit_step) {
                int run = 0;  // stages in the accumulator so far
                for (int i = kb; i < ke && ok; ++i) {
                    const bool start = run == 0, end = i + 1 == ke || run + 1 == kChunk;
                    ok = (!start || wait(&sh->dempty[d.s], d.round ^ 1u)) && wait(&sh->xfull[x.s], x.round) &&
                         wait(&sh->afull[t.s], t.round);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (tc::elect_one()) {
                        const uint64_t b = xdesc + static_cast<uint64_t>(x.s * (Cf::kXBytes / 16));
#pragma unroll
                        for (int kk = 0; kk < kI8StageK / 16; ++kk)
                            tc::mma_f16_ta(tmem + d.s * NT, tmem_a + t.s * kACols + kk * 8,
                                           b + ((kk / 4) * NT * 128 + (kk % 4) * 32) / 16, idesc,
                                           (start && kk == 0) ? 0u : 1u);
                        tc::commit(&sh->xempty[x.s]);
                        tc::commit(&sh->aempty[t.s]);
                        if (end) tc::commit(&sh->dfull[d.s]);
                    }
                    __syncwarp();
                    x.step(kXStages);
                    t.step(kAStages);
                    run = end ? 0 : run + 1;
                    if (end) d.step(2);
                }
                pass_exchange();
            }
            if (!ok && tc::elect_one()) {  // no teardown under a running MMA
                tc::commit(&sh->drained);
                mbar_wait(&sh->drained, 0, a.status);
            }
            __syncwarp();
        } else {
            // -------------------------------------------- the tokens' rows to FP16 (two warps)
            constexpr int kPieces = NT / 8, kBatch = kPieces < 4 ? kPieces : 4;  // 16-byte pieces of a stage a thread expands
            const int me = tid - 64;
            const int kc = me % 8, up = kc / 4, c = (kc % 4) * 2;  // 16 k of a row; rows me / 8, me / 8 + 8, ..
            const int sw = (me / 8) & 7;                           // a row's place in its group of 8
            Ring r, x;
            int unit = 0;
            bool ok = true;
            for (int u = first_unit; u < units; u += unit_step, ++unit) {
                if (SPLIT && !Cf::kXchgOwn && unit > 0)
                    ok = __all_sync(0xffffffffu, ok && wait(&sh->xchg_read, (unit - 1) & 1));
                for (int i = kb; i < ke && ok; ++i, r.step(S), x.step(kXStages)) {
                    ok = wait(&sh->full[r.s], r.round) && wait(&sh->xempty[x.s], x.round ^ 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint8_t *src = ring + r.s * Cf::kStage + kBBytes + (me / 8) * 128 + (kc ^ sw) * 16;
                    uint8_t *dst = ring_x + x.s * Cf::kXBytes + up * NT * 128 + (me / 8) * 128;
#pragma unroll
                    for (int j0 = 0; j0 < kPieces; j0 += kBatch) {
                        uint4 v[kBatch];
#pragma unroll
                        for (int j = 0; j < kBatch; ++j)
                            v[j] = *reinterpret_cast<const uint4 *>(src + (j0 + j) * 1024);
#pragma unroll
                        for (int j = 0; j < kBatch; ++j) {
                            // a row's eight lanes write 16-byte columns 2 kc (kc < 4) and
                            // 2 kc + 1 (kc >= 4, in the other box) first, then the other of
                            // the two: eight distinct columns either time
                            uint4 o0, o1;
                            int8x4_to_f16(up ? v[j].z : v[j].x, o0.x, o0.y);
                            int8x4_to_f16(up ? v[j].w : v[j].y, o0.z, o0.w);
                            int8x4_to_f16(up ? v[j].x : v[j].z, o1.x, o1.y);
                            int8x4_to_f16(up ? v[j].y : v[j].w, o1.z, o1.w);
                            *reinterpret_cast<uint4 *>(dst + (j0 + j) * 1024 + (((c + up) ^ sw) * 16)) = o0;
                            *reinterpret_cast<uint4 *>(dst + (j0 + j) * 1024 + (((c + 1 - up) ^ sw) * 16)) = o1;
                        }
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh->xfull[x.s]);
                        mbar_arrive(&sh->empty[r.s]);
                    }
                }
                pass_exchange();
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------ B to FP16, into tensor memory
        const int row = (warp % 4) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        Ring r, t;
        int stored = -1;  // the stage in tensor memory whose stores have not been waited for
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
            for (int i = kb; i < ke && ok; ++i, r.step(S), t.step(kAStages)) {
                // the stage before is handed on while this one is read, unless
                // this one has yet to land
                if (!__all_sync(0xffffffffu, mbar_try_wait(&sh->full[r.s], r.round))) {
                    flush();
                    ok = __all_sync(0xffffffffu, wait(&sh->full[r.s], r.round));
                    if (!ok) break;
                }
                const uint8_t *src = ring + r.s * Cf::kStage + row * kI8StageK;
                uint4 w[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) w[c] = *reinterpret_cast<const uint4 *>(src + ((c ^ (row & 7)) * 16));
                flush();
                ok = __all_sync(0xffffffffu, wait(&sh->aempty[t.s], t.round ^ 1u));
                if (!ok) break;
                tc::fence_after_sync();
                expand_to_tmem(w, tmem_a + t.s * kACols + lanes);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->empty[r.s]);
                stored = t.s;
            }
            flush();
            pass_exchange();
        }
    } else {
        // ------------------------------------------------ accumulators to C
        if (Cf::kRegs) regs_more<Cf::kRegsEpilogue>();
        const int ch = (warp % 4) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        Ring d;
        bool ok = true;
        for (int u = first_unit; u < units; u += unit_step) {
            const I8Unit q = unit_of<NT, kI8TileN, false>(bound, tiles, nullptr, a, ch_tiles, u);
            // What the epilogue needs of global memory, asked for before the sums
            // are ready: the channel's scale and bias, and lane l's share of the
            // token scales (handed round by shuffles).
            const int n = q.ch0 + ch;
            const long long at = static_cast<long long>(q.e) * a.N + n;
            const float sb = n < a.N ? __ldcg(a.scaleB + at) : 0.f;
            const float bias = n < a.N && a.bias ? __ldcg(a.bias + at) : 0.f;
            const int per = SPLIT ? NT / splits : NT;  // this CTA's columns of the result
            const int first = q.t0 + (SPLIT ? rank * per : 0);
            float sa[(NT + 31) / 32];
#pragma unroll
            for (int c = 0; c < (NT + 31) / 32; ++c)
                sa[c] = c * 32 + lane < per && first + c * 32 + lane < q.tend ? __ldcg(a.scaleA + first + c * 32 + lane) : 0.f;
            // (its own room: ready as soon as the last unit's sums have been read)
            if (SPLIT && Cf::kXchgOwn) {
                __syncwarp();
                cluster_arrive();
            }
            int acc[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j] = 0;
            for (int i = kb; i < ke && ok; i += kChunk, d.step(2)) {
                ok = __all_sync(0xffffffffu, wait(&sh->dfull[d.s], d.round));
                if (!ok) break;
                tc::fence_after_sync();
                drain<Take::kAdd>(tmem + d.s * NT + lanes, acc);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->dempty[d.s]);
            }
            if (!SPLIT) {
                if (ok)
                    with_out_type(a.out_type, [&](auto out) {
                        using Out = decltype(out);
                        write_columns<Out, false>(static_cast<typename Out::T *>(a.C) + static_cast<long long>(first) * a.ldc + n,
                                                  a.ldc, n < a.N ? q.tend - first : 0, acc, sa, sb, bias);
                    });
            } else {
                __syncwarp();
                if (!Cf::kXchgOwn) cluster_arrive();
                cluster_wait_acquire();
                // Column j belongs to CTA j / per of the cluster (powers of two).  The
                // partial sums of a channel stand kV columns together, so that they
                // cross in pieces of up to 16 bytes.
                constexpr int kV = NT == 16 ? 2 : 4;  // at most NT / 8, the fewest columns a CTA has
                using Vec = typename ExchangeVec<kV>::T;
                Vec *slots = reinterpret_cast<Vec *>(xchg);  // [CTA][column / kV][channel]
                const int groups = per / kV;
                if (ok) {
                    const int shift = 31 - __clz(groups);
                    const uint32_t mine = smem_u32(slots + rank * groups * kI8TileN + ch);
                    uint32_t to = 0;
#pragma unroll
                    for (int j = 0; j < NT / kV; ++j) {
                        if ((j & (groups - 1)) == 0)
                            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(mine), "r"(j >> shift));
                        const uint32_t at = to + (j & (groups - 1)) * (kI8TileN * kV * 4);
                        if (kV == 2)
                            asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};"
                                         ::"r"(at), "r"(acc[kV * j]), "r"(acc[kV * j + 1]) : "memory");
                        else
                            asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};"
                                         ::"r"(at), "r"(acc[kV * j]), "r"(acc[kV * j + 1]), "r"(acc[kV * j + kV - 2]),
                                           "r"(acc[kV * j + kV - 1]) : "memory");
                    }
                }
                __syncwarp();
                cluster_sync();
                if (ok)
                    with_out_type(a.out_type, [&](auto out) {
                        using Out = decltype(out);
                        auto *C = static_cast<typename Out::T *>(a.C) + static_cast<long long>(first) * a.ldc + n;
                        for (int g = 0; g < groups; ++g) {
                            int sum[kV] = {};
#pragma unroll
                            for (int r = 0; r < 8; ++r)  // all loads in flight at once
                                if (r < splits) {
                                    const Vec v = slots[(r * groups + g) * kI8TileN + ch];
                                    sum[0] += v.x;
                                    sum[1] += v.y;
                                    ExchangeVec<kV>::rest(v, sum);
                                }
#pragma unroll
                            for (int c = 0; c < kV; c += 2) {
                                const int col = g * kV + c;
                                const float f0 = __shfl_sync(0xffffffffu, sa[0], col), f1 = __shfl_sync(0xffffffffu, sa[0], col + 1);
                                const typename Out::Two v =
                                    Out::two(int8_value(sum[c], sb, f0, bias), int8_value(sum[c + 1], sb, f1, bias));
                                if (n < a.N && first + col < q.tend) C[static_cast<long long>(col) * a.ldc] = Out::lo(v);
                                if (n < a.N && first + col + 1 < q.tend) C[static_cast<long long>(col + 1) * a.ldc] = Out::hi(v);
                            }
                        }
                    });
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->xchg_read);
            }
        }
    }
    // ---------------------------------------------------- teardown
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kDirectTmemCols);
    }
}

// ---- CTA pairs: 256 channels x T = 128 or 256 tokens ---------------------------------
constexpr int kPairN = 256;  // channels of a pair's tile
constexpr int kPairASlots = 2, kPairMaxB = 8, kPairMaxX = 3;  // a slot: two stages
constexpr int kPairThreads = 512;
constexpr uint32_t kPairTmemCols = 512;

struct PairShared {
    uint64_t bfull[kPairMaxB], bempty[kPairMaxB];
    // Tokens, and B in tensor memory, two stages (256 k) at a time: what the
    // issuing lane spends on a wait and on a commit it spends half as often.
    uint64_t xfull[2][kPairMaxX];   // (even CTA) both CTAs' tokens of a half have landed
    uint64_t xempty[2][kPairMaxX];  // the MMAs have read them (both CTAs are told)
    uint64_t afull[kPairASlots];    // (even CTA) B stands in both CTAs' tensor memory
    uint64_t aempty[kPairASlots];
    uint64_t dfull[2];              // a half accumulator holds up to `chunk` stages
    uint64_t dempty[2];             // (even CTA) both CTAs have read it
    uint64_t drained;
    uint32_t tmem_base;
    int abort;
    int units;
    int chunk;                      // stages between drains of an accumulator
    // then bound[experts + 1], tiles[experts + 1], tails[experts + 1]
};

template <int T>
struct PairCfg {
    static constexpr int kXBytes = T / 2 * kI8StageK * 2;  // this CTA's half of the tokens, FP16
    static constexpr int kBStages = T == 256 ? 5 : 6, kXSlots = T == 256 ? 2 : 3;
    static constexpr int kFixed = 1024 + kBStages * kBBytes + kXSlots * 2 * kXBytes + static_cast<int>(sizeof(PairShared));
    static constexpr int smem(int experts) { return kFixed + 3 * 4 * (experts + 1); }
    // Registers a thread of each warpgroup: control, conversion, two epilogue
    // warpgroups (T / 2 sums a thread).  Their sum stays within 4 x 128, what the
    // block is launched with.
    static constexpr int kRegsControl = 56, kRegsConvert = 96, kRegsEpilogue = 176;
    static_assert(kRegsControl + kRegsConvert + 2 * kRegsEpilogue <= 4 * 128, "register split");
    static_assert(T + kPairASlots * 2 * kACols <= static_cast<int>(kPairTmemCols), "tensor memory");
    static_assert(smem(kMaxExperts) <= kSmemLimit && kBStages <= kPairMaxB && kXSlots <= kPairMaxX, "shared memory");
};

template <int T>
__global__ void __launch_bounds__(kPairThreads, 1)
int8_tc_pair_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA, const Int8Args a) {
    using Cf = PairCfg<T>;
    constexpr int SB = Cf::kBStages, SX = Cf::kXSlots;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;  // the same in both CTAs
    uint8_t *ring_x = smem_raw + pad, *ring_b = ring_x + SX * 2 * Cf::kXBytes;
    PairShared *sh = reinterpret_cast<PairShared *>(ring_b + SB * kBBytes);
    int *bound = reinterpret_cast<int *>(sh + 1), *tiles = bound + a.experts + 1, *tails = tiles + a.experts + 1;
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
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sh->xfull[h][s], 1);
                mbar_init(&sh->xempty[h][s], 1);
            }
        }
        for (int s = 0; s < kPairASlots; ++s) {
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
        tc::tmem_alloc_pair(&sh->tmem_base, kPairTmemCols);
        tc::tmem_relinquish_pair();
    }
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 2) {
        const int n = sum_tiles<true>(bound, tiles, tails, a, T, lane);
        if (lane == 0) sh->units = n * ch_tiles;
    }
    if (warp == 3) {
        const int c = chunk_of(a, lane);
        if (lane == 0) sh->chunk = c;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync_all();  // both CTAs' barriers are initialised before any cross-CTA arrive
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
    const uint32_t tmem_a = tmem + T;
    volatile int *abort_flag = &sh->abort;
    const int units = sh->units, chunk_stages = sh->chunk;
    // A tile of up to T / 2 tokens (the last of an expert) leaves half 1 out.
    auto halves_of = [](const I8Unit &q) { return q.tend - q.t0 > T / 2 ? 2 : 1; };
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (mbar_wait(bar, parity, a.status)) return true;
        *abort_flag = 1;
        return false;
    };

    if (warp < 4) {
        regs_fewer<Cf::kRegsControl>();
        if (warp == 0) {
            // -------------------------------------------- TMA producer of B
            Ring r;
            int issued = 0;
            bool ok = true;
            if (lane == 0) {
                for (int u = first_unit; u < units && ok; u += unit_step) {
                    const I8Unit q = unit_of<T, kPairN, true>(bound, tiles, tails, a, ch_tiles, u);
                    for (int i = 0; i < kt; ++i, r.step(SB), ++issued) {
                        if (!wait(&sh->bempty[r.s], r.round ^ 1u)) { ok = false; break; }
                        mbar_arrive_expect_tx(&sh->bfull[r.s], kBBytes);
                        tma_load_3d(ring_b + r.s * kBBytes, &tmB, &sh->bfull[r.s], i * kI8StageK, q.ch0 + rank * kI8TileN,
                                    q.e);
                    }
                }
                // no copy outlives the CTA
                for (int t = max(0, issued - SB); t < issued; ++t) mbar_wait(&sh->bfull[t % SB], (t / SB) & 1, a.status);
            }
            __syncwarp();
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------- MMA issuer (even CTA)
            constexpr uint32_t idesc = tc::idesc_f16_kmajor(2 * kI8TileN, T / 2);
            const uint64_t xdesc = tc::smem_desc(smem_u32(ring_x), 16, 1024, tc::kLayoutSwizzle128);
            Ring xr[2], tr;          // each half of the tokens goes round a ring of its own
            uint32_t round[2] = {};  // of the half accumulators
            bool ok = true;
            for (int u = first_unit; u < units && ok; u += unit_step) {
                const int halves = halves_of(unit_of<T, kPairN, true>(bound, tiles, tails, a, ch_tiles, u));
                // A slot of two stages at a time: both for half 0 of the accumulators,
                // then both for half 1, so that at the end of `chunk` stages either
                // half has the time of 16 MMAs (1024 cycles) to be drained in while
                // the other is added to.
                int run = 0;  // stages in the accumulators so far
                for (int i = 0; i < kt; i += 2) {
                    const int two = i + 1 < kt ? 2 : 1;
                    const bool start = run == 0, end = i + two == kt || run + two == chunk_stages;
                    ok = wait(&sh->afull[tr.s], tr.round);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h >= halves) break;
                        const int x = xr[h].s;
                        ok = ok && (!start || wait(&sh->dempty[h], round[h] ^ 1u)) && wait(&sh->xfull[h][x], xr[h].round);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc::fence_after_sync();
                        if (tc::elect_one()) {
                            const uint64_t b = xdesc + static_cast<uint64_t>(x * (2 * Cf::kXBytes / 16) + h * (T / 4 * 128 / 16));
                            const uint32_t ta = tmem_a + tr.s * (2 * kACols);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                if (j >= two) break;
#pragma unroll
                                for (int kk = 0; kk < kI8StageK / 16; ++kk)
                                    tc::mma_f16_ta_pair(tmem + h * (T / 2), ta + j * kACols + kk * 8,
                                                        b + (j * Cf::kXBytes + (kk / 4) * (T / 2 * 128) + (kk % 4) * 32) / 16,
                                                        idesc, (start && j == 0 && kk == 0) ? 0u : 1u);
                            }
                            tc::commit_pair(&sh->xempty[h][x], 0x3);
                            if (h + 1 == halves) tc::commit_pair(&sh->aempty[tr.s], 0x3);
                            if (end) tc::commit_pair(&sh->dfull[h], 0x3);
                        }
                        __syncwarp();
                        xr[h].step(SX);
                    }
                    if (!ok) break;
                    tr.step(kPairASlots);
                    run = end ? 0 : run + two;
                    if (end) {
                        round[0] ^= 1u;
                        if (halves == 2) round[1] ^= 1u;
                    }
                }
            }
            if (!ok && tc::elect_one()) {  // no teardown under a running MMA
                tc::commit_pair(&sh->drained, 0x1);
                mbar_wait(&sh->drained, 0, a.status);
            }
            __syncwarp();
        } else if (warp == 2) {
            // -------------------------------------------- TMA producer of the tokens
            // Half h of the accumulators covers T / 2 tokens from t0 + h T / 2, half of
            // them from each CTA: this CTA's rows h T / 4 .. of a stage.  Both
            // CTAs' bytes count on the even CTA's barrier.
            // They are fetched in the MMAs' order: half 0 of two stages, then half 1.
            Ring r[2];
            bool ok = true;
            if (lane == 0) {
                const uint32_t xfull = tc::map_shared_rank(smem_u32(&sh->xfull[0][0]), 0);
                for (int u = first_unit; u < units && ok; u += unit_step) {
                    const I8Unit q = unit_of<T, kPairN, true>(bound, tiles, tails, a, ch_tiles, u);
                    const int row = q.t0 - a.row0 + rank * (T / 4), halves = halves_of(q);
                    for (int i = 0; i < kt && ok; i += 2) {
                        const int two = i + 1 < kt ? 2 : 1;
                        for (int h = 0; h < halves; ++h) {
                            const int x = r[h].s;
                            ok = ok && wait(&sh->xempty[h][x], r[h].round ^ 1u);
                            if (!ok) break;
                            uint8_t *st = ring_x + x * (2 * Cf::kXBytes) + h * (T / 4 * 128);
                            if (rank == 0) mbar_arrive_expect_tx(&sh->xfull[h][x], two * Cf::kXBytes);
                            for (int j = 0; j < two; ++j)
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    tc::tma_load_2d_pair(st + j * Cf::kXBytes + k * (T / 2 * 128), &tmA,
                                                         xfull + (h * kPairMaxX + x) * 8, (i + j) * kI8StageK + k * 64,
                                                         row + h * (T / 2));
                            r[h].step(SX);
                        }
                    }
                }
                // No copy outlives its CTA: the MMAs that read the last ones have
                // finished (a slot that was never loaded stands at its first round).
                for (int h = 0; h < 2; ++h)
                    for (int x = 0; x < SX; ++x, r[h].step(SX)) mbar_wait(&sh->xempty[h][r[h].s], r[h].round ^ 1u, a.status);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        // ------------------------------------------------ B to FP16, into tensor memory
        regs_fewer<Cf::kRegsConvert>();
        const int row = (warp % 4) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        const uint32_t afull = tc::map_shared_rank(smem_u32(&sh->afull[0]), 0);
        Ring r, t;
        int stored = -1;  // the slot in tensor memory whose stores have not been waited for
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
            for (int i = 0; i < kt && ok; i += 2) {
                const int two = i + 1 < kt ? 2 : 1;
                for (int j = 0; j < two; ++j, r.step(SB)) {
                    if (!__all_sync(0xffffffffu, mbar_try_wait(&sh->bfull[r.s], r.round))) {
                        flush();
                        ok = __all_sync(0xffffffffu, wait(&sh->bfull[r.s], r.round));
                        if (!ok) break;
                    }
                    const uint8_t *src = ring_b + r.s * kBBytes + row * kI8StageK;
                    uint4 w[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) w[c] = *reinterpret_cast<const uint4 *>(src + ((c ^ (row & 7)) * 16));
                    if (j == 0) {
                        flush();
                        ok = __all_sync(0xffffffffu, wait(&sh->aempty[t.s], t.round ^ 1u));
                        if (!ok) break;
                        tc::fence_after_sync();
                    }
                    expand_to_tmem(w, tmem_a + t.s * (2 * kACols) + j * kACols + lanes);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->bempty[r.s]);
                }
                stored = t.s;
                t.step(kPairASlots);
            }
            flush();
        }
    } else {
        // ------------------------------------------------ accumulators to C: warpgroup h reads half h
        regs_more<Cf::kRegsEpilogue>();
        constexpr int kCols = T / 2;
        const int h = (warp - 8) / 4;
        const int ch = (warp % 4) * 32 + lane;
        const uint32_t src = tmem + h * kCols + (static_cast<uint32_t>(warp % 4 * 32) << 16);
        const uint32_t dempty = tc::map_shared_rank(smem_u32(&sh->dempty[h]), 0);
        uint32_t round = 0;
        bool ok = true;
        for (int u = first_unit; u < units && ok; u += unit_step) {
            const I8Unit q = unit_of<T, kPairN, true>(bound, tiles, tails, a, ch_tiles, u);
            if (h >= halves_of(q)) continue;
            const int n = q.ch0 + rank * kI8TileN + ch;
            const long long at = static_cast<long long>(q.e) * a.N + n;
            const float sb = n < a.N ? __ldcg(a.scaleB + at) : 0.f;
            const float bias = n < a.N && a.bias ? __ldcg(a.bias + at) : 0.f;
            const int first = q.t0 + h * kCols;
            float sa[kCols / 32];
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c)
                sa[c] = first + c * 32 + lane < q.tend ? __ldcg(a.scaleA + first + c * 32 + lane) : 0.f;
            int acc[kCols];
            auto take = [&](auto how) {
                ok = __all_sync(0xffffffffu, wait(&sh->dfull[h], round));
                if (!ok) return;
                tc::fence_after_sync();
                drain<decltype(how)::value>(src, acc);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_remote(dempty);
                round ^= 1u;
            };
            auto write = [&](auto floats) {
                with_out_type(a.out_type, [&](auto out) {
                    using Out = decltype(out);
                    write_columns<Out, decltype(floats)::value>(
                        static_cast<typename Out::T *>(a.C) + static_cast<long long>(first) * a.ldc + n, a.ldc,
                        n < a.N ? q.tend - first : 0, acc, sa, sb, bias);
                });
            };
            if (kt <= chunk_stages) {
                take(std::integral_constant<Take, Take::kOnly>{});
                if (ok) write(std::true_type{});
            } else {
#pragma unroll
                for (int j = 0; j < kCols; ++j) acc[j] = 0;
                for (int i = 0; i < kt && ok; i += chunk_stages) take(std::integral_constant<Take, Take::kAdd>{});
                if (ok) write(std::false_type{});
            }
        }
    }
    // ---------------------------------------------------- teardown
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync_all();  // the peer is done with this CTA's barriers and tensor memory
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(tmem, kPairTmemCols);
    }
}

template <int NT, bool SPLIT>
cudaError_t launch_split(const Int8Args &a, const CUtensorMap &tmB, const CUtensorMap &tmA, int num_sms,
                         int smem_override, cudaStream_t stream) {
    using Cf = DirectCfg<NT, SPLIT>;
    const int ch_tiles = (a.N + kI8TileN - 1) / kI8TileN, splits = SPLIT ? a.ksplit : 1;
    const long long units = int8_most_tiles(a.rows, a.experts, NT) * ch_tiles, most = 2 * num_sms / splits;
    return launch_dependent(int8_tc_kernel<NT, SPLIT>,
                            dim3(static_cast<unsigned>(splits * (units < most ? units : most))), dim3(kDirectThreads),
                            smem_override > 0 ? smem_override : Cf::smem(a.experts), stream, splits, tmB, tmA, a);
}

template <int NT>
cudaError_t launch_direct(const Int8Args &a, const CUtensorMap &tmB, const CUtensorMap &tmA, int num_sms,
                          int smem_override, cudaStream_t stream) {
    return a.ksplit > 1 ? launch_split<NT, true>(a, tmB, tmA, num_sms, smem_override, stream)
                        : launch_split<NT, false>(a, tmB, tmA, num_sms, smem_override, stream);
}

template <int T>
cudaError_t launch_pair(const Int8Args &a, const CUtensorMap &tmB, const CUtensorMap &tmA, int num_sms,
                        int smem_override, cudaStream_t stream) {
    const int ch_tiles = (a.N + kPairN - 1) / kPairN;
    const long long units = int8_most_tiles(a.rows, a.experts, T) * ch_tiles, most = num_sms / 2;
    return launch_dependent(int8_tc_pair_kernel<T>, dim3(static_cast<unsigned>(2 * (units < most ? units : most))),
                            dim3(kPairThreads), smem_override > 0 ? smem_override : PairCfg<T>::smem(a.experts), stream,
                            2, tmB, tmA, a);
}

template <int NT>
cudaError_t prepare_direct() {
    const cudaError_t e = cudaFuncSetAttribute(int8_tc_kernel<NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               DirectCfg<NT, false>::smem(kMaxExperts));
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(int8_tc_kernel<NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   DirectCfg<NT, true>::smem(kMaxExperts));
}

template <int T>
cudaError_t prepare_pair() {
    return cudaFuncSetAttribute(int8_tc_pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                PairCfg<T>::smem(kMaxExperts));
}

}  // namespace

cudaError_t int8_prepare() {
    cudaError_t e = cudaSuccess;
    for (cudaError_t r : {prepare_direct<16>(), prepare_direct<32>(), prepare_direct<64>(), prepare_pair<128>(),
                          prepare_pair<256>()})
        if (e == cudaSuccess) e = r;
    for (auto *k : {int8_few_kernel<1, false>, int8_few_kernel<1, true>, int8_few_kernel<2, false>,
                    int8_few_kernel<2, true>, int8_few_kernel<4, false>, int8_few_kernel<4, true>,
                    int8_few_kernel<8, false>, int8_few_kernel<8, true>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kI8FewBytes);
    return e;
}

cudaError_t launch_int8_tc(const Int8Args &a, const CUtensorMap &tmB, const CUtensorMap &tmA, int num_sms,
                           int smem_override, cudaStream_t stream) {
    switch (a.nt) {
        case 16: return launch_direct<16>(a, tmB, tmA, num_sms, smem_override, stream);
        case 32: return launch_direct<32>(a, tmB, tmA, num_sms, smem_override, stream);
        case 64: return launch_direct<64>(a, tmB, tmA, num_sms, smem_override, stream);
        case 128: return launch_pair<128>(a, tmB, tmA, num_sms, smem_override, stream);
        default: return launch_pair<256>(a, tmB, tmA, num_sms, smem_override, stream);
    }
}

template <int MT>
static cudaError_t launch_few(const Int8Args &a, int num_sms, cudaStream_t stream) {
    const bool vec = reinterpret_cast<uintptr_t>(a.B) % 16 == 0 && a.ldb % 16 == 0;
    const int a_vec = reinterpret_cast<uintptr_t>(a.A) % 16 == 0 && a.lda % 16 == 0;
    const int pieces = (a.K + 15) / 16, steps = (pieces + 31) / 32;
    // warps share a channel's K range while that leaves each of them a step and
    // all CTAs run at once (32 warps an SM)
    constexpr int C = kFewC;
    int split = 1;
    const long long warps = (static_cast<long long>(a.N) + C - 1) / C;
    while (split < kFewThreads / 32 && steps >= 2 * split && warps * split * 2 <= 32ll * num_sms) split *= 2;
    const int per = kFewThreads / 32 / split * C;
    return launch_dependent(vec ? int8_few_kernel<MT, true> : int8_few_kernel<MT, false>,
                            dim3((a.N + per - 1) / per), dim3(kFewThreads), MT * pieces * 16, stream, 1, a, split, a_vec);
}

cudaError_t launch_int8_few(const Int8Args &a, int num_sms, cudaStream_t stream) {
    if (a.rows <= 1) return launch_few<1>(a, num_sms, stream);
    if (a.rows <= 2) return launch_few<2>(a, num_sms, stream);
    if (a.rows <= 4) return launch_few<4>(a, num_sms, stream);
    return launch_few<8>(a, num_sms, stream);
}

cudaError_t launch_int8_generic(const Int8Args &a, cudaStream_t stream) {
    const int y = (a.rows + kGTile - 1) / kGTile;
    const dim3 grid((a.N + kGTile - 1) / kGTile, y < 65535 ? y : 65535, a.experts);
    return launch_dependent(int8_generic_kernel, grid, dim3(256), 0, stream, 1, a);
}

cudaError_t launch_int8_copies(Int8Copies *c, cudaStream_t stream) {
    c->a_vec = reinterpret_cast<uintptr_t>(c->A) % 16 == 0 && c->lda % 16 == 0;
    const bool words = reinterpret_cast<uintptr_t>(c->B) % 4 == 0 && c->ldb % 4 == 0 && c->strideB % 4 == 0;
    auto capped = [](long long blocks) { return static_cast<int>(blocks < kI8Peaks ? blocks : kI8Peaks); };
    c->a_blocks = !c->a_dst ? 0
                  : c->peaks ? capped((static_cast<long long>(c->a_rows) * (c->a_ld / 16) + 255) / 256)
                             : capped(realign_blocks(c->a_rows, c->a_ld));
    if (!c->b_dst) c->b_blocks = 0;
    else if (c->b_trans) c->b_blocks = capped(realign_blocks(static_cast<long long>(c->experts) * c->N, c->b_ld));
    else c->b_blocks = capped(static_cast<long long>(c->experts) * ((c->b_ld + kTK - 1) / kTK) * ((c->N + kTN - 1) / kTN));
    return launch_dependent(words ? int8_copies_kernel<true> : int8_copies_kernel<false>, dim3(c->a_blocks + c->b_blocks),
                            dim3(256), 0, stream, 1, *c);
}

}  // namespace sg
