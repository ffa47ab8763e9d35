// Rows to 8-bit integers, and rows sorted by expert and back, for sm_103a.
//
//  * quantize_kernel -- per row i of X (FP32, BF16 or FP16): with m = max_p
//    |x_ip|, scale_i = m / 127 and q_ip = rint(x_ip * (127 / m)) (both
//    quotients, the product and the rounding correctly rounded, ties to even),
//    an int8 in [-127, 127] by construction.  The row may go to several
//    destinations (dispatch): it is read and quantized once, written
//    `choices` times.  One pass over HBM: a row stays in the registers of the
//    TPR threads that share it (up to 4 x 8 elements a thread; longer rows are
//    read a second time, from L2).  8192 x 8192 BF16: 31 us, 6.5 TB/s (with a
//    branch for the end of a row around each load, and so one load in flight at a
//    time, 58 us).
//  * sort_kernel -- the (token, choice) slots in a stable order by expert: a
//    counting sort.  Within a warp the 32 slots of one step that name the same
//    expert find one another by ballots and take consecutive places, which
//    stay in registers; every warp keeps its own counts in shared memory, whose
//    exclusive sums over the warps (and, with several CTAs, over the CTAs before)
//    place each slot.
//    Integers only and no atomic whose order matters: the same order every time.
//    32768 slots over 64 experts: 6.9 us, of which two launches are about 5.5;
//    2048 slots and fewer take one CTA and one launch (2.7 us).
//  * move_kernel, gather_kernel, combine_grad_kernel -- the rows' way to the
//    experts, back, and the gradients; each reads and writes every row once
//    (16 bytes a thread and step where alignment allows), sums in FP32 in
//    ascending choice order and rounds once.  8192 tokens, 4 choices, 4096 elements
//    of 16 bits: 51.6 us out (6.5 TB/s), 54.6 back (6.1), the weighted gradient 88
//    (6.8).  Rows of an odd number of 16-bit elements take 2-byte accesses and up to
//    twice as long a byte (2475 elements: 45, 60 and 89 us).  Put together instead from
//    aligned 16-byte pieces of their rows by shuffles, with the stores on 16-byte
//    boundaries, they took still longer (5453 rows of 3515 59 us instead of 23): the
//    shifts' instructions then bound them.
// No load is a read-only-cache load (ld.global.nc): what is read may have been
// written by the kernel before, whose end the launch overlaps.  Rows, read once, go
// past L1 (ld.global.cg); row numbers and weights, which a block's warps share, do
// not (ld.global.ca; past L1 the gathers take 61 us instead of 55).
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "internal.h"
#include "sgemm.h"

namespace sg {
namespace {

// ---- element types -----------------------------------------------------------
// Eight consecutive elements of a row as FP32, and back (rounded to nearest even).
struct ElF32 {
    using T = float;
    static __device__ __forceinline__ float up(T x) { return x; }
    static __device__ __forceinline__ T down(float x) { return x; }
};
struct ElBF16 {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float up(T x) { return __bfloat162float(x); }
    static __device__ __forceinline__ T down(float x) { return __float2bfloat16_rn(x); }
};
struct ElF16 {
    using T = __half;
    static __device__ __forceinline__ float up(T x) { return __half2float(x); }
    static __device__ __forceinline__ T down(float x) { return __float2half_rn(x); }
};

constexpr int kV = 8;  // elements a thread takes per step

template <class T>
struct alignas(16) Pack8 {
    T v[kV];
};

// Piece c of a row of `width` elements that `TPR` threads share: 8 elements a
// thread, in accesses of A consecutive elements (up to 16 bytes; rows start on
// such boundaries and divide into them) that are TPR * A elements apart, so that
// a warp's loads and stores are contiguous.  One layout for loads and stores,
// and no branch between the loads of several pieces: they are all in flight
// together.
template <int BYTES>
struct AccessOf;
template <>
struct AccessOf<2> { using T = uint16_t; };
template <>
struct AccessOf<4> { using T = uint32_t; };
template <>
struct AccessOf<8> { using T = uint2; };
template <>
struct AccessOf<16> { using T = uint4; };

template <class T, int TPR, int A>
__device__ __forceinline__ Pack8<T> load8(const T *row, int c, int lane, int width) {
    using W = typename AccessOf<static_cast<int>(sizeof(T)) * A>::T;
    Pack8<T> r;
    const int at = c * kV * TPR + lane * A;
    const W *p = reinterpret_cast<const W *>(row + at);
    W *d = reinterpret_cast<W *>(&r);
#pragma unroll
    for (int i = 0; i < kV / A; ++i) d[i] = at + i * TPR * A < width ? __ldcg(p + i * TPR) : W{};
    return r;
}
template <class T, int TPR, int A>
__device__ __forceinline__ void store8(T *row, int c, int lane, int width, const Pack8<T> &r) {
    using W = typename AccessOf<static_cast<int>(sizeof(T)) * A>::T;
    const int at = c * kV * TPR + lane * A;
    W *p = reinterpret_cast<W *>(row + at);
    const W *s = reinterpret_cast<const W *>(&r);
#pragma unroll
    for (int i = 0; i < kV / A; ++i)
        if (at + i * TPR * A < width) p[i * TPR] = s[i];
}

// (Tokens, rows and choices are counted in unsigned integers where a step may go past
// the last one: there may be 2^31 - 1 of them.)

// Sorted row of a slot, or -1 for one that has none: a value outside [0, slots)
// is no row, whatever wrote it.
__device__ __forceinline__ int row_of(const int *rows, long long slot, int slots) {
    const int r = __ldca(rows + slot);
    return static_cast<unsigned>(r) < static_cast<unsigned>(slots) ? r : -1;
}

// ---- quantization -------------------------------------------------------------
// Below this row maximum 127 / m overflows or the scale loses bits: the row is
// stored as zeros with scale 0.
constexpr float kSmallestMax = 127.f * 1.17549435e-38f;

// 1.5 * 2^23: adding it rounds a value of magnitude < 2^22 to an integer (ties
// to even) that sits in the low bits of the sum.
constexpr float kRoundMagic = 12582912.f;

// 256-thread CTAs that an SM has to hold: five of four 16-bit pieces a thread (8192 x
// 4096 17.7 us, four 18.7), four of 32-bit ones (25.4; five 32.2, the pieces no longer
// fit the registers).
template <class T>
constexpr int quantize_ctas(int held) { return held == 1 ? 6 : sizeof(T) == 2 ? 5 : 4; }

template <class El, int TPR, int A, int HELD>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR < 512 ? quantize_ctas<typename El::T>(HELD) : HELD == 1 ? 3 : 2)
quantize_kernel(const typename El::T *__restrict__ X, long long ldx, int M, int K, int8_t *__restrict__ Q,
                long long ldq, float *__restrict__ scale, const int *__restrict__ rows, int choices) {
    using T = typename El::T;
    constexpr int kThreads = TPR < 256 ? 256 : TPR;
    constexpr int kRows = kThreads / TPR, kHeld = HELD;  // pieces in registers
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % TPR;
    const unsigned i = blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = i < static_cast<unsigned>(M);
    const T *x = X + static_cast<long long>(live ? i : 0) * ldx;
    const int width = live ? K : 0;

    Pack8<T> held[kHeld];
#pragma unroll
    for (int c = 0; c < kHeld; ++c) held[c] = load8<T, TPR, A>(x, c, lane, width);
    unsigned top = 0;  // max of |x| as bits: NaN above infinity above every number
#pragma unroll
    for (int c = 0; c < kHeld; ++c)
#pragma unroll
        for (int e = 0; e < kV; ++e) top = max(top, __float_as_uint(El::up(held[c].v[e])) & 0x7fffffffu);
    for (int c = kHeld; c * kV * TPR < width; ++c) {
        const Pack8<T> h = load8<T, TPR, A>(x, c, lane, width);
#pragma unroll
        for (int e = 0; e < kV; ++e) top = max(top, __float_as_uint(El::up(h.v[e])) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (TPR > 32) {
        __shared__ unsigned part[kThreads / 32];
        if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = top;
        __syncthreads();
        const int w0 = threadIdx.x / TPR * (TPR / 32);
        top = 0;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) top = max(top, part[w0 + w]);
    }
    if (!live) return;

    const float m = __uint_as_float(top);
    const bool finite = top < 0x7f800000u;
    const bool zero = !finite || m < kSmallestMax;
    const float inv = zero ? 0.f : __fdiv_rn(127.f, m);
    const float s = !finite ? __uint_as_float(0x7fc00000u) : zero ? 0.f : __fdiv_rn(m, 127.f);
    const unsigned keep = zero ? 0u : 0xffffffffu;

    auto quantized = [&](const Pack8<T> &h) {
        unsigned b[kV];
#pragma unroll
        for (int e = 0; e < kV; ++e)
            b[e] = __float_as_uint(__fadd_rn(__fmul_rn(El::up(h.v[e]), inv), kRoundMagic));
        uint2 w;
        w.x = keep & __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        w.y = keep & __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
        return w;
    };
    // the quantized bytes in the accesses' layout: A at a time
    auto put = [&](int8_t *q, int c, uint2 w) {
        const int at = c * kV * TPR + lane * A;
#pragma unroll
        for (int i = 0; i < kV / A; ++i) {
            if (at + i * TPR * A >= K) continue;
            int8_t *p = q + at + i * TPR * A;
            const uint32_t word = i * A < 4 ? w.x >> (8 * (i * A % 4)) : w.y >> (8 * (i * A % 4));
            if (A == 8) *reinterpret_cast<uint2 *>(p) = w;
            else if (A == 4) *reinterpret_cast<uint32_t *>(p) = word;
            else if (A == 2) *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(word);
            else *p = static_cast<int8_t>(word);
        }
    };
    uint2 packed[kHeld];
#pragma unroll
    for (int c = 0; c < kHeld; ++c) packed[c] = quantized(held[c]);
    for (int j = 0; j < choices; ++j) {
        const int r = rows ? row_of(rows, static_cast<long long>(i) * choices + j, M * choices) : static_cast<int>(i);
        if (r < 0) continue;
        int8_t *q = Q + static_cast<long long>(r) * ldq;
#pragma unroll
        for (int c = 0; c < kHeld; ++c) put(q, c, packed[c]);
        for (int c = kHeld; c * kV * TPR < K; ++c) put(q, c, quantized(load8<T, TPR, A>(x, c, lane, K)));
        if (lane == 0) scale[r] = s;
    }
}

// Blocks of `per` of n > 0 rows (n up to 2^31 - 1).
constexpr unsigned blocks_of(int n, int per) { return static_cast<unsigned>((n - 1) / per + 1); }

template <class El, int A>
cudaError_t quantize_typed(const MoveArgs &a, int num_sms, cudaStream_t stream) {
    using T = typename El::T;
    const T *X = static_cast<const T *>(a.X);
    int8_t *Q = static_cast<int8_t *>(a.Y);
    // Threads a row: enough that it stays in registers (32 elements a thread),
    // and, with too few rows to fill the GPU, more of them so that each thread
    // loads less.  Rows of at most eight elements a thread take a kernel without the
    // other three pieces' loads and stores (16 x 4096 BF16 2.1 us in a graph instead
    // of 2.7, 7900 x 45 3.0 instead of 5.8).
    const bool few = a.tokens <= 4 * num_sms;
    const int per = few ? kV : 4 * kV;
    const int want = (a.width + per - 1) / per;
    const int share = want <= 32 ? 32 : want <= 64 ? 64 : want <= 128 ? 128 : want <= 256 ? 256 : 512;
    const bool one = a.width <= kV * share;
#define SG_QUANT(TPR)                                                                                            \
    return launch_dependent(one ? quantize_kernel<El, TPR, A, 1> : quantize_kernel<El, TPR, A, 4>,             \
                            dim3(blocks_of(a.tokens, TPR < 256 ? 256 / TPR : 1)),                               \
                            dim3(TPR < 256 ? 256 : TPR), 0, stream, 1, X, a.ldx, a.tokens, a.width, Q, a.ldy,    \
                            a.scale, a.rows, a.choices)
    if (share == 32) SG_QUANT(32);
    if (share == 64) SG_QUANT(64);
    if (share == 128) SG_QUANT(128);
    if (share == 256) SG_QUANT(256);
    SG_QUANT(512);
#undef SG_QUANT
}

// ---- sort ---------------------------------------------------------------------
// A CTA takes STEPS * 1024 slots, its 32 warps runs of STEPS * 32.  Shared memory:
// 32 * E counts of the warps, E places of the CTA.
// PASS 0: one CTA does it all.  PASS 1: each CTA writes the counts of its own
// slots to hist[cta][E].  PASS 2: each CTA places its slots.
constexpr int kSortWarps = 32, kSortThreads = kSortWarps * 32;

// The lanes whose key agrees with this lane's in its lowest `bits` bits: a ballot a
// bit (7 for 64 experts; match.any takes about as long for every distinct key).
__device__ __forceinline__ unsigned same_key(int key, int bits) {
    unsigned same = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const unsigned v = __ballot_sync(0xffffffffu, (key >> b) & 1);
        same &= (key >> b) & 1 ? v : ~v;
    }
    return same;
}

template <int PASS, int STEPS>
__global__ void __launch_bounds__(kSortThreads)
sort_kernel(const int *__restrict__ ids, int slots, int experts, int *__restrict__ offsets, int *__restrict__ rows,
            int *__restrict__ source, int *__restrict__ hist) {
    extern __shared__ int sh[];
    int *counts = sh, *place = sh + kSortWarps * experts;
    __shared__ int carry[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned below = (1u << lane) - 1u;
    const int bits = 33 - __clz(experts - 1);  // of 0 .. experts - 1 and of -1, told apart by one bit more
    for (int e = tid; e < kSortWarps * experts; e += kSortThreads) counts[e] = 0;
    griddep_wait();
    griddep_launch_dependents();
    const long long first = (static_cast<long long>(blockIdx.x) * kSortWarps + warp) * (STEPS * 32) + lane;
    int e[STEPS], rank[STEPS];  // the slots' experts (-1: dropped), their places among the warp's
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        e[s] = first + s * 32 < slots ? __ldcg(ids + first + s * 32) : -1;
        if (static_cast<unsigned>(e[s]) >= static_cast<unsigned>(experts)) e[s] = -1;
    }
    __syncthreads();
    int *mine = counts + warp * experts;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const unsigned same = same_key(e[s], bits);
        rank[s] = (e[s] >= 0 ? mine[e[s]] : 0) + __popc(same & below);
        __syncwarp();
        if (e[s] >= 0 && (same & below) == 0) mine[e[s]] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // counts -> exclusive sums over the warps; place[x] = the CTA's slots of expert x
    for (int x = tid; x < experts; x += kSortThreads) {
        int n = 0;
#pragma unroll
        for (int w0 = 0; w0 < kSortWarps; w0 += 16) {
            int c[16];
#pragma unroll
            for (int w = 0; w < 16; ++w) c[w] = counts[(w0 + w) * experts + x];
#pragma unroll
            for (int w = 0; w < 16; ++w) {
                counts[(w0 + w) * experts + x] = n;
                n += c[w];
            }
        }
        if (PASS == 1) hist[static_cast<long long>(blockIdx.x) * experts + x] = n;
        place[x] = n;
    }
    if (PASS == 1) return;
    __syncthreads();
    // the slots of every expert, their exclusive sum over the experts (offsets),
    // and those of the CTAs before (at most kMaxExperts experts: one each)
    const int ctas = static_cast<int>(gridDim.x);
    int total = 0, before = 0;
    if (tid < experts) {
        if (PASS == 0) {
            total = place[tid];
        } else {
            for (int c0 = 0; c0 < ctas; c0 += 8) {
                int n[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    n[c] = c0 + c < ctas ? __ldcg(hist + static_cast<long long>(c0 + c) * experts + tid) : 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    total += n[c];
                    if (c0 + c < static_cast<int>(blockIdx.x)) before += n[c];
                }
            }
        }
    }
    int sum = total;  // inclusive over the warp
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
    }
    if (lane == 31) carry[warp] = sum;
    __syncthreads();
    int all = carry[lane];  // of warp `lane`; then inclusive over the warps
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, all, d);
        if (lane >= d) all += up;
    }
    const int kept = __shfl_sync(0xffffffffu, all, 31);
    const int lower = warp > 0 ? __shfl_sync(0xffffffffu, all, warp - 1) : 0;
    if (tid < experts) {
        place[tid] = lower + sum - total + before;
        if (blockIdx.x == 0) offsets[tid] = lower + sum - total;
    }
    if (blockIdx.x == 0 && tid == 0) offsets[experts] = kept;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const long long slot = first + s * 32;
        if (slot >= slots) continue;
        const int r = e[s] >= 0 ? place[e[s]] + mine[e[s]] + rank[s] : -1;
        rows[slot] = r;
        if (r >= 0) source[r] = static_cast<int>(slot);
        if (slot >= kept) source[slot] = -1;  // rows past the last expert's hold no slot
    }
}

// ---- rows to the experts --------------------------------------------------------
// Row t of X to rows[t * choices + j] of Y: read once, written up to `choices`
// times.  PER threads a row, four units (the widest that the rows' alignment
// allows, up to 16 bytes; eight of 2 bytes) each, all loaded before the first store.
template <class Unit>
constexpr int kMovesOf = sizeof(Unit) == 2 ? 8 : 4;

template <class Unit, int PER>
__global__ void __launch_bounds__(256)
move_kernel(const Unit *__restrict__ X, long long ldx, int tokens, int choices, int width, const int *__restrict__ rows,
            Unit *__restrict__ Y, long long ldy) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kMoves = kMovesOf<Unit>;
    const int slots = tokens * choices;
    const int c0 = blockIdx.x * (PER * kMoves) + threadIdx.x % PER;
    for (unsigned t = blockIdx.y * (256 / PER) + threadIdx.x / PER; t < static_cast<unsigned>(tokens);
         t += gridDim.y * (256 / PER)) {
        const Unit *x = X + static_cast<long long>(t) * ldx;
        Unit v[kMoves];
#pragma unroll
        for (int m = 0; m < kMoves; ++m) v[m] = c0 + m * PER < width ? __ldcg(x + c0 + m * PER) : Unit{};
        for (int j = 0; j < choices; ++j) {
            const int r = row_of(rows, static_cast<long long>(t) * choices + j, slots);
            if (r < 0) continue;
            Unit *y = Y + static_cast<long long>(r) * ldy;
#pragma unroll
            for (int m = 0; m < kMoves; ++m)
                if (c0 + m * PER < width) y[c0 + m * PER] = v[m];
        }
    }
}

// ---- rows from the experts ------------------------------------------------------
// out[t] = sum_j w[t,j] * Y[rows[t,j]] (w NULL: the plain sum); J rows' loads in
// flight at a time, TPR threads a token.
template <class El, int J, int TPR, int A>
__global__ void __launch_bounds__(256)
gather_kernel(const typename El::T *__restrict__ Y, long long ldy, int tokens, int choices, int width,
              const int *__restrict__ rows, const float *__restrict__ weights, typename El::T *__restrict__ out,
              long long ldo) {
    using T = typename El::T;
    griddep_wait();
    griddep_launch_dependents();
    const int slots = tokens * choices, c = blockIdx.x, lane = threadIdx.x % TPR;
    for (unsigned t = blockIdx.y * (256 / TPR) + threadIdx.x / TPR; t < static_cast<unsigned>(tokens);
         t += gridDim.y * (256 / TPR)) {
        float sum[kV] = {};
        for (unsigned j0 = 0; j0 < static_cast<unsigned>(choices); j0 += J) {
            Pack8<T> y[J];
            float w[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const long long slot = static_cast<long long>(t) * choices + j0 + j;
                const int r = j0 + j < static_cast<unsigned>(choices) ? row_of(rows, slot, slots) : -1;
                w[j] = r >= 0 && weights ? __ldca(weights + slot) : 1.f;
                // (a row that does not exist has no elements: zeros)
                y[j] = load8<T, TPR, A>(Y + static_cast<long long>(r >= 0 ? r : 0) * ldy, c, lane, r >= 0 ? width : 0);
            }
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < kV; ++e) sum[e] = fmaf(w[j], El::up(y[j].v[e]), sum[e]);
        }
        Pack8<T> o;
#pragma unroll
        for (int e = 0; e < kV; ++e) o.v[e] = El::down(sum[e]);
        store8<T, TPR, A>(out + static_cast<long long>(t) * ldo, c, lane, width, o);
    }
}

// ---- gradient of the weighted return --------------------------------------------
// dY[rows[t,j]] = w[t,j] * dO[t] and dw[t,j] = <dO[t], Y[rows[t,j]]>: TPR
// threads a token (a warp or the block), J choices at a time; the dot products are
// reduced in a fixed order (within the warp, then over the warps).
template <class El, int J, int TPR, int A>
__global__ void __launch_bounds__(256)
combine_grad_kernel(const typename El::T *__restrict__ dO, long long lddo, const typename El::T *__restrict__ Y,
                    long long ldy, int tokens, int choices, int width, const int *__restrict__ rows,
                    const float *__restrict__ weights, typename El::T *__restrict__ dY, long long lddy,
                    float *__restrict__ dw) {
    using T = typename El::T;
    __shared__ float part[8][J];
    griddep_wait();
    griddep_launch_dependents();
    const int slots = tokens * choices, lane = threadIdx.x % TPR;
    const unsigned t = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;  // (with a block a token, the whole block's)
    if (t >= static_cast<unsigned>(tokens)) return;
    const T *g = dO + static_cast<long long>(t) * lddo;
    for (unsigned j0 = 0; j0 < static_cast<unsigned>(choices); j0 += J) {
        int r[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const long long slot = static_cast<long long>(t) * choices + j0 + j;
            r[j] = j0 + j < static_cast<unsigned>(choices) ? row_of(rows, slot, slots) : -1;
            w[j] = r[j] >= 0 ? __ldca(weights + slot) : 0.f;
            dot[j] = 0.f;
        }
        for (int c = 0; c * TPR * kV < width; ++c) {
            const Pack8<T> gv = load8<T, TPR, A>(g, c, lane, width);
            Pack8<T> y[J];
#pragma unroll
            for (int j = 0; j < J; ++j)
                y[j] = load8<T, TPR, A>(Y + static_cast<long long>(r[j] >= 0 ? r[j] : 0) * ldy, c, lane,
                                          r[j] >= 0 ? width : 0);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                Pack8<T> o;
#pragma unroll
                for (int e = 0; e < kV; ++e) {
                    const float d = El::up(gv.v[e]);
                    dot[j] = fmaf(d, El::up(y[j].v[e]), dot[j]);
                    o.v[e] = El::down(w[j] * d);
                }
                if (r[j] >= 0) store8<T, TPR, A>(dY + static_cast<long long>(r[j]) * lddy, c, lane, width, o);
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (r[j] < 0) dot[j] = 0.f;  // not 0 * dO, which a non-finite dO makes NaN
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
            if (TPR > 32 && (threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = dot[j];
            if (TPR == 32 && lane == 0 && j0 + j < static_cast<unsigned>(choices))
                dw[static_cast<long long>(t) * choices + j0 + j] = dot[j];
        }
        if (TPR == 32) continue;
        __syncthreads();
        if (threadIdx.x < J && j0 + threadIdx.x < static_cast<unsigned>(choices)) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += part[k][threadIdx.x];
            dw[static_cast<long long>(t) * choices + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

// The largest power of two, up to 16, that divides every row's start and length in
// bytes.
template <class... Rows>
int common_alignment(Rows... rows) {
    const uintptr_t all = (static_cast<uintptr_t>(rows) | ...) | 16u;
    return static_cast<int>(all & (~all + 1));
}

// Call f with the elements of an access (an integral constant): 16, 8 or 4 bytes or
// one element.
template <int SIZE, class F>
cudaError_t with_access(int alignment, F &&f) {
    if (alignment >= 16) return f(std::integral_constant<int, 16 / SIZE>{});
    if (alignment >= 8) return f(std::integral_constant<int, 8 / SIZE>{});
    if (SIZE < 4 && alignment >= 4) return f(std::integral_constant<int, SIZE < 4 ? 4 / SIZE : 1>{});
    return f(std::integral_constant<int, 1>{});
}

constexpr unsigned kMaxGridY = 65535;

template <class El, int J, int TPR>
cudaError_t gather_tpr(const MoveArgs &a, cudaStream_t stream) {
    using T = typename El::T;
    constexpr int kSize = sizeof(T);
    const int al = common_alignment(reinterpret_cast<uintptr_t>(a.X), reinterpret_cast<uintptr_t>(a.Y), a.ldx * kSize,
                                    a.ldy * kSize, static_cast<long long>(a.width) * kSize);
    const unsigned blocks = blocks_of(a.tokens, 256 / TPR);
    const dim3 grid((a.width + TPR * kV - 1) / (TPR * kV), blocks < kMaxGridY ? blocks : kMaxGridY);
    return with_access<kSize>(al, [&](auto n) {
        return launch_dependent(gather_kernel<El, J, TPR, decltype(n)::value>, grid, dim3(256), 0, stream, 1,
                                static_cast<const T *>(a.Y), a.ldy, a.tokens, a.choices, a.width, a.rows, a.weights,
                                static_cast<T *>(const_cast<void *>(a.X)), a.ldx);
    });
}

// A warp a token (and 256 elements) where a row does not give a block's threads eight
// elements each: 3000 tokens, 4 choices, 512 elements of 16 bits 3.4 us against 6.4,
// 1024 6.2 against 7.8; 4096 elements, 8192 tokens 56.1 against 54.9.
template <class El, int J>
cudaError_t gather_j(const MoveArgs &a, cudaStream_t stream) {
    return a.width < 256 * kV ? gather_tpr<El, J, 32>(a, stream) : gather_tpr<El, J, 256>(a, stream);
}

template <class El>
cudaError_t gather_typed(const MoveArgs &a, cudaStream_t stream) {
    if (a.choices == 1) return gather_j<El, 1>(a, stream);
    if (a.choices == 2) return gather_j<El, 2>(a, stream);
    return gather_j<El, 4>(a, stream);
}

template <class El, int J, int TPR>
cudaError_t combine_grad_tpr(const MoveArgs &a, cudaStream_t stream) {
    using T = typename El::T;
    constexpr int kSize = sizeof(T);
    const int al = common_alignment(reinterpret_cast<uintptr_t>(a.X), reinterpret_cast<uintptr_t>(a.Y),
                                    reinterpret_cast<uintptr_t>(a.dY), a.ldx * kSize, a.ldy * kSize, a.lddy * kSize,
                                    static_cast<long long>(a.width) * kSize);
    return with_access<kSize>(al, [&](auto n) {
        return launch_dependent(combine_grad_kernel<El, J, TPR, decltype(n)::value>,
                                dim3(blocks_of(a.tokens, 256 / TPR)), dim3(256), 0, stream, 1,
                                static_cast<const T *>(a.X), a.ldx, static_cast<const T *>(a.Y), a.ldy, a.tokens,
                                a.choices, a.width, a.rows, a.weights, static_cast<T *>(a.dY), a.lddy, a.scale);
    });
}

// A warp a token under the same condition, if there are tokens enough that their
// warps fill the GPU: with the forward 3000 tokens, 4 choices, 512 elements of 16 bits
// 8.9 us against 17.4, 2048 28.2 either way, 8192 tokens of 4096 152.6 against 143.2;
// 30 tokens of 1024 5.5 against 3.8.
template <class El, int J>
cudaError_t combine_grad_j(const MoveArgs &a, cudaStream_t stream) {
    return a.width < 256 * kV && a.tokens >= a.width / 2 ? combine_grad_tpr<El, J, 32>(a, stream) : combine_grad_tpr<El, J, 256>(a, stream);
}

template <class El>
cudaError_t combine_grad_typed(const MoveArgs &a, cudaStream_t stream) {
    if (a.choices == 1) return combine_grad_j<El, 1>(a, stream);
    if (a.choices == 2) return combine_grad_j<El, 2>(a, stream);
    return combine_grad_j<El, 4>(a, stream);
}

template <class Unit, int PER>
cudaError_t move_per(const MoveArgs &a, int size, int width, cudaStream_t stream) {
    constexpr int kUnits = PER * kMovesOf<Unit>;
    const unsigned blocks = blocks_of(a.tokens, 256 / PER);
    const dim3 grid((width + kUnits - 1) / kUnits, blocks < kMaxGridY ? blocks : kMaxGridY);
    return launch_dependent(move_kernel<Unit, PER>, grid, dim3(256), 0, stream, 1, static_cast<const Unit *>(a.X),
                            a.ldx * size / static_cast<int>(sizeof(Unit)), a.tokens, a.choices, width, a.rows,
                            static_cast<Unit *>(a.Y), a.ldy * size / static_cast<int>(sizeof(Unit)));
}

// A warp a row where that leaves no thread of it more than its units, else the block.
template <class Unit>
cudaError_t move_units(const MoveArgs &a, int size, cudaStream_t stream) {
    const int width = static_cast<int>(static_cast<long long>(a.width) * size / static_cast<int>(sizeof(Unit)));
    return width <= 32 * kMovesOf<Unit> ? move_per<Unit, 32>(a, size, width, stream)
                                          : move_per<Unit, 256>(a, size, width, stream);
}

}  // namespace

template <class El>
static cudaError_t quantize_aligned(const MoveArgs &a, int num_sms, cudaStream_t stream) {
    constexpr int kSize = sizeof(typename El::T);
    // an access's bytes of Q are aligned as its elements of X are
    const int al = common_alignment(reinterpret_cast<uintptr_t>(a.X), a.ldx * kSize, static_cast<long long>(a.width) * kSize,
                                    reinterpret_cast<uintptr_t>(a.Y) * kSize, a.ldy * kSize);
    return with_access<kSize>(al, [&](auto n) { return quantize_typed<El, decltype(n)::value>(a, num_sms, stream); });
}

cudaError_t launch_quantize(int type, const MoveArgs &a, int num_sms, cudaStream_t stream) {
    if (type == SGEMM_IN_F32) return quantize_aligned<ElF32>(a, num_sms, stream);
    if (type == SGEMM_IN_BF16) return quantize_aligned<ElBF16>(a, num_sms, stream);
    return quantize_aligned<ElF16>(a, num_sms, stream);
}

cudaError_t sort_prepare() {
    const int most = (kSortWarps + 1) * kMaxExperts * static_cast<int>(sizeof(int));
    for (auto *k : {sort_kernel<0, 1>, sort_kernel<0, 2>, sort_kernel<1, 1>, sort_kernel<2, 1>,
                    sort_kernel<1, 4>, sort_kernel<2, 4>, sort_kernel<1, 16>, sort_kernel<2, 16>}) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Counting and placing in two launches, each CTA reading the counts of all.
template <int STEPS>
static cudaError_t sort_two(const int *ids, int slots, int experts, int *offsets, int *rows, int *source, int *hist,
                            int smem, cudaStream_t stream) {
    const dim3 ctas(static_cast<unsigned>((static_cast<long long>(slots) + kSortThreads * STEPS - 1) / (kSortThreads * STEPS)));
    const cudaError_t e = launch_dependent(sort_kernel<1, STEPS>, ctas, dim3(kSortThreads), smem, stream, 1, ids, slots,
                                           experts, offsets, rows, source, hist);
    if (e != cudaSuccess) return e;
    return launch_dependent(sort_kernel<2, STEPS>, ctas, dim3(kSortThreads), smem, stream, 1, ids, slots, experts,
                            offsets, rows, source, hist);
}

int sort_most_slots(size_t hist_ints, int experts) {
    const unsigned long long most = hist_ints / experts * (16ull * kSortThreads);
    return most < 0x7fffffffull ? static_cast<int>(most) : 0x7fffffff;
}

cudaError_t launch_sort(const int *ids, int slots, int experts, int *offsets, int *rows, int *source, int *hist,
                        int *launches, cudaStream_t stream) {
    const int smem = (kSortWarps + 1) * experts * static_cast<int>(sizeof(int));
    // Up to 2048 slots in one CTA, one launch; beyond (4096 slots, 64 experts: 4.8 us
    // against 6.2), CTAs of 1024 slots up to 32 of them, then 4096, and 16384
    // where that would be more than 128 (each CTA reads the counts of all).
    *launches = slots <= 2 * kSortThreads ? 1 : 2;
    if (slots <= kSortThreads)
        return launch_dependent(sort_kernel<0, 1>, dim3(1), dim3(kSortThreads), smem, stream, 1, ids, slots, experts,
                                offsets, rows, source, hist);
    if (slots <= 2 * kSortThreads)
        return launch_dependent(sort_kernel<0, 2>, dim3(1), dim3(kSortThreads), smem, stream, 1, ids, slots, experts,
                                offsets, rows, source, hist);
    if (slots <= 32 * kSortThreads) return sort_two<1>(ids, slots, experts, offsets, rows, source, hist, smem, stream);
    if (slots <= 512 * kSortThreads) return sort_two<4>(ids, slots, experts, offsets, rows, source, hist, smem, stream);
    return sort_two<16>(ids, slots, experts, offsets, rows, source, hist, smem, stream);
}

cudaError_t launch_dispatch(int type, const MoveArgs &a, cudaStream_t stream) {
    const int size = type == SGEMM_IN_F32 ? 4 : 2;
    const int al = common_alignment(reinterpret_cast<uintptr_t>(a.X), reinterpret_cast<uintptr_t>(a.Y), a.ldx * size,
                                    a.ldy * size, static_cast<long long>(a.width) * size);
    if (al >= 16) return move_units<uint4>(a, size, stream);
    if (al >= 8) return move_units<uint2>(a, size, stream);
    if (al >= 4) return move_units<uint32_t>(a, size, stream);
    return move_units<uint16_t>(a, size, stream);
}

cudaError_t launch_gather(int type, const MoveArgs &a, cudaStream_t stream) {
    if (type == SGEMM_IN_F32) return gather_typed<ElF32>(a, stream);
    if (type == SGEMM_IN_BF16) return gather_typed<ElBF16>(a, stream);
    return gather_typed<ElF16>(a, stream);
}

cudaError_t launch_combine_grad(int type, const MoveArgs &a, cudaStream_t stream) {
    if (type == SGEMM_IN_F32) return combine_grad_typed<ElF32>(a, stream);
    if (type == SGEMM_IN_BF16) return combine_grad_typed<ElBF16>(a, stream);
    return combine_grad_typed<ElF16>(a, stream);
}

}  // namespace sg
