// Rows to 8-bit integers, and rows sorted by expert and back, for sm_103a.
//
//  * quantize_kernel -- per row i of X (FP32, BF16 or FP16): with m = max_p
//    |x_ip|, scale_i = m / 127 and q_ip = rint(x_ip * (127 / m)) (both
//    quotients, the product and the rounding correctly rounded, ties to even),
//    an int8 in [-127, 127] by construction.  The row may go to several
//    destinations (dispatch): it is read and quantized once, written
//    `choices` times.  One pass over HBM: a row stays in the registers of the
//    TPR threads that share it (up to 4 x 8 elements a thread; longer rows are
//    read a second time, from L2).
//  * sort_kernel -- the (token, choice) slots in a stable order by expert: a
//    counting sort.  Within a warp the 32 slots of one step that name the same
//    expert find one another with match.any and take consecutive places; every
//    warp keeps its own counts in shared memory, whose exclusive sums over the
//    warps (and, with several CTAs, over the CTAs before) place each slot.
//    Integers only and no atomic whose order matters: the same order every time.
//  * move_kernel, gather_kernel, combine_grad_kernel -- the rows' way to the
//    experts, back, and the gradients; each reads and writes every row once
//    (16 bytes a thread and step where alignment allows), sums in FP32 in
//    ascending choice order and rounds once.
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

// Piece c of a row of `width` elements that `TPR` threads share: 8 consecutive
// elements a thread where VEC says that rows start on 16-byte boundaries and
// divide into eights, else 8 elements TPR apart, so that a warp's loads and
// stores are contiguous either way.  One layout for loads and stores, and no
// branch between the loads of several pieces: they are all in flight together.
template <int TPR, bool VEC>
__device__ __forceinline__ bool inside(int c, int lane, int width) {
    return (VEC ? (c * TPR + lane) * kV : c * kV * TPR + lane) < width;
}
template <class T, int TPR, bool VEC>
__device__ __forceinline__ Pack8<T> load8(const T *row, int c, int lane, int width) {
    Pack8<T> r;
    if (VEC) {
        constexpr int kWords = static_cast<int>(sizeof(T)) * kV / 16;
        const uint4 *p = reinterpret_cast<const uint4 *>(row + (c * TPR + lane) * kV);
        uint4 *d = reinterpret_cast<uint4 *>(&r);
#pragma unroll
        for (int i = 0; i < kWords; ++i) d[i] = inside<TPR, VEC>(c, lane, width) ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            const int at = (c * kV + e) * TPR + lane;
            r.v[e] = at < width ? row[at] : T(0.f);
        }
    }
    return r;
}
template <class T, int TPR, bool VEC>
__device__ __forceinline__ void store8(T *row, int c, int lane, int width, const Pack8<T> &r) {
    if (VEC) {
        constexpr int kWords = static_cast<int>(sizeof(T)) * kV / 16;
        const uint4 *s = reinterpret_cast<const uint4 *>(&r);
        if (inside<TPR, VEC>(c, lane, width))
#pragma unroll
            for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4 *>(row + (c * TPR + lane) * kV)[i] = s[i];
    } else {
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            const int at = (c * kV + e) * TPR + lane;
            if (at < width) row[at] = r.v[e];
        }
    }
}

// Sorted row of a slot, or -1 for one that has none: a value outside [0, slots)
// is no row, whatever wrote it.
__device__ __forceinline__ int row_of(const int *rows, long long slot, int slots) {
    const int r = __ldg(rows + slot);
    return static_cast<unsigned>(r) < static_cast<unsigned>(slots) ? r : -1;
}

// ---- quantization -------------------------------------------------------------
// Below this row maximum 127 / m overflows or the scale loses bits: the row is
// stored as zeros with scale 0.
constexpr float kSmallestMax = 127.f * 1.17549435e-38f;

// 1.5 * 2^23: adding it rounds a value of magnitude < 2^22 to an integer (ties
// to even) that sits in the low bits of the sum.
constexpr float kRoundMagic = 12582912.f;

template <class El, int TPR, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
quantize_kernel(const typename El::T *__restrict__ X, long long ldx, int M, int K, int8_t *__restrict__ Q,
                long long ldq, float *__restrict__ scale, const int *__restrict__ rows, int choices) {
    using T = typename El::T;
    constexpr int kThreads = TPR < 256 ? 256 : TPR;
    constexpr int kRows = kThreads / TPR, kHeld = 4;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % TPR;
    const int i = blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = i < M;
    const T *x = X + static_cast<long long>(live ? i : 0) * ldx;
    const int width = live ? K : 0;

    Pack8<T> held[kHeld];
#pragma unroll
    for (int c = 0; c < kHeld; ++c) held[c] = load8<T, TPR, VEC>(x, c, lane, width);
    unsigned top = 0;  // max of |x| as bits: NaN above infinity above every number
#pragma unroll
    for (int c = 0; c < kHeld; ++c)
#pragma unroll
        for (int e = 0; e < kV; ++e) top = max(top, __float_as_uint(El::up(held[c].v[e])) & 0x7fffffffu);
    for (int c = kHeld; c * kV * TPR < width; ++c) {
        const Pack8<T> h = load8<T, TPR, VEC>(x, c, lane, width);
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
    auto put = [&](int8_t *q, int c, uint2 w) {
        if (VEC) {
            if (inside<TPR, VEC>(c, lane, K)) *reinterpret_cast<uint2 *>(q + (c * TPR + lane) * kV) = w;
        } else {
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const int at = (c * kV + e) * TPR + lane;
                if (at < K) q[at] = static_cast<int8_t>((e < 4 ? w.x >> (8 * e) : w.y >> (8 * (e - 4))) & 0xffu);
            }
        }
    };
    uint2 packed[kHeld];
#pragma unroll
    for (int c = 0; c < kHeld; ++c) packed[c] = quantized(held[c]);
    for (int j = 0; j < choices; ++j) {
        const int r = rows ? row_of(rows, static_cast<long long>(i) * choices + j, M * choices) : i;
        if (r < 0) continue;
        int8_t *q = Q + static_cast<long long>(r) * ldq;
#pragma unroll
        for (int c = 0; c < kHeld; ++c) put(q, c, packed[c]);
        for (int c = kHeld; c * kV * TPR < K; ++c) put(q, c, quantized(load8<T, TPR, VEC>(x, c, lane, K)));
        if (lane == 0) scale[r] = s;
    }
}

template <class El, bool VEC>
cudaError_t quantize_typed(const MoveArgs &a, int num_sms, cudaStream_t stream) {
    using T = typename El::T;
    const T *X = static_cast<const T *>(a.X);
    int8_t *Q = static_cast<int8_t *>(a.Y);
    // Threads a row: enough that it stays in registers (32 elements a thread),
    // and, with too few rows to fill the GPU, more of them so that each thread
    // loads less.
    const bool few = a.tokens <= 4 * num_sms;
    const int per = few ? kV : 4 * kV;
    const int want = (a.width + per - 1) / per;
#define SG_QUANT(TPR)                                                                                            \
    return launch_dependent(quantize_kernel<El, TPR, VEC>,                                                       \
                            dim3((a.tokens + (TPR < 256 ? 256 / TPR : 1) - 1) / (TPR < 256 ? 256 / TPR : 1)),    \
                            dim3(TPR < 256 ? 256 : TPR), 0, stream, 1, X, a.ldx, a.tokens, a.width, Q, a.ldy,    \
                            a.scale, a.rows, a.choices)
    if (want <= 32) SG_QUANT(32);
    if (want <= 128) SG_QUANT(128);
    if (want <= 256) SG_QUANT(256);
    SG_QUANT(512);
#undef SG_QUANT
}

// ---- sort ---------------------------------------------------------------------
constexpr int kSortWarps = 8, kSortThreads = kSortWarps * 32;

// Shared memory: kSortWarps * E counts of the warps, E places of the CTA.
// PASS 0: one CTA does it all.  PASS 1: each CTA writes the counts of its own
// slots to hist[cta][E].  PASS 2: each CTA places its slots.
template <int PASS>
__global__ void __launch_bounds__(kSortThreads)
sort_kernel(const int *__restrict__ ids, int slots, int experts, int steps, int *__restrict__ offsets,
            int *__restrict__ rows, int *__restrict__ source, int *__restrict__ hist) {
    extern __shared__ int sh[];
    int *counts = sh, *place = sh + kSortWarps * experts;
    __shared__ int carry[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const unsigned below = (1u << lane) - 1u;
    griddep_wait();
    griddep_launch_dependents();
    for (int e = tid; e < kSortWarps * experts; e += kSortThreads) counts[e] = 0;
    __syncthreads();

    // the CTA's slots: kSortWarps runs of steps * 32, one a warp
    const long long first = (static_cast<long long>(blockIdx.x) * kSortWarps + warp) * steps * 32;
    int *mine = counts + warp * experts;
    auto expert_of = [&](long long slot) {
        const int e = slot < slots ? __ldg(ids + slot) : -1;
        return static_cast<unsigned>(e) < static_cast<unsigned>(experts) ? e : -1;
    };
    for (int s = 0; s < steps; ++s) {
        const int e = expert_of(first + s * 32 + lane);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // counts -> exclusive sums over the warps; place[e] = the CTA's slots of expert e
    for (int e = tid; e < experts; e += kSortThreads) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = counts[w * experts + e];
            counts[w * experts + e] = n;
            n += c;
        }
        if (PASS == 1) hist[static_cast<long long>(blockIdx.x) * experts + e] = n;
        place[e] = n;
    }
    if (PASS == 1) return;
    __syncthreads();
    // total[e] over all CTAs, its exclusive sum over the experts (offsets), and
    // the slots of earlier CTAs
    int base = 0;  // sum over the experts done so far
    for (int e0 = 0; e0 < experts; e0 += kSortThreads) {
        const int e = e0 + tid;
        int total = 0, before = 0;
        if (e < experts) {
            if (PASS == 0) {
                total = place[e];
            } else {
                for (int c = 0; c < static_cast<int>(gridDim.x); ++c) {
                    const int n = __ldcg(hist + static_cast<long long>(c) * experts + e);
                    if (c < static_cast<int>(blockIdx.x)) before += n;
                    total += n;
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
        int all = 0, lower = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            if (w < warp) lower += carry[w];
            all += carry[w];
        }
        const int start = base + lower + sum - total;
        if (e < experts) {
            place[e] = start + before;
            if (blockIdx.x == 0) offsets[e] = start;
        }
        base += all;
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) offsets[experts] = base;
    for (int s = 0; s < steps; ++s) {
        const long long slot = first + s * 32 + lane;
        const int e = expert_of(slot);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int r = -1;
        if (e >= 0) r = place[e] + mine[e] + __popc(same & below);
        __syncwarp();
        if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
        __syncwarp();
        if (slot < slots) {
            rows[slot] = r;
            if (r >= 0) source[r] = static_cast<int>(slot);
            if (slot >= base) source[slot] = -1;  // rows past the last expert's hold no slot
        }
    }
}

// ---- rows to the experts --------------------------------------------------------
// Row t of X to rows[t * choices + j] of Y: read once, written up to `choices`
// times.  kMoves units (the widest that the rows' alignment allows, up to 16
// bytes) a thread, all loaded before the first store.
constexpr int kMoves = 4;

template <class Unit>
__global__ void __launch_bounds__(256)
move_kernel(const Unit *__restrict__ X, long long ldx, int tokens, int choices, int width, const int *__restrict__ rows,
            Unit *__restrict__ Y, long long ldy) {
    griddep_wait();
    griddep_launch_dependents();
    const int slots = tokens * choices;
    const int c0 = blockIdx.x * (256 * kMoves) + threadIdx.x;
    for (int t = blockIdx.y; t < tokens; t += gridDim.y) {
        const Unit *x = X + static_cast<long long>(t) * ldx;
        Unit v[kMoves];
#pragma unroll
        for (int m = 0; m < kMoves; ++m) v[m] = c0 + m * 256 < width ? x[c0 + m * 256] : Unit{};
        for (int j = 0; j < choices; ++j) {
            const int r = row_of(rows, static_cast<long long>(t) * choices + j, slots);
            if (r < 0) continue;
            Unit *y = Y + static_cast<long long>(r) * ldy;
#pragma unroll
            for (int m = 0; m < kMoves; ++m)
                if (c0 + m * 256 < width) y[c0 + m * 256] = v[m];
        }
    }
}

// ---- rows from the experts ------------------------------------------------------
// out[t] = sum_j w[t,j] * Y[rows[t,j]] (w NULL: the plain sum); four rows' loads
// in flight at a time.
template <class El, bool VEC>
__global__ void __launch_bounds__(256)
gather_kernel(const typename El::T *__restrict__ Y, long long ldy, int tokens, int choices, int width,
              const int *__restrict__ rows, const float *__restrict__ weights, typename El::T *__restrict__ out,
              long long ldo) {
    using T = typename El::T;
    griddep_wait();
    griddep_launch_dependents();
    const int slots = tokens * choices, c = blockIdx.x, lane = threadIdx.x;
    for (int t = blockIdx.y; t < tokens; t += gridDim.y) {
        float sum[kV] = {};
        for (int j0 = 0; j0 < choices; j0 += 4) {
            Pack8<T> y[4];
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const long long slot = static_cast<long long>(t) * choices + j0 + j;
                const int r = j0 + j < choices ? row_of(rows, slot, slots) : -1;
                w[j] = r >= 0 && weights ? __ldg(weights + slot) : 1.f;
                // (a row that does not exist has no elements: zeros)
                y[j] = load8<T, 256, VEC>(Y + static_cast<long long>(r >= 0 ? r : 0) * ldy, c, lane, r >= 0 ? width : 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < kV; ++e) sum[e] = fmaf(w[j], El::up(y[j].v[e]), sum[e]);
        }
        Pack8<T> o;
#pragma unroll
        for (int e = 0; e < kV; ++e) o.v[e] = El::down(sum[e]);
        store8<T, 256, VEC>(out + static_cast<long long>(t) * ldo, c, lane, width, o);
    }
}

// ---- gradient of the weighted return --------------------------------------------
// dY[rows[t,j]] = w[t,j] * dO[t] and dw[t,j] = <dO[t], Y[rows[t,j]]>: 256
// threads a token, J choices at a time; the dot products are reduced in a
// fixed order (within the warp, then over the warps).
template <class El, int J, bool VEC>
__global__ void __launch_bounds__(256)
combine_grad_kernel(const typename El::T *__restrict__ dO, long long lddo, const typename El::T *__restrict__ Y,
                    long long ldy, int tokens, int choices, int width, const int *__restrict__ rows,
                    const float *__restrict__ weights, typename El::T *__restrict__ dY, long long lddy,
                    float *__restrict__ dw) {
    using T = typename El::T;
    __shared__ float part[8][J];
    griddep_wait();
    griddep_launch_dependents();
    const int slots = tokens * choices, lane = threadIdx.x;
    for (int t = blockIdx.x; t < tokens; t += gridDim.x) {
        const T *g = dO + static_cast<long long>(t) * lddo;
        for (int j0 = 0; j0 < choices; j0 += J) {
            int r[J];
            float w[J], dot[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const long long slot = static_cast<long long>(t) * choices + j0 + j;
                r[j] = j0 + j < choices ? row_of(rows, slot, slots) : -1;
                w[j] = r[j] >= 0 ? __ldg(weights + slot) : 0.f;
                dot[j] = 0.f;
            }
            for (int c = 0; c * 256 * kV < width; ++c) {
                const Pack8<T> gv = load8<T, 256, VEC>(g, c, lane, width);
                Pack8<T> y[J];
#pragma unroll
                for (int j = 0; j < J; ++j)
                    y[j] = load8<T, 256, VEC>(Y + static_cast<long long>(r[j] >= 0 ? r[j] : 0) * ldy, c, lane,
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
                    if (r[j] >= 0) store8<T, 256, VEC>(dY + static_cast<long long>(r[j]) * lddy, c, lane, width, o);
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (r[j] < 0) dot[j] = 0.f;  // not 0 * dO, which a non-finite dO makes NaN
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
                if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < J && j0 + threadIdx.x < choices) {
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += part[k][threadIdx.x];
                dw[static_cast<long long>(t) * choices + j0 + threadIdx.x] = sum;
            }
            __syncthreads();
        }
    }
}

inline bool vec_ok(const void *p, long long ld, int size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * size) % 16 == 0;
}

constexpr int kMaxGridY = 65535;

template <class El>
cudaError_t gather_typed(const MoveArgs &a, cudaStream_t stream) {
    using T = typename El::T;
    const bool vec = a.width % kV == 0 && vec_ok(a.Y, a.ldy, sizeof(T)) && vec_ok(a.X, a.ldx, sizeof(T));
    const dim3 grid((a.width + 256 * kV - 1) / (256 * kV), a.tokens < kMaxGridY ? a.tokens : kMaxGridY);
    return launch_dependent(vec ? gather_kernel<El, true> : gather_kernel<El, false>, grid, dim3(256), 0, stream, 1,
                            static_cast<const T *>(a.Y), a.ldy, a.tokens, a.choices, a.width, a.rows, a.weights,
                            static_cast<T *>(const_cast<void *>(a.X)), a.ldx);
}

template <class El, int J>
cudaError_t combine_grad_j(const MoveArgs &a, cudaStream_t stream) {
    using T = typename El::T;
    const bool vec = a.width % kV == 0 && vec_ok(a.X, a.ldx, sizeof(T)) && vec_ok(a.Y, a.ldy, sizeof(T)) &&
                     vec_ok(a.dY, a.lddy, sizeof(T));
    return launch_dependent(vec ? combine_grad_kernel<El, J, true> : combine_grad_kernel<El, J, false>,
                            dim3(a.tokens), dim3(256), 0, stream, 1, static_cast<const T *>(a.X), a.ldx,
                            static_cast<const T *>(a.Y), a.ldy, a.tokens, a.choices, a.width, a.rows, a.weights,
                            static_cast<T *>(a.dY), a.lddy, a.scale);
}

template <class El>
cudaError_t combine_grad_typed(const MoveArgs &a, cudaStream_t stream) {
    if (a.choices == 1) return combine_grad_j<El, 1>(a, stream);
    if (a.choices == 2) return combine_grad_j<El, 2>(a, stream);
    return combine_grad_j<El, 4>(a, stream);
}

template <class Unit>
cudaError_t move_units(const MoveArgs &a, int size, cudaStream_t stream) {
    const int width = static_cast<int>(static_cast<long long>(a.width) * size / static_cast<int>(sizeof(Unit)));
    const dim3 grid((width + 256 * kMoves - 1) / (256 * kMoves), a.tokens < kMaxGridY ? a.tokens : kMaxGridY);
    return launch_dependent(move_kernel<Unit>, grid, dim3(256), 0, stream, 1, static_cast<const Unit *>(a.X),
                            a.ldx * size / static_cast<int>(sizeof(Unit)), a.tokens, a.choices, width, a.rows,
                            static_cast<Unit *>(a.Y), a.ldy * size / static_cast<int>(sizeof(Unit)));
}

}  // namespace

cudaError_t launch_quantize(int type, const MoveArgs &a, int num_sms, cudaStream_t stream) {
    const bool vec = a.width % kV == 0 && vec_ok(a.X, a.ldx, type == SGEMM_IN_F32 ? 4 : 2) &&
                     reinterpret_cast<uintptr_t>(a.Y) % kV == 0 && a.ldy % kV == 0;
    if (type == SGEMM_IN_F32)
        return vec ? quantize_typed<ElF32, true>(a, num_sms, stream) : quantize_typed<ElF32, false>(a, num_sms, stream);
    if (type == SGEMM_IN_BF16)
        return vec ? quantize_typed<ElBF16, true>(a, num_sms, stream)
                   : quantize_typed<ElBF16, false>(a, num_sms, stream);
    return vec ? quantize_typed<ElF16, true>(a, num_sms, stream) : quantize_typed<ElF16, false>(a, num_sms, stream);
}

cudaError_t sort_prepare() {
    const int most = (kSortWarps + 1) * kMaxExperts * static_cast<int>(sizeof(int));
    for (auto *k : {sort_kernel<0>, sort_kernel<1>, sort_kernel<2>}) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_sort(const int *ids, int slots, int experts, int *offsets, int *rows, int *source, int *hist,
                        size_t hist_ints, int *launches, cudaStream_t stream) {
    const int smem = (kSortWarps + 1) * experts * static_cast<int>(sizeof(int));
    // Up to 16 steps of 256 slots in one CTA (one launch); beyond, CTAs of 4
    // steps, or as many steps as keep the counts within the workspace and
    // under 256 CTAs (each CTA reads the counts of all).
    *launches = 1;
    if (slots <= 16 * kSortThreads) {
        const int steps = slots > kSortThreads ? (slots + kSortThreads - 1) / kSortThreads : 1;
        return launch_dependent(sort_kernel<0>, dim3(1), dim3(kSortThreads), smem, stream, 1, ids, slots, experts,
                                steps, offsets, rows, source, hist);
    }
    const long long most = static_cast<long long>(hist_ints) / experts;
    const int ctas_most = static_cast<int>(most < 256 ? most : 256);
    int steps = (slots + kSortThreads * ctas_most - 1) / (kSortThreads * ctas_most);
    if (steps < 4) steps = 4;
    const int ctas = (slots + kSortThreads * steps - 1) / (kSortThreads * steps);
    *launches = 2;
    const cudaError_t e = launch_dependent(sort_kernel<1>, dim3(ctas), dim3(kSortThreads), smem, stream, 1, ids, slots,
                                           experts, steps, offsets, rows, source, hist);
    if (e != cudaSuccess) return e;
    return launch_dependent(sort_kernel<2>, dim3(ctas), dim3(kSortThreads), smem, stream, 1, ids, slots, experts,
                            steps, offsets, rows, source, hist);
}

cudaError_t launch_dispatch(int type, const MoveArgs &a, cudaStream_t stream) {
    const int size = type == SGEMM_IN_F32 ? 4 : 2;
    // the largest power of two that divides every row's start and length
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.Y) |
                          static_cast<uintptr_t>(a.ldx * size) | static_cast<uintptr_t>(a.ldy * size) |
                          static_cast<uintptr_t>(static_cast<long long>(a.width) * size);
    if (all % 16 == 0) return move_units<uint4>(a, size, stream);
    if (all % 8 == 0) return move_units<uint2>(a, size, stream);
    if (all % 4 == 0) return move_units<uint32_t>(a, size, stream);
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
