// The gradient of the RMS norm for sm_103a.  With y = h r w, r = 1 / sqrt(mean(h^2)
// + eps) and g = w dy, row by row
//     dh_p = r g_p - h_p r^3 (sum_q g_q h_q) / K  (+ the gradient that reaches h from elsewhere)
//     dw_p = sum over the rows of dy_p h_p r
//
//  * norm_grad_kernel -- each row's threads go through rows a grid apart: dy, h and
//    what reaches h are read once and stay in registers for the row's sum and its
//    gradient, the columns' sums in registers from row to row; at the end each group
//    of threads writes its sums, a row of `parts`.
//  * norm_grad_ring_kernel -- the same for long rows on 16-byte boundaries: 8192 x 4096 BF16
//    with the gradient that reaches h 43 us, floor 40, and 5 for the columns' sums, which
//    overlap.
//  * columns_kernel -- dw: the rows of `parts` added up.
//  * norm_grad_wide_kernel, columns_wide_kernel -- the same for rows longer than the
//    registers of 512 threads hold: each row is read twice, and the columns' sums are
//    taken from dy and h by a kernel of their own.
//
// Every sum is in FP32 and in an order that only the sizes and the GPU's SM count set: no
// atomics, the same bits every time.
#include "device_common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "sgemm.h"

namespace sg {
namespace {

// Sum over the TPR threads of a row; `part` has a float for each of the block's warps.
template <int TPR>
__device__ __forceinline__ float row_sum(float sum, float *part) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = sum;
        __syncthreads();
        const int w0 = threadIdx.x / TPR * (TPR / 32);
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) sum += part[w0 + w];
    }
    return sum;
}

template <int TPR>
constexpr int kGradThreads = TPR < 256 ? 256 : TPR;

template <class El, int TPR, int A, int HELD>
__global__ void __launch_bounds__(kGradThreads<TPR>, TPR < 512 ? 2 : 1)
norm_grad_kernel(const NormGradArgs a) {
    using T = typename El::T;
    constexpr int kRows = kGradThreads<TPR> / TPR;
    __shared__ float part[2][kGradThreads<TPR> / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % TPR, group = blockIdx.x * kRows + threadIdx.x / TPR;
    const unsigned step = gridDim.x * kRows;
    const T *w = static_cast<const T *>(a.W);
    Pack8<T> g[HELD];
    float dw[HELD][kV];
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
        g[c] = load8<T, TPR, A, true>(w, c, lane, a.K);
#pragma unroll
        for (int e = 0; e < kV; ++e) dw[c][e] = 0.f;
    }
    struct Row {
        Pack8<T> d[HELD], x[HELD], more[HELD];
        float r;
    };
    auto load = [&](unsigned i) {
        Row q;
        const bool live = i < static_cast<unsigned>(a.M);
        const long long row = live ? i : 0;
        const int width = live ? a.K : 0;
        const T *dy = static_cast<const T *>(a.dY) + row * a.lddy, *h = static_cast<const T *>(a.H) + row * a.ldh;
        const T *dh = static_cast<const T *>(a.dH) + (a.dH ? row * a.lddh : 0);
#pragma unroll
        for (int c = 0; c < HELD; ++c) {
            q.d[c] = load8<T, TPR, A>(dy, c, lane, width);
            q.x[c] = load8<T, TPR, A>(h, c, lane, width);
        }
        if (a.dH) {
#pragma unroll
            for (int c = 0; c < HELD; ++c) q.more[c] = load8<T, TPR, A>(dh, c, lane, width);
        }
        q.r = live ? __ldca(a.rstd + i) : 0.f;
        return q;
    };
    // The next row is on its way while one is added up and written (one row at a time: 8192 x 4096
    // BF16 with both gradients 71 us); rows of 32 elements a thread leave no registers for it.
    constexpr bool kEarly = HELD < 4;
    // (every group makes as many rounds as the first: the barriers are the block's)
    int turn = 0;
    unsigned i0 = blockIdx.x * kRows;
    const unsigned mine = threadIdx.x / TPR;
    Row next;
    if (kEarly) next = load(i0 + mine);
    for (; i0 < static_cast<unsigned>(a.M); i0 += step, turn ^= 1) {
        const unsigned i = i0 + mine;
        const bool live = i < static_cast<unsigned>(a.M);
        const Row q = kEarly ? next : load(i);
        if (kEarly && i0 + step < static_cast<unsigned>(a.M)) next = load(i + step);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < HELD; ++c)
#pragma unroll
            for (int e = 0; e < kV; ++e) sum = fmaf(El::up(q.d[c].v[e]) * El::up(g[c].v[e]), El::up(q.x[c].v[e]), sum);
        sum = row_sum<TPR>(sum, part[turn]);
        const float f = sum * q.r * q.r / static_cast<float>(a.K);
        T *dx = static_cast<T *>(a.dX) + (live ? i * a.lddx : 0);
#pragma unroll
        for (int c = 0; c < HELD; ++c) {
            Pack8<T> o;
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const float dv = El::up(q.d[c].v[e]), hv = El::up(q.x[c].v[e]);
                // (lanes behind a row's end and rows behind the last hold zeros: nothing is added)
                dw[c][e] = fmaf(dv, hv * q.r, dw[c][e]);
                float v = q.r * fmaf(-hv, f, dv * El::up(g[c].v[e]));
                if (a.dH) v += El::up(q.more[c].v[e]);
                o.v[e] = El::down(v);
            }
            if (live) store8<T, TPR, A>(dx, c, lane, a.K, o);
        }
    }
    float *to = a.parts + static_cast<long long>(group) * a.K;
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
        const int at = c * kV * TPR + lane * A;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            const int p = at + e / A * TPR * A + e % A;
            if (p < a.K) to[p] = dw[c][e];
        }
    }
}

// The same for rows that start on 16-byte boundaries and are copied as a whole (cp.async.bulk)
// into a ring of shared memory, several rows ahead of the one that is added up: as many
// bytes are on their way as HBM's latency wants, where a row ahead in registers is half of that.
// One row at a time for the whole block.
constexpr int kGradStages = 4;
template <class El, int TPR, int HELD>
__global__ void __launch_bounds__(TPR, TPR == 256 ? 2 : 1)
norm_grad_ring_kernel(const NormGradArgs a, int stages) {
    using T = typename El::T;
    constexpr int A = 16 / sizeof(T);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kGradStages];
    __shared__ float part[2][TPR / 32];
    const int lane = threadIdx.x, step = gridDim.x;
    const int row_bytes = a.K * static_cast<int>(sizeof(T)), arrays = a.dH ? 3 : 2, stage_bytes = 3 * ((row_bytes + 127) & ~127);
    if (lane == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    auto part_of = [&](int s, int k) { return smem + s * stage_bytes + k * (stage_bytes / 3); };
    auto issue = [&](int s, long long i) {
        auto copy = [&](int k, const void *from, long long ld) {
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                         ::"r"(smem_u32(part_of(s, k))), "l"(static_cast<const T *>(from) + i * ld), "r"(row_bytes), "r"(smem_u32(&full[s])) : "memory");
        };
        mbar_arrive_expect_tx(&full[s], arrays * row_bytes);
        copy(0, a.dY, a.lddy);
        copy(1, a.H, a.ldh);
        if (a.dH) copy(2, a.dH, a.lddh);
    };
    const long long first = blockIdx.x;
    if (lane == 0)
        for (int s = 0; s < stages && first + static_cast<long long>(s) * step < a.M; ++s) issue(s, first + static_cast<long long>(s) * step);
    Pack8<T> g[HELD];
    float dw[HELD][kV];
#pragma unroll
    for (int c = 0; c < HELD; ++c) {
        g[c] = load8<T, TPR, A, true>(static_cast<const T *>(a.W), c, lane, a.K);
#pragma unroll
        for (int e = 0; e < kV; ++e) dw[c][e] = 0.f;
    }
    // one piece of a row in shared memory, as load8 takes it
    auto piece = [&](const uint8_t *row, int c) {
        Pack8<T> r;
        const int at = c * kV * TPR + lane * A;
#pragma unroll
        for (int i = 0; i < kV / A; ++i)
            reinterpret_cast<uint4 *>(&r)[i] = at + i * TPR * A < a.K ? *reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(row) + at + i * TPR * A) : uint4{};
        return r;
    };
    int s = 0, turn = 0;
    uint32_t round = 0;
    bool ok = true;  // (after a wait that ran out the block still meets at its barriers)
    float next_r = first < a.M ? __ldca(a.rstd + first) : 0.f;
    for (long long i = first; i < a.M; i += step, turn ^= 1) {
        const float r = next_r;
        if (i + step < a.M) next_r = __ldca(a.rstd + i + step);
        ok = ok && mbar_wait(&full[s], round, a.status);
        Pack8<T> d[HELD], x[HELD], more[HELD];
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < HELD; ++c) {
            d[c] = piece(part_of(s, 0), c);
            x[c] = piece(part_of(s, 1), c);
            if (a.dH) more[c] = piece(part_of(s, 2), c);
#pragma unroll
            for (int e = 0; e < kV; ++e) sum = fmaf(El::up(d[c].v[e]) * El::up(g[c].v[e]), El::up(x[c].v[e]), sum);
        }
        sum = row_sum<TPR>(sum, part[turn]);  // (and every thread has taken its part of the row)
        const long long then = i + static_cast<long long>(stages) * step;
        if (lane == 0 && ok && then < a.M) issue(s, then);
        if (++s == stages) {
            s = 0;
            round ^= 1u;
        }
        const float f = sum * r * r / static_cast<float>(a.K);
        T *dx = static_cast<T *>(a.dX) + i * a.lddx;
#pragma unroll
        for (int c = 0; c < HELD; ++c) {
            Pack8<T> o;
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const float dv = El::up(d[c].v[e]), hv = El::up(x[c].v[e]);
                dw[c][e] = fmaf(dv, hv * r, dw[c][e]);
                float v = r * fmaf(-hv, f, dv * El::up(g[c].v[e]));
                if (a.dH) v += El::up(more[c].v[e]);
                o.v[e] = El::down(v);
            }
            if (ok) store8<T, TPR, A>(dx, c, lane, a.K, o);
        }
    }
    if (!ok && lane == 0)  // no copy outlives the CTA
        for (int k = 0; k < stages; ++k) mbar_wait(&full[k], k < s ? round : round ^ 1u, a.status);
    float *to = a.parts + static_cast<long long>(blockIdx.x) * a.K;
#pragma unroll
    for (int c = 0; c < HELD; ++c)
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            const int p = c * kV * TPR + lane * A + e / A * TPR * A + e % A;
            if (p < a.K) to[p] = dw[c][e];
        }
}

// dw[p] = sum of column p of `parts` (n rows): 32 columns a block, each of its 32 warps
// the rows 32 apart, then the warps' sums.
__global__ void __launch_bounds__(1024) columns_kernel(const float *parts, int n, int K, float *dw) {
    __shared__ float sums[32][33];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int p = blockIdx.x * 32 + lane;
    float s[4] = {};
    for (int i = warp; i < n; i += 128) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (p < K && i + 32 * j < n) s[j] += __ldcg(parts + static_cast<long long>(i + 32 * j) * K + p);
    }
    sums[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    // warp w adds up column w of this block's
    float sum = sums[lane][warp];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0 && blockIdx.x * 32 + warp < K) dw[blockIdx.x * 32 + warp] = sum;
}

// Rows of any length: one block of 512 threads a row.
template <class El>
__global__ void __launch_bounds__(512) norm_grad_wide_kernel(const NormGradArgs a) {
    using T = typename El::T;
    __shared__ float part[16];
    griddep_wait();
    griddep_launch_dependents();
    for (unsigned i = blockIdx.x; i < static_cast<unsigned>(a.M); i += gridDim.x) {
        const T *dy = static_cast<const T *>(a.dY) + i * a.lddy, *h = static_cast<const T *>(a.H) + i * a.ldh;
        const T *dh = a.dH ? static_cast<const T *>(a.dH) + i * a.lddh : nullptr, *w = static_cast<const T *>(a.W);
        const float r = __ldca(a.rstd + i);
        float sum = 0.f;
        for (int p = threadIdx.x; p < a.K; p += 512)
            sum = fmaf(El::up(__ldcg(dy + p)) * El::up(__ldca(w + p)), El::up(__ldcg(h + p)), sum);
        sum = row_sum<512>(sum, part);
        const float f = sum * r * r / static_cast<float>(a.K);
        T *dx = static_cast<T *>(a.dX) + i * a.lddx;
        for (int p = threadIdx.x; p < a.K; p += 512) {
            float v = r * fmaf(-El::up(__ldcg(h + p)), f, El::up(__ldcg(dy + p)) * El::up(__ldca(w + p)));
            if (dh) v += El::up(__ldcg(dh + p));
            dx[p] = El::down(v);
        }
        __syncthreads();
    }
}

// Column sums of dy h r over the rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <class El>
__global__ void __launch_bounds__(256) columns_wide_kernel(const NormGradArgs a) {
    using T = typename El::T;
    griddep_wait();
    griddep_launch_dependents();
    const int p = blockIdx.x * 256 + threadIdx.x;
    if (p >= a.K) return;
    float sum = 0.f;
    for (unsigned i = blockIdx.y; i < static_cast<unsigned>(a.M); i += gridDim.y)
        sum = fmaf(El::up(__ldcg(static_cast<const T *>(a.dY) + i * a.lddy + p)),
                   El::up(__ldcg(static_cast<const T *>(a.H) + i * a.ldh + p)) * __ldca(a.rstd + i), sum);
    a.parts[static_cast<long long>(blockIdx.y) * a.K + p] = sum;
}

cudaError_t add_parts(const NormGradArgs &a, int n, cudaStream_t stream) {
    return launch_dependent(columns_kernel, dim3(blocks_of(a.K, 32)), dim3(1024), 0, stream, 1, static_cast<const float *>(a.parts), n, a.K, a.dW);
}

template <class El, int TPR, int A, int HELD>
cudaError_t grad_typed(const NormGradArgs &a, int num_sms, size_t ws_floats, cudaStream_t stream) {
    constexpr int kRows = kGradThreads<TPR> / TPR;
    const size_t fit = ws_floats / (static_cast<size_t>(a.K) * kRows);  // blocks whose sums the workspace holds
    size_t blocks = blocks_of(a.M, kRows);
    blocks = blocks < static_cast<size_t>(2 * num_sms) ? blocks : static_cast<size_t>(2 * num_sms);
    blocks = blocks < fit ? blocks : fit;
    const cudaError_t e = launch_dependent(norm_grad_kernel<El, TPR, A, HELD>, dim3(static_cast<unsigned>(blocks)), dim3(kGradThreads<TPR>), 0, stream, 1, a);
    return e != cudaSuccess ? e : add_parts(a, static_cast<int>(blocks) * kRows, stream);
}

// Shared memory that a block of the ring kernel may take: two of 256 threads an SM, or one of 512.
template <int TPR>
constexpr int kRingRoom = TPR == 256 ? 112 << 10 : 224 << 10;

template <class El, int TPR, int HELD>
cudaError_t grad_ring(const NormGradArgs &a, int num_sms, size_t ws_floats, cudaStream_t stream) {
    const int stage = 3 * ((a.K * static_cast<int>(sizeof(typename El::T)) + 127) & ~127);
    const int fit = kRingRoom<TPR> / stage, stages = fit < kGradStages ? fit : kGradStages;
    size_t blocks = static_cast<size_t>(TPR == 256 ? 2 : 1) * num_sms;
    blocks = blocks < static_cast<size_t>(a.M) ? blocks : static_cast<size_t>(a.M);
    blocks = blocks < ws_floats / a.K ? blocks : ws_floats / a.K;
    const cudaError_t e = launch_dependent(norm_grad_ring_kernel<El, TPR, HELD>, dim3(static_cast<unsigned>(blocks)), dim3(TPR), stages * stage, stream, 1, a, stages);
    return e != cudaSuccess ? e : add_parts(a, static_cast<int>(blocks), stream);
}

template <class El, int A>
cudaError_t grad_shared(const NormGradArgs &a, int num_sms, size_t ws_floats, cudaStream_t stream) {
    // threads a row: 16 elements each where the rows are that long, 32 in the longest
    if (a.K <= 256) return grad_typed<El, 32, A, 1>(a, num_sms, ws_floats, stream);
    if (a.K <= 512) return grad_typed<El, 32, A, 2>(a, num_sms, ws_floats, stream);
    if (a.K <= 2048) return grad_typed<El, 128, A, 2>(a, num_sms, ws_floats, stream);
    if (a.K <= 4096) return grad_typed<El, 256, A, 2>(a, num_sms, ws_floats, stream);
    if (a.K <= 8192) return grad_typed<El, 512, A, 2>(a, num_sms, ws_floats, stream);
    return grad_typed<El, 512, A, 4>(a, num_sms, ws_floats, stream);
}

template <class El>
cudaError_t grad_for(const NormGradArgs &a, int num_sms, size_t ws_floats, cudaStream_t stream) {
    using T = typename El::T;
    constexpr int V = 16 / sizeof(T);
    if (a.K > kNormHeld) {
        cudaError_t e = launch_dependent(norm_grad_wide_kernel<El>, dim3(a.M < 4 * num_sms ? a.M : 4 * num_sms), dim3(512), 0, stream, 1, a);
        if (e != cudaSuccess) return e;
        const size_t fit = ws_floats / a.K;  // at least one: checked where the call starts
        const int most = a.M < 64 ? a.M : 64, n = fit < static_cast<size_t>(most) ? static_cast<int>(fit) : most;
        e = launch_dependent(columns_wide_kernel<El>, dim3(blocks_of(a.K, 256), n), dim3(256), 0, stream, 1, a);
        return e != cudaSuccess ? e : add_parts(a, n, stream);
    }
    auto unit = [](const void *p, long long ld, int n) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (n * sizeof(T)) == 0 && ld % n == 0);
    };
    auto fits = [&](int n) {
        return a.K % n == 0 && unit(a.dY, a.lddy, n) && unit(a.H, a.ldh, n) && unit(a.dH, a.lddh, n) && unit(a.W, 0, n) && unit(a.dX, a.lddx, n);
    };
    if (fits(V)) {
        // Rows long enough that a block has one at a time, and enough of them to go round (us with the
        // columns' sums, BF16 with both gradients, ring against registers: 8192 x 4096 47.4, 61.3; 912 x 2056
        // 8.9, 9.7; 640 x 4096 11.3, 12.0).  With fewer the two are near (608 x 4096 11.5, 11.9; 64 x 2056 4.5,
        // 4.3) but in rows of 8192, which take the registers of 512 threads (608 of them 14.2, 21.4).
        if (a.K > 2048 && a.M > 4 * num_sms) {
            if (a.K <= 4096) return grad_ring<El, 256, 2>(a, num_sms, ws_floats, stream);
            if (a.K <= 8192) return grad_ring<El, 512, 2>(a, num_sms, ws_floats, stream);
        }
        return grad_shared<El, V>(a, num_sms, ws_floats, stream);
    }
    if (fits(2)) return grad_shared<El, 2>(a, num_sms, ws_floats, stream);
    return grad_shared<El, 1>(a, num_sms, ws_floats, stream);
}

}  // namespace

template <class El>
static cudaError_t prepare_ring() {
    const cudaError_t e = cudaFuncSetAttribute(norm_grad_ring_kernel<El, 256, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingRoom<256>);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(norm_grad_ring_kernel<El, 512, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingRoom<512>);
}

cudaError_t norm_prepare() {
    cudaError_t e = cudaSuccess;
    for (cudaError_t r : {prepare_ring<ElF32>(), prepare_ring<ElBF16>(), prepare_ring<ElF16>()})
        if (e == cudaSuccess) e = r;
    return e;
}

int norm_grad_launches(int K) { return K > kNormHeld ? 3 : 2; }

cudaError_t launch_rms_norm_grad(int type, const NormGradArgs &a, int num_sms, size_t ws_floats, cudaStream_t stream) {
    switch (type) {
        case SGEMM_IN_F32: return grad_for<ElF32>(a, num_sms, ws_floats, stream);
        case SGEMM_IN_BF16: return grad_for<ElBF16>(a, num_sms, ws_floats, stream);
        default: return grad_for<ElF16>(a, num_sms, ws_floats, stream);
    }
}

}  // namespace sg
