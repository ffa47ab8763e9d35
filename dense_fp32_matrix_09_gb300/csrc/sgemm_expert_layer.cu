// A whole mixture-of-experts layer for a few tokens, for sm_103a:
//   out_t = sum_j w_tj D_e act(U_e x_t),  e = ids_tj
// with U_e and D_e in int8, a scale a channel, and act = silu, or silu of one half of
// U_e's channels times the other.  Two kernels: the first makes the hidden values of every
// expert that some token asks for, the second multiplies them and adds up each token's.
// Their floor is the weights' way from HBM, which every asked expert's make once.
//
//  * up_stream_kernel, down_stream_kernel -- rows on 16-byte boundaries: the weights stream
//    through shared memory by TMA.  One token, four of 32 experts of 4096 x 2048, gated, BF16
//    (100 MB): 31 us, 15 of them HBM's, 5 the launches, 4 the routing and the first loads of
//    both kernels; 8 tokens (530 MB) 117 us, 4.6 TB/s.  The first kernel runs at 5 TB/s,
//    the second at 3.7: its instructions (half of the issue slots, by four warps a scheduler)
//    and what they wait for, no one thing among it.
//  * up_kernel, down_kernel -- any alignment: the weights straight into registers (the sizes
//    above less one 71 us; 8 tokens, width 3001, 1501 hidden 198).
//
// Every CTA works the routing out by itself: no kernel before, nothing on the host.  Up to 32
// choices are sorted by one warp, more (up to 1024) by a counting sort in shared memory.  The
// groups -- up to 8 * NT tokens of one expert -- are then dealt out in a fixed order.
//
// The products run on mma.sync (m16n8k16, FP32 sums): a tile of 16 channels x 8 tokens takes
// each weight once.  (The MMA's rate does not show: without the MMAs the kernels take 5 %
// less.  What does is the conversion, two instructions a weight.)  The order of k within an MMA
// is free, so a lane's 16 bytes are the k of four MMAs.  An int8 is exact in BF16 and in FP16;
// the tokens' elements go in as they are or, FP32, as sums of three BF16 values, exact as well (but
// from 3.396e38 on, which BF16 rounds to infinity, and what is below 2^-133 of tiny ones).
// The hidden values are kept as two BF16 values, 16 bits of fraction, and with FP32 rows as three:
// rounded to the rows' type they would halve the second kernel's loads and MMAs (8 tokens 126 us -> 116
// with stages of 16 rows), but also add as much error to the result as its own rounding does, and in FP16 they
// could overflow.  Within a warp sums run along k; the warps' sums, the experts' and the
// choices' are added in a fixed order in FP32.
#include <type_traits>

#include "context.h"
#include "device_common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "sgemm.h"
#include "tcgen05.cuh"

namespace sg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;  // (those that multiply)
constexpr int kChunk = 64;  // k of a step: 16 bytes of each of 16 channels from four lanes each
constexpr int kPad = 128;   // hidden rows are made longer to a multiple of it, with zeros
constexpr int kSlots = kLayerSlots;

template <class El>
struct Parts;  // 16-bit values that an element and a hidden value become, and the former's type
template <> struct Parts<ElBF16> { static constexpr int in = 1, hidden = 2; using Mma = ElBF16; };
template <> struct Parts<ElF16> { static constexpr int in = 1, hidden = 2; using Mma = ElF16; };  // (as they are, U in FP16)
template <> struct Parts<ElF32> { static constexpr int in = 3, hidden = 3; using Mma = ElBF16; };

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// x as a sum of P BF16 values, the largest first: x_p is what the ones before leave,
// rounded.  (Of an infinity or a NaN the first alone: a difference would be a NaN.)
template <int P>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&to)[P]) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
        to[p] = pack_bf16(x, y);
        if (p + 1 < P) {
            const float u = __uint_as_float(to[p] << 16), v = __uint_as_float(to[p] & 0xffff0000u);
            x = fabsf(u) < __int_as_float(0x7f800000) ? x - u : 0.f;
            y = fabsf(v) < __int_as_float(0x7f800000) ? y - v : 0.f;
        }
    }
}

// Four int8 to two pairs of FP16: 0x6400 + u is 1024 + u, and with u = b + 128 (the byte's
// sign bit flipped) less 1152 exactly b.  To two pairs of BF16: 0x4300 + u is 128 + u for u
// < 128, and 0x4380 is 256, so with a byte b's low seven bits u and its sign s, (0x4300 +
// u) - (0x4300 + 128 s) is u - 128 s, exactly b.
template <class Mma>
__device__ __forceinline__ void expand_int8(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (std::is_same<Mma, ElF16>::value) {
        w ^= 0x80808080u;
        auto less = [](uint32_t p) {
            const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&p), __half2{__ushort_as_half(0x6480), __ushort_as_half(0x6480)});
            return *reinterpret_cast<const uint32_t *>(&d);
        };
        lo = less(__byte_perm(w, 0x64646464u, 0x4140));
        hi = less(__byte_perm(w, 0x64646464u, 0x4342));
        return;
    }
    auto one = [](uint32_t p) {
        const uint32_t a = p & 0xff7fff7fu, s = p & 0xff80ff80u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&s));
        return *reinterpret_cast<const uint32_t *>(&d);
    };
    lo = one(__byte_perm(w, 0x43434343u, 0x4140));
    hi = one(__byte_perm(w, 0x43434343u, 0x4342));
}

template <class Mma>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
#define SG_MMA(T)                                                                                                       \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." T "." T ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};" \
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                                \
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1))
    if (std::is_same<Mma, ElF16>::value) SG_MMA("f16");
    else SG_MMA("bf16");
#undef SG_MMA
}

// The routing, as every CTA works it out.  Columns: the choices that count, sorted
// by expert, the earlier first.  A token that names an expert twice has one column
// with the sum of both weights.
struct Routing {
    struct Column {
        int token;
        float weight;
    } column[kSlots];
    struct alignas(8) Group {
        int expert;
        short first, cols;  // its columns: up to 8 * NT of one expert's
    } group[kSlots];
    int groups;
};

// What the sort needs meanwhile.
struct RouteScratch {
    int id[kSlots];              // the slot's expert, -1: none of its own
    float weight[kSlots];        // by slot
    int start[kMaxExperts + 1];  // an expert's columns, then its first
};

// Up to 32 choices: one warp, a choice a lane.
__device__ __forceinline__ void route_warp(Routing &r, const LayerArgs &a, int per_group) {
    const int lane = threadIdx.x, slots = a.tokens * a.choices;
    const int id0 = lane < slots ? __ldcg(a.ids + lane) : -1;
    const float w0 = lane < slots ? __ldcg(a.weights + lane) : 0.f;
    const int token = lane / a.choices;
    int id = static_cast<unsigned>(id0) < static_cast<unsigned>(a.experts) ? id0 : -1;
    float weight = 0.f;
    bool own = id >= 0;
    for (int q = 0; q < a.choices; ++q) {  // the token's choices, in their order
        const int at = (token * a.choices + q) & 31, other = __shfl_sync(0xffffffffu, id, at);
        const float w = __shfl_sync(0xffffffffu, w0, at);
        if (other == id && at < lane) own = false;
        if (other == id && at >= lane) weight += w;
    }
    if (!own) id = -1;
    // columns before this lane's, columns of its expert; then the experts' groups before its own
    int before = 0, same = 0, rank = 0;
#pragma unroll
    for (int q = 0; q < 32; ++q) {
        const int other = __shfl_sync(0xffffffffu, id, q);
        before += other >= 0 && other < id;
        same += other == id;
        rank += other == id && q < lane;
    }
    const bool leads = own && rank == 0;
    const int mine = leads ? (same + per_group - 1) / per_group : 0;
    int groups = 0, first_group = 0;
#pragma unroll
    for (int q = 0; q < 32; ++q) {
        const int n = __shfl_sync(0xffffffffu, mine, q), other = __shfl_sync(0xffffffffu, id, q);
        groups += n;
        if (other < id) first_group += n;
    }
    for (int k = 0; k < mine; ++k)
        r.group[first_group + k] = {id, static_cast<short>(before + k * per_group), static_cast<short>(min(per_group, same - k * per_group))};
    if (own) r.column[before + rank] = {token, weight};
    if (lane == 0) r.groups = groups;
}

template <int THREADS>
__device__ void route(Routing &r, RouteScratch &w, const LayerArgs &a, int per_group) {
    constexpr int kEach = (kSlots + THREADS - 1) / THREADS;
    const int slots = a.tokens * a.choices, tid = threadIdx.x;
    if (slots <= 32) {
        if (tid < 32) route_warp(r, a, per_group);
        __syncthreads();
        return;
    }
    for (int e = tid; e <= a.experts; e += THREADS) w.start[e] = 0;
    for (int s = tid; s < slots; s += THREADS) {
        const int id = __ldcg(a.ids + s);
        const float weight = __ldcg(a.weights + s);
        w.id[s] = static_cast<unsigned>(id) < static_cast<unsigned>(a.experts) ? id : -1;
        w.weight[s] = weight;
    }
    __syncthreads();
    // slots that repeat an earlier choice of their token add to its weight
    float mine[kEach];
    bool own[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int s = tid + k * THREADS;
        own[k] = s < slots && w.id[s] >= 0;
        mine[k] = 0.f;
        if (!own[k]) continue;
        const int t0 = s / a.choices * a.choices;
        for (int q = t0; q < s; ++q) own[k] = own[k] && w.id[q] != w.id[s];
        for (int q = s; q < t0 + a.choices; ++q)
            if (w.id[q] == w.id[s]) mine[k] += w.weight[q];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int s = tid + k * THREADS;
        if (s >= slots) continue;
        if (own[k]) atomicAdd(&w.start[w.id[s]], 1);
        else w.id[s] = -1;
    }
    __syncthreads();
    if (tid < 32) {  // counts to first columns; the groups
        int cols = 0, groups = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + tid, n = e < a.experts ? w.start[e] : 0, g = (n + per_group - 1) / per_group;
            int sn = n, sg = g;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int un = __shfl_up_sync(0xffffffffu, sn, d), ug = __shfl_up_sync(0xffffffffu, sg, d);
                if (tid >= d) {
                    sn += un;
                    sg += ug;
                }
            }
            if (e < a.experts) w.start[e] = cols + sn - n;
            for (int k = 0; k < g; ++k)
                r.group[groups + sg - g + k] = {e, static_cast<short>(cols + sn - n + k * per_group),
                                                static_cast<short>(min(per_group, n - k * per_group))};
            cols += __shfl_sync(0xffffffffu, sn, 31);
            groups += __shfl_sync(0xffffffffu, sg, 31);
        }
        if (tid == 0) r.groups = groups;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int s = tid + k * THREADS;
        if (s >= slots || w.id[s] < 0) continue;
        int c = w.start[w.id[s]];
        for (int q = 0; q < s; ++q) c += w.id[q] == w.id[s];
        r.column[c] = {s / a.choices, mine[k]};
    }
    __syncthreads();
}

// 16 bytes of a weight row from k on, on any address: the five aligned words that they lie in,
// shifted.  Words behind the row's last byte are zeros; bytes behind it within its last word
// may be anything (they meet elements that are zero), and lie in memory that the row's do.
__device__ __forceinline__ uint4 load_weights(const int8_t *row, int k, int K) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
    const uint32_t *p = reinterpret_cast<const uint32_t *>(at & ~static_cast<uintptr_t>(3));
    const int off = static_cast<int>(at & 3);  // of the first byte in the first word
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = (i < 4 || off) && k + 4 * i - off < K ? __ldcg(p + i) : 0u;
    const unsigned s = 8 * off;
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
}

// 32 bytes on a 32-byte boundary in one access: a sector, of which two of 16 bytes would
// each use half.
__device__ __forceinline__ void load32(const void *p, uint32_t (&to)[8]) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(to[0]), "=r"(to[1]), "=r"(to[2]), "=r"(to[3]), "=r"(to[4]), "=r"(to[5]), "=r"(to[6]), "=r"(to[7])
                 : "l"(p) : "memory");
}

// 16 elements of a token from k on, zeros behind its end, as they lie in memory and
// as P x 8 pairs of BF16.
template <class El>
struct Raw {
    alignas(16) typename El::T v[16];
};
template <class El, bool VEC>
__device__ __forceinline__ Raw<El> fetch_token(const typename El::T *row, int k, int K) {
    using T = typename El::T;
    constexpr int V = 16 / sizeof(T);
    Raw<El> r;
    if (VEC) {
#pragma unroll
        for (int e = 0; e < 16; e += 2 * V) {
            uint32_t w[8] = {};
            if (row && k + e < K) load32(row + k + e, w);
#pragma unroll
            for (int x = 0; x < 8; ++x) reinterpret_cast<uint32_t *>(r.v + e)[x] = w[x];
        }
    } else if (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 16; ++e) r.v[e] = k + e < K ? __ldca(row + k + e) : El::down(0.f);
    } else {  // the aligned words that they lie in, as load_weights
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
        const uint32_t *p = reinterpret_cast<const uint32_t *>(at & ~static_cast<uintptr_t>(3));
        const int off = static_cast<int>(at & 3) / 2;
        uint32_t w[9];
#pragma unroll
        for (int i = 0; i < 9; ++i) w[i] = (i < 8 || off) && k + 2 * i - off < K ? __ldca(p + i) : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t v = __funnelshift_r(w[i], w[i + 1], 16 * off);
            if (k + 2 * i + 1 >= K) v = k + 2 * i < K ? v & 0xffffu : 0u;
            reinterpret_cast<uint32_t *>(r.v)[i] = v;
        }
    }
    return r;
}
template <class El>
__device__ __forceinline__ void split_token(const Raw<El> &r, uint32_t (&to)[Parts<El>::in][8]) {
    constexpr int P = Parts<El>::in;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        uint32_t p[P];
        if (P == 1) p[0] = *reinterpret_cast<const uint32_t *>(r.v + 2 * e);
        else split2<P>(El::up(r.v[2 * e]), El::up(r.v[2 * e + 1]), p);
#pragma unroll
        for (int q = 0; q < P; ++q) to[q][e] = p[q];
    }
}

// acc += 16 channels x 64 k (lo: channel g, hi: channel g + 8) times 8 tokens.  An MMA truncates its sum:
// FP32 tokens' 64 k are summed by themselves, the low parts first, and added with rounding to nearest
// (a chain of 12 MMAs every 64 k: errors of 2e-6 to 4e-6 of the result where FP32 products on the
// CUDA cores have 2e-7 to 4e-7).
template <class Mma, int P>
__device__ __forceinline__ void multiply(float (&acc)[4], const uint32_t (&a)[4][4], const uint32_t (&x)[P][8]) {
    float sum[4] = {};
    float(&to)[4] = P == 3 ? sum : acc;
#pragma unroll
    for (int q = 0; q < 4 * P; ++q) {
        const int s = P == 3 ? q % 4 : q / P, p = P == 3 ? P - 1 - q / 4 : P - 1 - q % P;
        mma16<Mma>(to, a[s], x[p][2 * s], x[p][2 * s + 1]);
    }
    if (P == 3) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += sum[j];
    }
}
template <class Mma>
__device__ __forceinline__ void expand_rows(const uint4 &lo, const uint4 &hi, uint32_t (&a)[4][4]) {
    const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        expand_int8<Mma>(l[s], a[s][0], a[s][2]);
        expand_int8<Mma>(h[s], a[s][1], a[s][3]);
    }
}

// The scales of the channels that a lane has of an MMA tile: g, and the one in its lower half.
template <bool GATED>
__device__ __forceinline__ void hidden_scales(const LayerArgs &a, int e, int f0, int g, float (&to)[2]) {
    const int fl = f0 + g, fh = GATED ? fl : fl + 8;
    const float *scale = a.up_scale + static_cast<long long>(e) * a.up_rows;
    to[0] = fl < a.hidden ? __ldca(scale + fl) : 0.f;
    to[1] = fh < a.hidden ? __ldca(scale + fh + (GATED ? a.hidden : 0)) : 0.f;
}

// The hidden values of 8 tokens from their sums: s.x, s.y channel g of tokens 2t and 2t + 1, s.z
// and s.w of the MMA's lower channel.  Channels behind the last hidden one are written as zeros.
template <bool GATED, int PH>
__device__ __forceinline__ void write_hidden(const LayerArgs &a, int first, int cols, int f0, int n, int g, int t, const float4 &s,
                                             const float (&scale)[2]) {
    const int fl = f0 + g, fh = GATED ? fl : fl + 8;
    const bool in_l = fl < a.hidden, in_h = fh < a.hidden;
    auto silu = [](float v) { return v / (1.f + expf(-v)); };
    auto put = [&](int col, int f, float v) {
        if (col >= cols || f >= a.hidden_ld) return;
        uint32_t p[PH];
        split2<PH>(v, 0.f, p);
#pragma unroll
        for (int q = 0; q < PH; ++q)
            a.h[q * a.h_part + static_cast<long long>(first + col) * a.hidden_ld + f] = static_cast<uint16_t>(p[q]);
    };
    const float y0 = silu(s.x * scale[0]), y1 = silu(s.y * scale[0]);
    put(n * 8 + 2 * t, fl, in_l ? GATED ? y0 * (s.z * scale[1]) : y0 : 0.f);
    put(n * 8 + 2 * t + 1, fl, in_l ? GATED ? y1 * (s.w * scale[1]) : y1 : 0.f);
    if (!GATED) {
        put(n * 8 + 2 * t, fh, in_h ? silu(s.z * scale[1]) : 0.f);
        put(n * 8 + 2 * t + 1, fh, in_h ? silu(s.w * scale[1]) : 0.f);
    }
}

// 16 hidden values from k on, PH x 8 pairs of BF16 (row NULL, a column that a group does not have:
// zeros; what a lane fetches in vain takes its share of the SM's 128 bytes a cycle).
template <int PH>
__device__ __forceinline__ void load_hidden(const uint16_t *row, long long part, int k, uint32_t (&to)[PH][8]) {
#pragma unroll
    for (int q = 0; q < PH; ++q) {
        if (row) load32(row + q * part + k, to[q]);
        else
#pragma unroll
            for (int x = 0; x < 8; ++x) to[q][x] = 0u;
    }
}

// A warp's sums of a group, scaled, to its own sums of the tokens.
constexpr int kOutPitch = 17;
template <int NT>
__device__ __forceinline__ void add_out(const Routing &r, float *mine, int first, int cols, int g, int t, float sl, float sh,
                                        const float (&acc)[NT][4], int pitch = kOutPitch) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = n * 8 + 2 * t + j;
            if (col >= cols) continue;
            const Routing::Column c = r.column[first + col];
            float *to = mine + c.token * pitch;
            to[g] = fmaf(acc[n][j] * sl, c.weight, to[g]);
            to[g + 8] = fmaf(acc[n][2 + j] * sh, c.weight, to[g + 8]);
        }
    __syncwarp();
}

// ---- any alignment: the weights straight into registers --------------------------------
constexpr int kAhead = 4;  // chunks whose loads are in flight

// hidden[part][column][f] = act(U x) of every group; an item is a group and 16 rows of
// U: with a gate 8 channels of it and the 8 that it goes with, in the MMA's upper and
// lower rows, so that one lane has both.  `share` warps of the CTA split an item's K.
template <class El, int NT, bool GATED>
__global__ void __launch_bounds__(kThreads, 2) up_kernel(const LayerArgs a, int share) {
    using T = typename El::T;
    using Mma = typename Parts<El>::Mma;
    constexpr int P = Parts<El>::in, PH = Parts<El>::hidden, kCh = GATED ? 8 : 16;
    __shared__ Routing r;
    __shared__ RouteScratch scratch;
    __shared__ float4 sums[kWarps][NT][32];
    griddep_wait();
    griddep_launch_dependents();
    route<kThreads>(r, scratch, a, 8 * NT);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int tiles = a.hidden_ld / kCh, teams = kWarps / share, team = warp / share, part = warp % share;
    const long long items = static_cast<long long>(r.groups) * tiles;
    const int chunks = (a.width + kChunk - 1) / kChunk;
    for (long long i0 = static_cast<long long>(blockIdx.x) * teams; i0 < items; i0 += static_cast<long long>(gridDim.x) * teams) {
        const long long item = i0 + team;
        const bool live = item < items;
        const int group = live ? static_cast<int>(item / tiles) : 0, f0 = live ? static_cast<int>(item % tiles) * kCh : 0;
        const Routing::Group here = r.group[group];
        const int e = here.expert, first = here.first, cols = here.cols;
        const int fl = f0 + g, fh = GATED ? fl : fl + 8;  // the hidden channels of the lane's rows
        const bool in_l = live && fl < a.hidden, in_h = live && fh < a.hidden;
        const long long row_l = static_cast<long long>(e) * a.up_rows + (in_l ? fl : 0);
        const long long row_h = static_cast<long long>(e) * a.up_rows + (in_h ? fh : 0) + (GATED ? a.hidden : 0);
        const int8_t *ul = a.up + row_l * a.width, *uh = a.up + row_h * a.width;
        const T *x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            x[n] = static_cast<const T *>(a.X) + static_cast<long long>(r.column[first + min(n * 8 + g, cols - 1)].token) * a.ldx;
        float acc[NT][4] = {};
        for (int c0 = part; c0 < chunks; c0 += share * kAhead) {
            uint4 wl[kAhead], wh[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int at = (c0 + k * share) * kChunk + t * 16;
                wl[k] = load_weights(ul, at, in_l ? a.width : 0);
                wh[k] = load_weights(uh, at, in_h ? a.width : 0);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (c0 + k * share >= chunks) break;
                const int at = (c0 + k * share) * kChunk + t * 16;
                uint32_t w[4][4];
                expand_rows<Mma>(wl[k], wh[k], w);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n * 8 >= cols) break;
                    uint32_t v[P][8];
                    split_token<El>(fetch_token<El, false>(x[n], at, a.width), v);
                    multiply<Mma, P>(acc[n], w, v);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) sums[warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
        __syncthreads();
        if (live) {
            for (int n = part; n < NT && n * 8 < cols; n += share) {
                float4 s = sums[team * share][n][lane];
                for (int q = 1; q < share; ++q) {
                    const float4 v = sums[team * share + q][n][lane];
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
                float scale[2];
                hidden_scales<GATED>(a, e, f0, g, scale);
                write_hidden<GATED, PH>(a, first, cols, f0, n, g, t, s, scale);
            }
        }
        __syncthreads();
    }
}

// out: an item is 16 channels of every token; the CTA's warps take consecutive runs of
// (group, chunk of k) pairs.  At the end of its run or of a group a warp adds what it
// has, scaled, to its own sums of the tokens.
template <class El, int NT>
__global__ void __launch_bounds__(kThreads, 2) down_kernel(const LayerArgs a) {
    constexpr int PH = Parts<El>::hidden;
    extern __shared__ float out_sums[];  // [warp][token][kOutPitch]
    __shared__ Routing r;
    __shared__ RouteScratch scratch;
    // (the routing and the sums touch nothing that the kernel before writes, and that
    // one has waited for what came before it)
    for (int k = threadIdx.x; k < kWarps * a.tokens * kOutPitch; k += kThreads) out_sums[k] = 0.f;
    route<kThreads>(r, scratch, a, 8 * NT);
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int chunks = a.hidden_ld / kChunk;
    const long long units = static_cast<long long>(r.groups) * chunks;
    const long long u_first = units * warp / kWarps, u_last = units * (warp + 1) / kWarps;
    float *mine = out_sums + warp * a.tokens * kOutPitch;
    const int d0 = blockIdx.x * 16, dl = d0 + g, dh = d0 + g + 8;
    const bool in_l = dl < a.width, in_h = dh < a.width;
    for (long long u = u_first; u < u_last;) {
        const int group = static_cast<int>(u / chunks), c_first = static_cast<int>(u % chunks);
        const int c_last = static_cast<int>(min(static_cast<long long>(chunks), c_first + (u_last - u)));
        u += c_last - c_first;
        const Routing::Group here = r.group[group];
        const int e = here.expert, first = here.first, cols = here.cols;
        const long long row_l = static_cast<long long>(e) * a.width + (in_l ? dl : 0), row_h = static_cast<long long>(e) * a.width + (in_h ? dh : 0);
        const int8_t *wl = a.down + row_l * a.hidden, *wh = a.down + row_h * a.hidden;
        const uint16_t *h[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) h[n] = a.h + static_cast<long long>(first + min(n * 8 + g, cols - 1)) * a.hidden_ld;
        float acc[NT][4] = {};
        for (int c0 = c_first; c0 < c_last; c0 += kAhead) {
            uint4 vl[kAhead], vh[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int at = (c0 + k) * kChunk + t * 16;
                vl[k] = load_weights(wl, at, in_l && c0 + k < c_last ? a.hidden : 0);
                vh[k] = load_weights(wh, at, in_h && c0 + k < c_last ? a.hidden : 0);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (c0 + k >= c_last) break;
                const int at = (c0 + k) * kChunk + t * 16;
                uint32_t w[4][4];
                expand_rows<ElBF16>(vl[k], vh[k], w);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n * 8 >= cols) break;
                    uint32_t v[PH][8];
                    load_hidden<PH>(h[n], a.h_part, at, v);
                    multiply<ElBF16, PH>(acc[n], w, v);
                }
            }
        }
        const float sl = in_l ? __ldca(a.down_scale + row_l) : 0.f, sh = in_h ? __ldca(a.down_scale + row_h) : 0.f;
        add_out<NT>(r, mine, first, cols, g, t, sl, sh, acc);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.tokens * 16; k += kThreads) {
        const int token = k / 16, d = d0 + k % 16;
        if (d >= a.width) continue;
        float sum = 0.f;
        for (int w = 0; w < kWarps; ++w) sum += out_sums[(w * a.tokens + token) * kOutPitch + k % 16];
        static_cast<typename El::T *>(a.out)[token * a.ldo + d] = El::down(sum);
    }
}

// ---- rows on 16-byte boundaries: the weights through shared memory --------------------
// One lane streams the weights of all the CTA's items, one behind the other, into a ring
// of stages of 1024 bytes of 32 or 16 rows by TMA, so that as many bytes are on their way while the others add up or
// write as at any other time.  Sixteen warps take a 64-byte column of every 1024 bytes;
// warps of their own add up the columns' sums and write the hidden values, their scales
// fetched ahead, so that the ring is not held up.
constexpr int kSeg = 1024;
constexpr int kTakers = kSeg / kChunk;
template <class El, int NT>
struct StreamCfg {
    static constexpr int kUpStages = NT <= 2 ? 4 : 3;              // of 32 rows
    static constexpr int kSums = NT <= 2 ? 2 : 1;                  // sets of sums
    static constexpr int kSumBytes = kTakers * 2 * NT * 512;       // of a set
    static constexpr int kUpThreads = (kTakers + 1 + NT) * 32, kDownThreads = (kTakers + 1) * 32;
    static constexpr int kUpRing = 1024 + kUpStages * 32 * kSeg, kUpSmem = kUpRing + kSums * kSumBytes;
    // Hidden values of two of a warp's stages in shared memory, where that has room for them: of
    // four columns.  What an expert has beyond is read where it is needed (with all eight kept the
    // ring had half the stages: 8 tokens on the same experts 58 us against 54, on all of
    // eight experts 86 against 73; on experts of their own 126 against 130, before the 32-row stages).
    static constexpr bool kHeld = NT == 1 && Parts<El>::hidden == 2;
    static constexpr int kHeldColumns = 4;
    static constexpr int kHeldPiece = kHeldColumns * 64, kHeldBytes = kHeld ? 4 * Parts<El>::hidden * kHeldPiece : 0;  // of a stage
    static constexpr int kMostTiles = NT == 1 ? 2 : 1;       // of 16 channels, of an item of down_stream_kernel
    static constexpr int kDownStages = NT == 1 ? 8 : 6;  // of 16 rows, or half as many of 32; half of them a team's
    static constexpr int kDownRing = 1024 + kDownStages * 16 * kSeg;
    static constexpr int down_smem(int tokens, int tiles) { return kDownRing + kTakers * (2 * kHeldBytes + tokens * (tiles * 16 + 1) * 4); }
    static_assert(sizeof(RouteScratch) <= 2 * 16 * kSeg, "the routing's scratch lies in the ring");
    // the most tokens of a call on this configuration; the routing takes less than 17 KiB
    static_assert(down_smem(NT == 1 ? 8 : kLayerTokens, kMostTiles) <= 232448 - 17408 && kUpSmem <= 232448 - 17408, "shared memory");
};
constexpr int kPrefetch = 64;  // boxes of 2 KiB
struct StreamShared {
    uint64_t full[8], empty[8], sums_full[2], sums_empty[2];
    int abort;
};

// First of the 16 k of a stage that a lane of a warp takes (see Stream::take).
__device__ __forceinline__ int lane_k(int warp, int t) { return warp / 2 * 128 + (2 * t + (warp & 1)) * 16; }

// Where a stage has piece `piece` (16 bytes) of column `column` (128 bytes) of a row.  With
// pieces 0, 2, 4, 6 or 1, 3, 5, 7 in a row's four lanes the swizzle puts any two rows that
// follow one another on all banks.
__device__ __forceinline__ int place_of(int row, int column, int piece) {
    return row / 16 * (16 * kSeg) + column * 2048 + row % 16 * 128 + ((piece ^ (row & 7)) * 16);
}

template <int STAGES, int ROWS>
struct Stream {
    static constexpr int kBytes = ROWS * kSeg;
    uint8_t *ring;
    StreamShared *sh;
    uint64_t *full, *empty;  // its slots' barriers
    int *status;
    int s = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step() {
        if (++s == STAGES) {
            s = 0;
            round ^= 1u;
        }
    }
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*static_cast<volatile int *>(&sh->abort)) return false;
        if (mbar_wait(bar, parity, status)) return true;
        *static_cast<volatile int *>(&sh->abort) = 1;
        return false;
    }
    // The producing lane: waits for its copies in flight.  Slot s still holds the last round's stage,
    // the slots before it this round's (one that was never loaded stands at its first round).
    __device__ __forceinline__ void drain() {
        for (int k = 0; k < STAGES; ++k, step()) mbar_wait(&full[s], round ^ 1u, status);
    }
    // The producing lane: a stage of 16 rows from `row0` and, of 32, 16 from `row1`; false after a
    // wait that ran out (drain is then due).
    __device__ __forceinline__ bool put(const CUtensorMap *map, int at, int row0, int row1) {
        if (!wait(&empty[s], round ^ 1u)) return false;
        mbar_arrive_expect_tx(&full[s], kBytes);
        uint8_t *to = ring + s * kBytes;
#pragma unroll
        for (int c = 0; c < kSeg / 128; ++c) {
            tma_load_2d(to + c * 2048, map, &full[s], at + c * 128, row0);
            if (ROWS == 32) tma_load_2d(to + kBytes / 2 + c * 2048, map, &full[s], at + c * 128, row1);
        }
        step();
        return true;
    }
    // A taking warp: the next stage has landed.
    __device__ __forceinline__ bool get() { return __all_sync(0xffffffffu, wait(&full[s], round)); }
    // The lane's 16 bytes of two rows of the stage, `lo` and `hi` bytes from its start (place_of).
    __device__ __forceinline__ void take(int lo_at, int hi_at, uint4 &lo, uint4 &hi) const {
        const uint8_t *at = ring + s * kBytes;
        lo = *reinterpret_cast<const uint4 *>(at + lo_at);
        hi = *reinterpret_cast<const uint4 *>(at + hi_at);
    }
    __device__ __forceinline__ void done(int lane) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        step();
    }
};

// The barriers of RINGS rings, one behind the other in shared memory, each read by `takers` warps;
// the whole CTA, which meets at a barrier afterwards.
template <int RINGS, int STAGES, int ROWS>
__device__ __forceinline__ void open_streams(Stream<STAGES, ROWS> (&q)[RINGS], uint8_t *smem, StreamShared *sh, int writers, int takers, int *status) {
    static_assert(RINGS * STAGES <= 8, "barriers");
    if (threadIdx.x == 0) {
        for (int s = 0; s < RINGS * STAGES; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], takers);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh->sums_full[s], kTakers);
            mbar_init(&sh->sums_empty[s], writers);
        }
        sh->abort = 0;
        fence_barrier_init();
    }
    smem += (1024u - (smem_u32(smem) & 1023u)) & 1023u;
#pragma unroll
    for (int r = 0; r < RINGS; ++r) {
        q[r].ring = smem + r * STAGES * Stream<STAGES, ROWS>::kBytes;
        q[r].sh = sh;
        q[r].full = sh->full + r * STAGES;
        q[r].empty = sh->empty + r * STAGES;
        q[r].status = status;
    }
}

// As up_kernel, an item 32 rows of U: the tokens' elements are then fetched and split once
// for two MMA tiles.
template <class El, int NT, bool GATED>
__global__ void __launch_bounds__(StreamCfg<El, NT>::kUpThreads, 1)
up_stream_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap next_map, const LayerArgs a) {
    using T = typename El::T;
    using Mma = typename Parts<El>::Mma;
    using Cf = StreamCfg<El, NT>;
    constexpr int P = Parts<El>::in, PH = Parts<El>::hidden, kCh = GATED ? 16 : 32;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ StreamShared shared;
    __shared__ Routing r;
    Stream<Cf::kUpStages, 32> streams[1], &q = streams[0];
    open_streams(streams, smem, &shared, NT, kTakers, a.status);
    float4 *sums = reinterpret_cast<float4 *>(smem + Cf::kUpRing);  // [set][warp][tile][n][lane]
    griddep_wait();
    griddep_launch_dependents();
    route<Cf::kUpThreads>(r, *reinterpret_cast<RouteScratch *>(q.ring), a, 8 * NT);  // (before anything lands there)
    tc::fence_proxy_async_smem();
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int tiles = (a.hidden_ld + kCh - 1) / kCh, items = r.groups * tiles, segs = (a.width + kSeg - 1) / kSeg;
    if (warp == kTakers) {
        if (lane > 0) return;
        for (int i = blockIdx.x; i < items; i += gridDim.x) {
            // (a tile behind the last hidden channel reads the rows that follow, and writes zeros)
            const int row = static_cast<int>(r.group[i / tiles].expert * a.up_rows) + i % tiles * kCh;
            for (int s = 0; s < segs; ++s)
                if (!q.put(&map, s * kSeg, row, row + (GATED ? a.hidden : 16))) {
                    q.drain();
                    return;
                }
        }
        // What this CTA's successor in down_stream_kernel reads first is fetched into L2 while
        // it starts (its weights may be: see there).  The CTA ends no earlier than this
        // loop, so that a load or a division in it shows: the expert looked up for every box, 1
        // token 33 us against 31; none fetched 31.5, 128 boxes 33.8.
        int left = kPrefetch;
        const int d0 = static_cast<int>(blockIdx.x) * a.channels;
        if (d0 >= a.width) return;
        for (int group = 0; group < r.groups; ++group) {
            const int row = r.group[group].expert * a.width + d0;
            for (int s = 0; s < a.hidden; s += 128) {
                if (left <= 0) return;
                tma_prefetch_2d(&next_map, s, row);
                if (a.channels > 16) tma_prefetch_2d(&next_map, s, row + a.channels - 16);
                left -= a.channels > 16 ? 2 : 1;
            }
        }
        return;
    }
    if (warp > kTakers) {
        // ------------------------------------------------ 8 tokens' sums to hidden values
        const int n = warp - kTakers - 1;
        int set = 0;
        uint32_t round = 0;
        for (int i = blockIdx.x; i < items; i += gridDim.x) {
            const int group = i / tiles, f0 = i % tiles * kCh;
            const Routing::Group here = r.group[group];
            const int e = here.expert, first = here.first, cols = here.cols;
            float scale[2][2];
            if (n * 8 < cols)
#pragma unroll
                for (int m = 0; m < 2; ++m) hidden_scales<GATED>(a, e, f0 + m * (kCh / 2), g, scale[m]);
            if (!__all_sync(0xffffffffu, q.wait(&shared.sums_full[set], round))) return;
            float4 s[2] = {};
            if (n * 8 < cols)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int p = 0; p < kTakers; ++p) {
                        const float4 v = sums[(((set * kTakers + p) * 2 + m) * NT + n) * 32 + lane];
                        s[m].x += v.x;
                        s[m].y += v.y;
                        s[m].z += v.z;
                        s[m].w += v.w;
                    }
            __syncwarp();
            if (lane == 0) mbar_arrive(&shared.sums_empty[set]);
            if (n * 8 < cols)
#pragma unroll
                for (int m = 0; m < 2; ++m) write_hidden<GATED, PH>(a, first, cols, f0 + m * (kCh / 2), n, g, t, s[m], scale[m]);
            if (++set == Cf::kSums) {
                set = 0;
                round ^= 1u;
            }
        }
        return;
    }
    const int k0 = lane_k(warp, t);  // the lane's k of a stage
    const int lo_at = place_of(g, warp / 2, 2 * t + (warp & 1)), hi_at = place_of(GATED ? 16 + g : 8 + g, warp / 2, 2 * t + (warp & 1));
    int set = 0;
    uint32_t round = 0;
    // the token row of the lane's column of an item's first eight
    auto row_of = [&](int i) {
        const Routing::Group of = r.group[i / tiles];
        return g < of.cols ? static_cast<const T *>(a.X) + static_cast<long long>(r.column[of.first + g].token) * a.ldx : nullptr;
    };
    // One stage ahead: the elements come from L2 where L1 does not hold them, and a warp that
    // waits for them holds the ring up.
    Raw<El> ahead{};
    if (static_cast<int>(blockIdx.x) < items) ahead = fetch_token<El, true>(row_of(blockIdx.x), k0, a.width);
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
        const bool another = i + static_cast<int>(gridDim.x) < items;
        const T *after = another ? row_of(i + gridDim.x) : nullptr;
        const int group = i / tiles;
        const Routing::Group here = r.group[group];
        const int e = here.expert, first = here.first, cols = here.cols;
        const T *x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            x[n] = n * 8 + g < cols ? static_cast<const T *>(a.X) + static_cast<long long>(r.column[first + n * 8 + g].token) * a.ldx : nullptr;
        float acc[2][NT][4] = {};
        for (int s = 0; s < segs; ++s) {
            const int k = s * kSeg + k0;
            uint32_t v[P][8];
            split_token<El>(ahead, v);
            if (s + 1 < segs) ahead = fetch_token<El, true>(x[0], k + kSeg, a.width);
            else if (another) ahead = fetch_token<El, true>(after, k0, a.width);
            if (!q.get()) return;
            if (k - 2 * t * 16 < a.width) {  // (the warp's first k)
                uint32_t w[2][4][4];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint4 lo, hi;
                    q.take(lo_at + (GATED ? 1024 : 16 * kSeg) * m, hi_at + (GATED ? 1024 : 16 * kSeg) * m, lo, hi);
                    expand_rows<Mma>(lo, hi, w[m]);
                    multiply<Mma, P>(acc[m][0], w[m], v);
                }
#pragma unroll
                for (int n = 1; n < NT; ++n) {
                    if (n * 8 >= cols) break;
                    split_token<El>(fetch_token<El, true>(x[n], k, a.width), v);
#pragma unroll
                    for (int m = 0; m < 2; ++m) multiply<Mma, P>(acc[m][n], w[m], v);
                }
            }
            q.done(lane);
        }
        if (!__all_sync(0xffffffffu, q.wait(&shared.sums_empty[set], round ^ 1u))) return;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (n * 8 < cols)
                    sums[(((set * kTakers + warp) * 2 + m) * NT + n) * 32 + lane] = make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&shared.sums_full[set]);
        if (++set == Cf::kSums) {
            set = 0;
            round ^= 1u;
        }
    }
}

// 16 bytes to shared memory, past L1 and without a register.
__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// As down_kernel, with a grid of as many CTAs as run at once; a stage is 16 MT channels' rows of up
// to 1024 hidden values of a group.  With MT = 2 a hidden value that a lane has fetched meets 32
// rows, and an item has as many channels as fall to an SM in a round of all: of 4096 on 152 SMs
// 27 each in 152 items, not 1.7 rounds of 16 (8 tokens, 4 of 32 experts, 4096 x 2048: 130 -> 117 us).
// The second tile's rows end with the item's; those that both tiles have come from L2 twice.  Two teams of eight warps take the groups in turn, 128
// bytes of a row each: while one team's loads, sums and waits take their time, the other
// multiplies (sixteen warps on every stage, 64 bytes each: 75 us for a batch of 8 tokens,
// most of it instructions that are not the product's).  A lane fetches the hidden values of
// its team's stages ahead, two where shared memory has room for them (one, in registers: 62 us
// for that batch), and the scales of its next group when it begins one.
template <class El, int NT, int MT>
__global__ void __launch_bounds__(StreamCfg<El, NT>::kDownThreads, 1) down_stream_kernel(const __grid_constant__ CUtensorMap map, const LayerArgs a) {
    using Cf = StreamCfg<El, NT>;
    constexpr int PH = Parts<El>::hidden, S = Cf::kDownStages / 2 / MT, kPitch = MT * 16 + 1;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ StreamShared shared;
    __shared__ Routing r;
    // A ring for each team: one that skipped the other's stages in a common ring could take the
    // parity of a slot's round before last for its own.
    Stream<S, MT * 16> streams[2];
    open_streams(streams, smem, &shared, 1, kTakers / 2, a.status);
    float *out_sums = reinterpret_cast<float *>(smem + Cf::kDownRing + kTakers * 2 * Cf::kHeldBytes);  // [warp][token][kPitch]
    for (int k = threadIdx.x; k < kTakers * a.tokens * kPitch; k += Cf::kDownThreads) out_sums[k] = 0.f;
    route<Cf::kDownThreads>(r, *reinterpret_cast<RouteScratch *>(streams[0].ring), a, 8 * NT);  // (before anything lands there)
    tc::fence_proxy_async_smem();
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    // An item's second tile ends with its channels: those that the first has too are left there.
    const int channels = MT == 1 ? 16 : a.channels, second = channels - 16;
    const int items = (a.width + channels - 1) / channels, step = static_cast<int>(gridDim.x), groups = r.groups;
    if (warp == kTakers) {
        if (lane > 0) return;
        // (the weights: the kernel before does not write them, and has waited for what came
        // before it, so that they may be under way before its end)
        int turn = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < items && ok; i += step)
            for (int group = 0; group < groups && ok; ++group, turn ^= 1)
                for (int k = 0; k < a.hidden && ok; k += kSeg) {
                    const int row = r.group[group].expert * a.width + i * channels;
                    ok = turn ? streams[1].put(&map, k, row, row + second) : streams[0].put(&map, k, row, row + second);
                }
        if (!ok) {
            streams[0].drain();
            streams[1].drain();
        }
        return;
    }
    const int team = warp / (kTakers / 2), column = warp % (kTakers / 2);  // of 128 bytes
    Stream<S, MT * 16> q = team ? streams[1] : streams[0];
    const int place[2] = {place_of(g, column, 2 * t), place_of(g, column, 2 * t + 1)};
    const bool idle = column * 128 >= a.hidden;                            // (short rows leave columns out)
    float *mine = out_sums + warp * a.tokens * kPitch;
    bool ok = true;
    // The team's groups: every other one, counted over all items, so that both have as many.
    struct Cursor {
        int group, item;
    };
    auto settle = [&](Cursor &c) {
        while (c.group >= groups && c.item < items) {
            c.group -= groups;
            c.item += step;
        }
        return c.item < items;
    };
    // The channels' scales of the next group, on their way while one is multiplied (the first
    // before the kernel before has ended, which does not write them).
    float next_l[MT] = {}, next_h[MT] = {};
    Cursor coming{team, static_cast<int>(blockIdx.x)};
    auto scales = [&]() {
        if (!settle(coming)) return;
        const float *scale = a.down_scale + static_cast<long long>(r.group[coming.group].expert) * a.width;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int d = coming.item * channels + m * second + g;
            next_l[m] = d < a.width ? __ldca(scale + d) : 0.f;
            next_h[m] = d + 8 < a.width ? __ldca(scale + d + 8) : 0.f;
        }
        coming.group += 2;
    };
    if (groups > 0) scales();
    griddep_wait();
    griddep_launch_dependents();
    // The lane's 32 hidden values of the team's stages, in the groups' first eight columns: two
    // stages ahead in shared memory, or the next one's in registers.
    const uint16_t *h_lane = a.h + column * 128 + t * 32;
    uint8_t *held = smem + Cf::kDownRing + warp * (2 * Cf::kHeldBytes) + lane * 16;
    uint32_t ahead[2][PH][8] = {};
    Cursor fetched{team, static_cast<int>(blockIdx.x)};
    int f_k = 0, f_slot = 0, slot = 0;
    auto fetch = [&]() {
        if (settle(fetched)) {
            const Routing::Group of = r.group[fetched.group];
            if (g < of.cols && (!Cf::kHeld || g < Cf::kHeldColumns) && f_k + column * 128 < a.hidden) {
                const uint16_t *h = h_lane + (static_cast<long long>(of.first + g) * a.hidden_ld + f_k);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (!Cf::kHeld) load_hidden<PH>(h + c * 16, a.h_part, 0, ahead[c]);
                    else
#pragma unroll
                        for (int p = 0; p < PH; ++p)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                copy_async16(held + f_slot * Cf::kHeldBytes + ((c * PH + p) * 2 + x) * Cf::kHeldPiece, h + p * a.h_part + c * 16 + x * 8);
                }
            }
            f_k += kSeg;
            if (f_k >= a.hidden) {
                f_k = 0;
                fetched.group += 2;
            }
        }
        f_slot ^= 1;
        if (Cf::kHeld) copy_async_commit();
    };
    if (groups > 0) {
        fetch();
        if (Cf::kHeld) fetch();
    }
    int turn = team;  // 0: the group is the team's
    for (int i = blockIdx.x; i < items; i += step) {
        for (int n_group = 0; n_group < groups; ++n_group, turn ^= 1) {
            if (turn) continue;
            const Routing::Group now = r.group[n_group];
            float sl[MT], sh[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                sl[m] = next_l[m];
                sh[m] = next_h[m];
            }
            scales();
            float acc[MT][NT][4] = {}, half[4] = {};  // (two chains, of the tiles or of a tile's halves: an MMA waits for the one before it)
            for (int k = 0; k < a.hidden; k += kSeg) {
                ok = ok && q.get();  // (after a wait that ran out the warps still meet at the barriers)
                if (!ok) break;
                if (Cf::kHeld) copy_async_wait<1>();
                if (k + column * 128 < a.hidden) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (Cf::kHeld && g >= Cf::kHeldColumns) {
                            if (g < now.cols) load_hidden<PH>(h_lane + static_cast<long long>(now.first + g) * a.hidden_ld, a.h_part, k + c * 16, ahead[c]);
                        } else if (Cf::kHeld)
#pragma unroll
                            for (int p = 0; p < PH; ++p)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
                                    *reinterpret_cast<uint4 *>(&ahead[c][p][4 * x]) = *reinterpret_cast<const uint4 *>(held + slot * Cf::kHeldBytes + ((c * PH + p) * 2 + x) * Cf::kHeldPiece);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            uint4 lo, hi;
                            q.take(place[c] + m * (16 * kSeg), place[c] + m * (16 * kSeg) + 1024, lo, hi);
                            uint32_t w[4][4];
                            expand_rows<ElBF16>(lo, hi, w);
                            multiply<ElBF16, PH>(MT == 1 && c ? half : acc[m][0], w, ahead[c]);
#pragma unroll
                            for (int n = 1; n < NT; ++n) {
                                if (n * 8 >= now.cols) break;
                                uint32_t v[PH][8];
                                load_hidden<PH>(n * 8 + g < now.cols ? h_lane + static_cast<long long>(now.first + n * 8 + g) * a.hidden_ld : nullptr, a.h_part, k + c * 16, v);
                                multiply<ElBF16, PH>(acc[m][n], w, v);
                            }
                        }
                    }
                }
                slot ^= 1;
                q.done(lane);
                fetch();
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[m][0][c] += half[c];
                if (!idle) add_out<NT>(r, mine + m * 16, now.first, now.cols, g, t, sl[m], sh[m], acc[m], kPitch);
            }
        }
        named_barrier_sync(1, kTakers * 32);
        for (int k = threadIdx.x; k < a.tokens * channels; k += kTakers * 32) {
            const int token = k / channels, at = k - token * channels, d = i * channels + at;
            const int slot = MT == 1 || at < 16 ? at : at - second + 16;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kTakers; ++w) {
                float &part = out_sums[(w * a.tokens + token) * kPitch + slot];
                sum += part;
                part = 0.f;
            }
            if (ok && d < a.width) static_cast<typename El::T *>(a.out)[token * a.ldo + d] = El::down(sum);
        }
        named_barrier_sync(1, kTakers * 32);
    }
    if (Cf::kHeld) copy_async_wait<0>();  // no copy outlives the CTA
}

// The weights' rows, boxes of 128 bytes x 16 rows with the 128-byte swizzle.
struct LayerMaps {
    CUtensorMap up, down;
};
constexpr long long kMostRows = (1ll << 31) - 64;  // coordinates are ints

template <class El, int NT>
cudaError_t layer_typed(LayerArgs a, bool boundaries, const LayerMaps &m, int num_sms, cudaStream_t stream) {
    // (the groups are on the device: so many there are at most)
    const long long slots = static_cast<long long>(a.tokens) * a.choices, asked = slots < a.experts ? slots : a.experts;
    auto grid = [](long long ctas, long long most) { return dim3(static_cast<unsigned>(ctas < 1 ? 1 : ctas < most ? ctas : most)); };
    if (boundaries) {
        using Cf = StreamCfg<El, NT>;
        const int kCh = a.gated ? 16 : 32;
        // An item of the second product: 16 channels or, where the SMs would take more than one
        // such each, up to 32, as many in each item of a round of all SMs.
        const int rounds = (a.width + 32 * num_sms - 1) / (32 * num_sms);
        const bool wide = Cf::kMostTiles == 2 && a.width > 16 * num_sms;
        a.channels = wide ? (a.width + rounds * num_sms - 1) / (rounds * num_sms) : 16;
        cudaError_t e = launch_dependent(a.gated ? up_stream_kernel<El, NT, true> : up_stream_kernel<El, NT, false>, grid(slots * ((a.hidden_ld + kCh - 1) / kCh), num_sms),
                                         dim3(Cf::kUpThreads), Cf::kUpSmem, stream, 1, m.up, m.down, a);
        if (e != cudaSuccess) return e;
        return launch_dependent(wide ? down_stream_kernel<El, NT, Cf::kMostTiles> : down_stream_kernel<El, NT, 1>, grid((a.width + a.channels - 1) / a.channels, num_sms), dim3(Cf::kDownThreads),
                                Cf::down_smem(a.tokens, wide ? 2 : 1), stream, 1, m.down, a);
    }
    const long long items = asked * (a.hidden_ld / (a.gated ? 8 : 16));
    // Warps that share an item's K: all eight unless that leaves a CTA many rounds (us, eight against the
    // rule: 16 tokens, 4 of 32 experts, 65 x 1001 66, 53; 64 tokens 100, 82; 64 tokens, 129 x 2001 199, 158).
    int share = kWarps;
    while (share > 1 && items > 4ll * num_sms * (kWarps / share) && (a.width + kChunk - 1) / kChunk <= 2 * share) share /= 2;
    cudaError_t e = launch_dependent(a.gated ? up_kernel<El, NT, true> : up_kernel<El, NT, false>, grid((items + kWarps / share - 1) / (kWarps / share), 2ll * num_sms),
                                     dim3(kThreads), 0, stream, 1, a, share);
    if (e != cudaSuccess) return e;
    return launch_dependent(down_kernel<El, NT>, dim3((a.width + 15) / 16), dim3(kThreads), kWarps * a.tokens * kOutPitch * 4, stream, 1, a);
}

template <class El>
cudaError_t layer_for(const LayerArgs &a, int num_sms, cudaStream_t stream) {
    auto at16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    LayerMaps m{};
    const long long up_rows = a.experts * a.up_rows, down_rows = static_cast<long long>(a.experts) * a.width;
    const bool boundaries = reinterpret_cast<uintptr_t>(a.X) % 32 == 0 && at16(a.up) && at16(a.down) && a.ldx * sizeof(typename El::T) % 32 == 0 && a.width % 16 == 0 &&
                            a.hidden % 16 == 0 && a.hidden > 0 && up_rows < kMostRows && down_rows < kMostRows &&
                            encode_map(&m.up, MapType::kInt8, 2, a.up, a.width, up_rows, 1, a.width, 0, 128, 16) &&
                            encode_map(&m.down, MapType::kInt8, 2, a.down, a.hidden, down_rows, 1, a.hidden, 0, 128, 16);
    // Tokens that share an expert's weights in one go: 8, 16 or 32, the last where there are more than 12
    // choices an expert (us in 16s and in 32s, gated, 2048 x 1408: 8 an expert, 64 tokens, 2 of 16: 71.5,
    // 89.5; 12, 24 tokens, 2 of 4: 28.8, 34.2; 16, 64 tokens, 4 of 16: 111, 120; 24, 48 tokens, 4 of 8: 83.5,
    // 77.2; but 32, 64 tokens, 2 of 4: 53.3, 60.6).
    if (a.tokens <= 8) return layer_typed<El, 1>(a, boundaries, m, num_sms, stream);
    if (a.tokens <= 16 || a.tokens * a.choices <= 12 * a.experts) return layer_typed<El, 2>(a, boundaries, m, num_sms, stream);
    return layer_typed<El, 4>(a, boundaries, m, num_sms, stream);
}

template <class El, int NT>
cudaError_t prepare_typed() {
    constexpr int kSums = kWarps * kLayerTokens * kOutPitch * 4;
    cudaError_t e = cudaFuncSetAttribute(down_kernel<El, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSums);
    for (auto *k : {up_stream_kernel<El, NT, false>, up_stream_kernel<El, NT, true>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, StreamCfg<El, NT>::kUpSmem);
    using Cf = StreamCfg<El, NT>;
    for (auto *k : {down_stream_kernel<El, NT, 1>, down_stream_kernel<El, NT, Cf::kMostTiles>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::down_smem(NT == 1 ? 8 : kLayerTokens, Cf::kMostTiles));
    return e;
}

}  // namespace

size_t layer_floats(int type, int slots, int hidden) {
    const size_t ld = (static_cast<size_t>(hidden) + kPad - 1) / kPad * kPad;
    return (type == SGEMM_IN_F32 ? 3 : 2) * static_cast<size_t>(slots) * ld / 2;
}

cudaError_t layer_prepare() {
    cudaError_t e = cudaSuccess;
    for (cudaError_t r : {prepare_typed<ElF32, 1>(), prepare_typed<ElF32, 2>(), prepare_typed<ElF32, 4>(), prepare_typed<ElBF16, 1>(),
                          prepare_typed<ElBF16, 2>(), prepare_typed<ElBF16, 4>(), prepare_typed<ElF16, 1>(), prepare_typed<ElF16, 2>(),
                          prepare_typed<ElF16, 4>()})
        if (e == cudaSuccess) e = r;
    return e;
}

cudaError_t launch_expert_layer(int type, LayerArgs a, int num_sms, cudaStream_t stream) {
    a.hidden_ld = (a.hidden + kPad - 1) / kPad * kPad;
    a.up_rows = static_cast<long long>(a.gated ? 2 : 1) * a.hidden;
    a.h_part = static_cast<long long>(a.tokens) * a.choices * a.hidden_ld;
    switch (type) {
        case SGEMM_IN_F32: return layer_for<ElF32>(a, num_sms, stream);
        case SGEMM_IN_BF16: return layer_for<ElBF16>(a, num_sms, stream);
        default: return layer_for<ElF16>(a, num_sms, stream);
    }
}

}  // namespace sg
