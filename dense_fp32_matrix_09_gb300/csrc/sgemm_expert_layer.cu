// A whole mixture-of-experts layer for a few tokens, for sm_103a:
//   out_t = sum_j w_tj D_e act(U_e x_t),  e = ids_tj
// with U_e and D_e in int8, a scale a channel, and act = silu, or silu of one half of
// U_e's channels times the other.  Two kernels: up_kernel makes the hidden rows of
// every expert that some token asks for, down_kernel multiplies them and adds
// up each token's.  Bound by the weights' way from HBM, which every asked expert's
// make once.
//
// Every CTA works the routing out by itself (a counting sort of up to 1024 choices in
// shared memory): no kernel before, nothing on the host.  The groups -- up to
// 8 * NT tokens of one expert -- are then dealt out in a fixed order.
//
// The weights go from HBM straight into registers, 16 bytes a lane, and are
// multiplied by mma.sync (m16n8k16, BF16, FP32 sums), whose rate is far above what HBM
// delivers for so few tokens: a tile of 16 channels x 8 tokens takes each weight once.
// The order of k within an MMA is free, so a lane's 16 bytes are the k of four
// MMAs.  An int8 is exact in BF16; the tokens' elements go in as sums of one (BF16), two
// (FP16) or three (FP32) BF16 values, exact as well.  The hidden rows
// are kept as two such values, 16 bits of fraction, and with FP32 rows as three.  Within
// a warp sums run along k; the warps' sums, the experts' and the choices' are added in a
// fixed order in FP32.
#include "device_common.cuh"
#include "internal.h"
#include "rows.cuh"
#include "sgemm.h"

namespace sg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 64;  // k of a step: 16 bytes of each of 16 channels from four lanes each
constexpr int kSlots = kLayerSlots;

template <class El>
struct Parts;  // BF16 values that an element and a hidden value become
template <> struct Parts<ElBF16> { static constexpr int in = 1, hidden = 2; };
template <> struct Parts<ElF16> { static constexpr int in = 2, hidden = 2; };
template <> struct Parts<ElF32> { static constexpr int in = 3, hidden = 3; };

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

// Four int8 to two pairs of BF16: 0x4300 + u is 128 + u for u < 128, and 0x4380 is 256,
// so with a byte b's low seven bits u and its sign s, (0x4300 + u) - (0x4300 + 128 s)
// is u - 128 s, exactly b.
__device__ __forceinline__ void expand_int8(uint32_t w, uint32_t &lo, uint32_t &hi) {
    auto one = [](uint32_t p) {
        const uint32_t a = p & 0xff7fff7fu, s = p & 0xff80ff80u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&s));
        return *reinterpret_cast<const uint32_t *>(&d);
    };
    lo = one(__byte_perm(w, 0x43434343u, 0x4140));
    hi = one(__byte_perm(w, 0x43434343u, 0x4342));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The routing, as every CTA works it out.  Columns: the choices that count, sorted
// by expert, the earlier first.  A token that names an expert twice has one column
// with the sum of both weights.
struct Routing {
    int id[kSlots];            // the slot's expert, -1: none of its own
    short token[kSlots];       // by column
    float weight[kSlots];
    int start[kMaxExperts + 1];  // first column of an expert
    int group_expert[kSlots], group_first[kSlots];  // first: column; a group ends with its expert's columns or after 8 * NT
    int groups;
};

__device__ void route(Routing &r, const LayerArgs &a, int per_group) {
    const int slots = a.tokens * a.choices, tid = threadIdx.x;
    for (int e = tid; e <= a.experts; e += kThreads) r.start[e] = 0;
    for (int s = tid; s < slots; s += kThreads) {
        const int id = __ldcg(a.ids + s);
        r.id[s] = static_cast<unsigned>(id) < static_cast<unsigned>(a.experts) ? id : -1;
    }
    __syncthreads();
    // slots that repeat an earlier choice of their token add to its weight
    float mine[kSlots / kThreads];
    bool own[kSlots / kThreads];
#pragma unroll
    for (int k = 0; k < kSlots / kThreads; ++k) {
        const int s = tid + k * kThreads;
        own[k] = s < slots && r.id[s] >= 0;
        mine[k] = 0.f;
        if (!own[k]) continue;
        const int t0 = s / a.choices * a.choices;
        for (int q = t0; q < s; ++q) own[k] = own[k] && r.id[q] != r.id[s];
        for (int q = s; q < t0 + a.choices; ++q)
            if (r.id[q] == r.id[s]) mine[k] += __ldcg(a.weights + q);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSlots / kThreads; ++k) {
        const int s = tid + k * kThreads;
        if (s >= slots) continue;
        if (own[k]) atomicAdd(&r.start[r.id[s]], 1);
        else r.id[s] = -1;
    }
    __syncthreads();
    if (tid < 32) {  // counts to first columns; the groups
        int cols = 0, groups = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + tid, n = e < a.experts ? r.start[e] : 0, g = (n + per_group - 1) / per_group;
            int sn = n, sg = g;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int un = __shfl_up_sync(0xffffffffu, sn, d), ug = __shfl_up_sync(0xffffffffu, sg, d);
                if (tid >= d) {
                    sn += un;
                    sg += ug;
                }
            }
            if (e < a.experts) r.start[e] = cols + sn - n;
            for (int k = 0; k < g; ++k) {
                r.group_expert[groups + sg - g + k] = e;
                r.group_first[groups + sg - g + k] = cols + sn - n + k * per_group;
            }
            cols += __shfl_sync(0xffffffffu, sn, 31);
            groups += __shfl_sync(0xffffffffu, sg, 31);
        }
        if (tid == 0) {
            r.start[a.experts] = cols;
            r.groups = groups;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSlots / kThreads; ++k) {
        const int s = tid + k * kThreads;
        if (s >= slots || r.id[s] < 0) continue;
        int c = r.start[r.id[s]];
        for (int q = 0; q < s; ++q) c += r.id[q] == r.id[s];
        r.token[c] = static_cast<short>(s / a.choices);
        r.weight[c] = mine[k];
    }
    __syncthreads();
}

// 16 bytes of a weight row from k on, zeros behind its end.
template <bool VEC>
__device__ __forceinline__ uint4 load_weights(const int8_t *row, int k, int K) {
    if (VEC) return k < K ? __ldcg(reinterpret_cast<const uint4 *>(row + k)) : make_uint4(0, 0, 0, 0);
    uint32_t w[4] = {};
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (k + e < K) w[e / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(__ldcg(row + k + e))) << (8 * (e % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 elements of a token from k on as P x 8 pairs of BF16, zeros behind its end.
template <class El, bool VEC>
__device__ __forceinline__ void load_token(const typename El::T *row, int k, int K, uint32_t (&to)[Parts<El>::in][8]) {
    using T = typename El::T;
    constexpr int P = Parts<El>::in, V = 16 / sizeof(T);
    alignas(16) T v[16];
    if (VEC) {
#pragma unroll
        for (int e = 0; e < 16; e += V)
            *reinterpret_cast<uint4 *>(v + e) = k + e < K ? __ldca(reinterpret_cast<const uint4 *>(row + k + e)) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = k + e < K ? __ldca(row + k + e) : El::down(0.f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        uint32_t p[P];
        if (P == 1) p[0] = *reinterpret_cast<const uint32_t *>(v + 2 * e);
        else split2<P>(El::up(v[2 * e]), El::up(v[2 * e + 1]), p);
#pragma unroll
        for (int q = 0; q < P; ++q) to[q][e] = p[q];
    }
}

// acc += 16 channels x 64 k (lo: channel g, hi: channel g + 8) times 8 tokens.
template <int P>
__device__ __forceinline__ void multiply(float (&acc)[4], const uint32_t (&a)[4][4], const uint32_t (&x)[P][8]) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int p = P - 1; p >= 0; --p) mma_bf16(acc, a[s], x[p][2 * s], x[p][2 * s + 1]);
}
__device__ __forceinline__ void expand_rows(const uint4 &lo, const uint4 &hi, uint32_t (&a)[4][4]) {
    const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        expand_int8(l[s], a[s][0], a[s][2]);
        expand_int8(h[s], a[s][1], a[s][3]);
    }
}

constexpr int kAhead = 4;  // chunks whose loads are in flight

// hidden[part][column][f] = act(U x) of every group; an item is a group and 16 rows of
// U: with a gate 8 channels of it and the 8 that it goes with, in the MMA's upper and
// lower rows, so that one lane has both.  `share` warps of the CTA split an item's K.
template <class El, int NT, bool GATED, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) up_kernel(const LayerArgs a, int share) {
    using T = typename El::T;
    constexpr int P = Parts<El>::in, PH = Parts<El>::hidden, kCh = GATED ? 8 : 16;
    __shared__ Routing r;
    __shared__ float4 sums[kWarps][NT][32];
    griddep_wait();
    griddep_launch_dependents();
    route(r, a, 8 * NT);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int tiles = a.hidden_ld / kCh, teams = kWarps / share, team = warp / share, part = warp % share;
    const long long items = static_cast<long long>(r.groups) * tiles;
    const int chunks = (a.width + kChunk - 1) / kChunk;
    for (long long i0 = static_cast<long long>(blockIdx.x) * teams; i0 < items; i0 += static_cast<long long>(gridDim.x) * teams) {
        const long long item = i0 + team;
        const bool live = item < items;
        const int group = live ? static_cast<int>(item / tiles) : 0, f0 = live ? static_cast<int>(item % tiles) * kCh : 0;
        const int e = r.group_expert[group], first = r.group_first[group], cols = min(r.start[e + 1] - first, 8 * NT);
        const int fl = f0 + g, fh = GATED ? fl : fl + 8;  // the hidden channels of the lane's rows
        const bool in_l = live && fl < a.hidden, in_h = live && fh < a.hidden;
        const long long row_l = static_cast<long long>(e) * a.up_rows + (in_l ? fl : 0);
        const long long row_h = static_cast<long long>(e) * a.up_rows + (in_h ? fh : 0) + (GATED ? a.hidden : 0);
        const int8_t *ul = a.up + row_l * a.width, *uh = a.up + row_h * a.width;
        const T *x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            x[n] = static_cast<const T *>(a.X) + static_cast<long long>(r.token[first + min(n * 8 + g, cols - 1)]) * a.ldx;
        float acc[NT][4] = {};
        for (int c0 = part; c0 < chunks; c0 += share * kAhead) {
            uint4 wl[kAhead], wh[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int at = (c0 + k * share) * kChunk + t * 16;
                wl[k] = load_weights<VEC>(ul, at, in_l ? a.width : 0);
                wh[k] = load_weights<VEC>(uh, at, in_h ? a.width : 0);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (c0 + k * share >= chunks) break;
                const int at = (c0 + k * share) * kChunk + t * 16;
                uint32_t w[4][4];
                expand_rows(wl[k], wh[k], w);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n * 8 >= cols) break;
                    uint32_t v[P][8];
                    load_token<El, VEC>(x[n], at, a.width, v);
                    multiply<P>(acc[n], w, v);
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
                const float sl = in_l ? __ldca(a.up_scale + row_l) : 0.f, sh = in_h ? __ldca(a.up_scale + row_h) : 0.f;
                auto silu = [](float v) { return v / (1.f + expf(-v)); };
                // tokens 2t, 2t + 1; channels behind the last hidden one are written as zeros
                const float y0 = GATED ? silu(s.x * sl) * (s.z * sh) : silu(s.x * sl), y1 = GATED ? silu(s.y * sl) * (s.w * sh) : silu(s.y * sl);
                const float z0 = GATED ? 0.f : silu(s.z * sh), z1 = GATED ? 0.f : silu(s.w * sh);
                auto put = [&](int col, int f, float v) {
                    if (col >= cols) return;
                    uint32_t p[PH];
                    split2<PH>(v, 0.f, p);
#pragma unroll
                    for (int q = 0; q < PH; ++q)
                        a.h[q * a.h_part + static_cast<long long>(first + col) * a.hidden_ld + f] = static_cast<uint16_t>(p[q]);
                };
                put(n * 8 + 2 * t, fl, in_l ? y0 : 0.f);
                put(n * 8 + 2 * t + 1, fl, in_l ? y1 : 0.f);
                if (!GATED) {
                    put(n * 8 + 2 * t, fh, in_h ? z0 : 0.f);
                    put(n * 8 + 2 * t + 1, fh, in_h ? z1 : 0.f);
                }
            }
        }
        __syncthreads();
    }
}

// out: an item is 16 channels of every token; the CTA's warps take consecutive runs of
// (group, chunk of k) pairs.  At the end of its run or of a group a warp adds what it
// has, scaled, to its own sums of the tokens.
constexpr int kOutPitch = 17;
template <class El, int NT, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) down_kernel(const LayerArgs a) {
    constexpr int PH = Parts<El>::hidden;
    extern __shared__ float out_sums[];  // [warp][token][kOutPitch]
    __shared__ Routing r;
    // (the routing and the sums touch nothing that the kernel before writes, and that
    // one has waited for what came before it)
    for (int k = threadIdx.x; k < kWarps * a.tokens * kOutPitch; k += kThreads) out_sums[k] = 0.f;
    route(r, a, 8 * NT);
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
        const int e = r.group_expert[group], first = r.group_first[group], cols = min(r.start[e + 1] - first, 8 * NT);
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
                vl[k] = load_weights<VEC>(wl, at, in_l && c0 + k < c_last ? a.hidden : 0);
                vh[k] = load_weights<VEC>(wh, at, in_h && c0 + k < c_last ? a.hidden : 0);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (c0 + k >= c_last) break;
                const int at = (c0 + k) * kChunk + t * 16;
                uint32_t w[4][4];
                expand_rows(vl[k], vh[k], w);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n * 8 >= cols) break;
                    uint32_t v[PH][8];
#pragma unroll
                    for (int q = 0; q < PH; ++q)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            *reinterpret_cast<uint4 *>(&v[q][4 * x]) =
                                __ldca(reinterpret_cast<const uint4 *>(h[n] + q * a.h_part + at + 8 * x));
                    multiply<PH>(acc[n], w, v);
                }
            }
        }
        const float sl = in_l ? __ldca(a.down_scale + row_l) : 0.f, sh = in_h ? __ldca(a.down_scale + row_h) : 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = n * 8 + 2 * t + j;
                if (col >= cols) continue;
                float *to = mine + r.token[first + col] * kOutPitch;
                const float w = r.weight[first + col];
                to[g] = fmaf(acc[n][j] * sl, w, to[g]);
                to[g + 8] = fmaf(acc[n][2 + j] * sh, w, to[g + 8]);
            }
        __syncwarp();
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

template <class El, int NT, bool VEC>
cudaError_t layer_typed(const LayerArgs &a, int num_sms, cudaStream_t stream) {
    // (the groups are on the device: so many there are at most)
    const long long slots = static_cast<long long>(a.tokens) * a.choices, asked = slots < a.experts ? slots : a.experts;
    const long long items = asked * (a.hidden_ld / (a.gated ? 8 : 16));
    // warps that share an item's K: all eight unless that leaves a CTA many rounds
    int share = kWarps;
    while (share > 1 && items > 4ll * num_sms * (kWarps / share) && (a.width + kChunk - 1) / kChunk <= 2 * share) share /= 2;
    const long long ctas = (items + kWarps / share - 1) / (kWarps / share), most = 2ll * num_sms;
    const dim3 grid(static_cast<unsigned>(ctas < 1 ? 1 : ctas < most ? ctas : most));  // (no hidden channels: nothing to do)
    cudaError_t e = launch_dependent(a.gated ? up_kernel<El, NT, true, VEC> : up_kernel<El, NT, false, VEC>, grid, dim3(kThreads), 0, stream, 1, a, share);
    if (e != cudaSuccess) return e;
    return launch_dependent(down_kernel<El, NT, VEC>, dim3((a.width + 15) / 16), dim3(kThreads), kWarps * a.tokens * kOutPitch * 4, stream, 1, a);
}

template <class El>
cudaError_t layer_for(const LayerArgs &a, int num_sms, cudaStream_t stream) {
    auto at16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const bool vec = at16(a.X) && at16(a.up) && at16(a.down) && a.ldx * sizeof(typename El::T) % 16 == 0 && a.width % 16 == 0 && a.hidden % 16 == 0;
    // tokens that share an expert's weights in one go: 8 or 32
    if (a.tokens <= 8) return vec ? layer_typed<El, 1, true>(a, num_sms, stream) : layer_typed<El, 1, false>(a, num_sms, stream);
    return vec ? layer_typed<El, 4, true>(a, num_sms, stream) : layer_typed<El, 4, false>(a, num_sms, stream);
}

}  // namespace

size_t layer_floats(int type, int slots, int hidden) {
    const size_t ld = (static_cast<size_t>(hidden) + kChunk - 1) / kChunk * kChunk;
    return (type == SGEMM_IN_F32 ? 3 : 2) * static_cast<size_t>(slots) * ld / 2;
}

cudaError_t layer_prepare() {
    cudaError_t e = cudaSuccess;
    for (auto *k : {down_kernel<ElF32, 1, false>, down_kernel<ElF32, 1, true>, down_kernel<ElF32, 4, false>, down_kernel<ElF32, 4, true>,
                    down_kernel<ElBF16, 1, false>, down_kernel<ElBF16, 1, true>, down_kernel<ElBF16, 4, false>, down_kernel<ElBF16, 4, true>,
                    down_kernel<ElF16, 1, false>, down_kernel<ElF16, 1, true>, down_kernel<ElF16, 4, false>, down_kernel<ElF16, 4, true>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kWarps * kLayerTokens * kOutPitch * 4);
    return e;
}

cudaError_t launch_expert_layer(int type, LayerArgs a, int num_sms, cudaStream_t stream) {
    a.hidden_ld = (a.hidden + kChunk - 1) / kChunk * kChunk;
    a.up_rows = static_cast<long long>(a.gated ? 2 : 1) * a.hidden;
    a.h_part = static_cast<long long>(a.tokens) * a.choices * a.hidden_ld;
    switch (type) {
        case SGEMM_IN_F32: return layer_for<ElF32>(a, num_sms, stream);
        case SGEMM_IN_BF16: return layer_for<ElBF16>(a, num_sms, stream);
        default: return layer_for<ElF16>(a, num_sms, stream);
    }
}

}  // namespace sg
