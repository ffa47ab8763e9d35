// The RMS norm of rows (with the residual's addition before it, and an output in
// the rows' type, in 8 bits or in 4), rows to 4 bits without a norm, and rows of 4
// bits back, for sm_103a.
//
//  * row_kernel -- per row: h = x + residual (rounded to the type), the sum of its
//    squares, r = 1 / sqrt(sum / K + eps), and then
//      y = h * r * w                                                  (OUT_Y)
//      v = h * w, q = rint(v * (127 / max|v|)), scale = max|v| * r / 127   (OUT_I8)
//      v = h * w in 4 bits with a scale a block, times r a row             (OUT_F4)
//    The quantized forms round v and not y: r is a factor of the whole row, which
//    the row's scale takes, so that no rounding of an element hangs on the last bit
//    of a sum, whatever its order.  Without a norm v = x and r = 1.
//    One pass over HBM: a row stays in the registers of the TPR threads that share
//    it (up to 4 x 8 elements a thread; longer rows are read a second time, from L2).
//    8192 x 8192 BF16 with the residual to 8 bits 67.8 us, HBM's rate; 32 x 4096 2.1 us in
//    a graph.  To 4 bits the instructions count too: 8192 x 8192 FP16 to MX 29.5 us (floor
//    25), to NV, whose scales wait for the whole row, 37.4.
//  * dequantize_kernel -- 4-bit rows to what they stand for: the same matrix 27.7 us (floor 25).
//
// No load is a read-only-cache load: what is read may have been written by the
// kernel before, whose end the launch overlaps.
#include "device_common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "rows.cuh"
#include "sgemm.h"

namespace sg {
namespace {

constexpr int OUT_Y = 0, OUT_I8 = 1, OUT_F4 = 2;

constexpr unsigned kInfBits = 0x7f800000u;
// Below these row maxima the quotient 127 / m or 2688 / m overflows: the row is stored as
// zeros.
constexpr float kLeastI8 = 127.f * 0x1p-126f, kLeastNV = 2688.f * 0x1p-126f;
// From kLeastNV up to here (2688 / m) / s may overflow, s being 2^-9 or more.  Such a row is
// taken 2^16 times larger, which is exact and changes none of its codes and scales.
constexpr float kTinyNV = 2688.f * 0x1p-118f, kLiftNV = 0x1p16f;
constexpr float kRoundMagic = 12582912.f;  // 1.5 * 2^23: added to a value below 2^22 it rounds it to an integer

// Sum and maximum over the TPR threads of a row, in the same order on every call.
template <int TPR>
__device__ __forceinline__ void row_reduce(float &sum, unsigned &top) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    top = __reduce_max_sync(0xffffffffu, top);
    if (TPR > 32) {
        constexpr int kWarps = (TPR < 256 ? 256 : TPR) / 32;
        __shared__ float sums[kWarps];
        __shared__ unsigned tops[kWarps];
        if ((threadIdx.x & 31) == 0) {
            sums[threadIdx.x / 32] = sum;
            tops[threadIdx.x / 32] = top;
        }
        __syncthreads();
        const int w0 = threadIdx.x / TPR * (TPR / 32);
        sum = 0.f;
        top = 0;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) {
            sum += sums[w0 + w];
            top = max(top, tops[w0 + w]);
        }
    }
}

// The largest magnitude of three values; a NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Bits of the largest magnitude of N values, those of a NaN above infinity's.
template <int N>
__device__ __forceinline__ unsigned top_of(const float *v) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e + 1 < N; e += 2) m = max_abs(m, v[e], v[e + 1]);
    if (N % 2) m = max_abs(m, v[N - 1], 0.f);
    return __float_as_uint(m) & 0x7fffffffu;
}

// Bits of the largest magnitude of the block that this lane's A elements belong to:
// `lanes` lanes hold it.
__device__ __forceinline__ unsigned block_max(unsigned top, int lanes) {
    for (int d = 1; d < lanes; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    return top;
}

// Where a row in 4 bits goes, and what its elements are multiplied by.
struct Fp4Row {
    uint8_t *q, *s;  // s: the row's first word of scales
    int K, format, words, vec;
    float up, near;  // NV: 2688 / m, 448 / m; up below 0 where v is taken -2^16 times
};

// One piece (see load8) of a row to 4 bits.  The whole warp.
template <int TPR, int A>
__device__ __forceinline__ void put_fp4(const Fp4Row &r, int c, int lane, const float (&v)[kV]) {
    const int at = c * kV * TPR + lane * A, block = fp4_block(r.format), per = block / A;  // lanes a block
    float f[kV / A];
#pragma unroll
    for (int i = 0; i < kV / A; ++i) {
        const unsigned top = block_max(top_of<A>(v + i * A), per);
        uint32_t code;
        if (r.format == SGEMM_FP4_MX) {
            // floor(log2) of the block's largest value, less 2 (the exponent of the
            // largest code), from its exponent bits
            const bool number = top < kInfBits;
            code = number ? static_cast<uint32_t>(max(static_cast<int>(top >> 23) - 2, 0)) : 255u;
            f[i] = number ? exp2_of(127 - static_cast<int>(code)) : 0.f;
        } else {
            code = to_e4m3(__fmul_rn(__uint_as_float(top), r.near));
            f[i] = code ? __fdiv_rn(r.up, from_e4m3(code)) : 0.f;
        }
        const int first = at + i * TPR * A, b = first / block;  // the lane's block
        if (4 * per <= 32) {  // a word of four scales within the warp: one store
            uint32_t word = code << (8 * (b & 3));
            word |= __shfl_xor_sync(0xffffffffu, word, per);
            word |= __shfl_xor_sync(0xffffffffu, word, 2 * per);
            if (lane % (4 * per) == 0 && first < r.K)
                *reinterpret_cast<uint32_t *>(r.s + static_cast<long long>(b / 4) * 512) = word;
        } else if (lane % per == 0 && b < 4 * r.words) {
            r.s[static_cast<long long>(b / 4) * 512 + (b & 3)] = static_cast<uint8_t>(code);
        }
    }
    float x[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) x[e] = __fmul_rn(v[e], f[e / A]);
    uint32_t w = to_e2m1x8(x);
    // (a factor of 0: infinities and NaNs among them, whose products are no zeros)
#pragma unroll
    for (int i = 0; i < kV / A; ++i)
        if (f[i] == 0.f) w &= ~((A == 8 ? 0xffffffffu : (1u << (4 * A % 32)) - 1u) << (4 * A * i));
#pragma unroll
    for (int i = 0; i < kV / A; ++i) {
        const int p = at + i * TPR * A;
        uint32_t bits = w >> (4 * A * i);
        if (A == 1) {
            const uint32_t other = __shfl_down_sync(0xffffffffu, bits, 1);
            bits = (bits & 15u) | (other & 15u) << 4;
            if (p < r.K && lane % 2 == 0) r.q[p / 2] = static_cast<uint8_t>(bits);
        } else if (p < r.K) {
            uint8_t *q = r.q + p / 2;
            if (A == 8 && r.vec) {
                *reinterpret_cast<uint32_t *>(q) = bits;
            } else if (A == 4 && r.vec) {
                *reinterpret_cast<uint16_t *>(q) = static_cast<uint16_t>(bits);
            } else {
#pragma unroll
                for (int j = 0; j < A / 2; ++j) q[j] = static_cast<uint8_t>(bits >> (8 * j));
            }
        }
    }
}

template <class El, int TPR, int A, int HELD, bool NORM, int OUT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
row_kernel(const RowArgs a) {
    using T = typename El::T;
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % TPR;
    const unsigned i = blockIdx.x * kRows + threadIdx.x / TPR;
    const bool live = i < static_cast<unsigned>(a.M);
    const long long row = live ? i : 0;
    const T *x = static_cast<const T *>(a.X) + row * a.ldx;
    const T *add = NORM && a.R ? static_cast<const T *>(a.R) + row * a.ldr : nullptr;
    T *keep = NORM && a.H ? static_cast<T *>(a.H) + row * a.ldh : nullptr;
    const T *w = static_cast<const T *>(a.W);
    const int width = live ? a.K : 0;

    // h of piece c; the sum is rounded to the type, as it is what goes on
    auto sum_of = [](Pack8<T> p, const Pack8<T> &q) {
#pragma unroll
        for (int e = 0; e < kV; ++e) p.v[e] = El::down(__fadd_rn(El::up(p.v[e]), El::up(q.v[e])));
        return p;
    };
    // v of piece c, what is quantized
    auto scaled = [&](const Pack8<T> &h, const Pack8<T> &g, float (&v)[kV]) {
#pragma unroll
        for (int e = 0; e < kV; ++e) v[e] = NORM ? __fmul_rn(El::up(h.v[e]), El::up(g.v[e])) : El::up(h.v[e]);
    };

    Pack8<T> h[HELD], g[HELD];
#pragma unroll
    for (int c = 0; c < HELD; ++c) h[c] = load8<T, TPR, A>(x, c, lane, width);
    if (NORM) {
#pragma unroll
        for (int c = 0; c < HELD; ++c) g[c] = load8<T, TPR, A, true>(w, c, lane, width);
    }
    if (add) {
        Pack8<T> more[HELD];
#pragma unroll
        for (int c = 0; c < HELD; ++c) more[c] = load8<T, TPR, A>(add, c, lane, width);
#pragma unroll
        for (int c = 0; c < HELD; ++c) h[c] = sum_of(h[c], more[c]);
    }
    if (keep) {
#pragma unroll
        for (int c = 0; c < HELD; ++c) store8<T, TPR, A>(keep, c, lane, width, h[c]);
    }
    float sum = 0.f;
    unsigned top = 0;  // max |v| as bits: NaN above infinity above every number
    auto look = [&](const Pack8<T> &p, const Pack8<T> &q) {
        float v[kV];
        if (OUT != OUT_Y) scaled(p, q, v);
#pragma unroll
        for (int e = 0; e < kV; ++e)
            if (NORM) sum = fmaf(El::up(p.v[e]), El::up(p.v[e]), sum);
        if (OUT != OUT_Y) top = max(top, top_of<kV>(v));
    };
    const bool whole = NORM || OUT == OUT_I8 || a.format == SGEMM_FP4_NV;  // whether anything is asked of the whole row
    if (whole) {
#pragma unroll
        for (int c = 0; c < HELD; ++c) look(h[c], g[c]);
    }
    for (int c = HELD; whole && c * kV * TPR < width; ++c) {
        Pack8<T> p = load8<T, TPR, A>(x, c, lane, width), q = p;
        if (add) p = sum_of(p, load8<T, TPR, A>(add, c, lane, width));
        if (keep) store8<T, TPR, A>(keep, c, lane, width, p);
        if (NORM) q = load8<T, TPR, A, true>(w, c, lane, width);
        look(p, q);
    }
    if (whole) row_reduce<TPR>(sum, top);
    if (!live) return;
    const float r = NORM ? __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(a.K)), a.eps)) : 1.f;

    // the pieces, those that are not held read again (h where it was written, by this very thread)
    const T *again = keep ? keep : x;
    auto each = [&](auto put) {
#pragma unroll
        for (int c = 0; c < HELD; ++c) put(c, h[c], g[c]);
        for (int c = HELD; c * kV * TPR < a.K; ++c) {
            const Pack8<T> p = load8<T, TPR, A>(again, c, lane, a.K);
            put(c, p, NORM ? load8<T, TPR, A, true>(w, c, lane, a.K) : p);
        }
    };
    if (OUT == OUT_Y) {
        T *y = static_cast<T *>(a.Y) + row * a.ldy;
        if (lane == 0 && a.row) a.row[i] = r;
        each([&](int c, const Pack8<T> &p, const Pack8<T> &q) {
            Pack8<T> o;
#pragma unroll
            for (int e = 0; e < kV; ++e) o.v[e] = El::down(__fmul_rn(__fmul_rn(El::up(p.v[e]), r), El::up(q.v[e])));
            store8<T, TPR, A>(y, c, lane, a.K, o);
        });
        return;
    }
    const float m = __uint_as_float(top), nan = __int_as_float(0x7fc00000);
    const bool number = top < kInfBits;
    if (OUT == OUT_I8) {
        int8_t *y = static_cast<int8_t *>(a.Y) + row * a.ldy;
        const bool zero = !number || m < kLeastI8;
        const float inv = zero ? 0.f : __fdiv_rn(127.f, m);
        if (lane == 0) a.row[i] = !number ? nan : zero ? 0.f : __fdiv_rn(__fmul_rn(m, r), 127.f);
        each([&](int c, const Pack8<T> &p, const Pack8<T> &q) {
            float v[kV];
            scaled(p, q, v);
            Pack8<int8_t> o;
#pragma unroll
            for (int e = 0; e < kV; ++e)
                o.v[e] = zero ? static_cast<int8_t>(0)
                              : static_cast<int8_t>(__float_as_uint(__fadd_rn(__fmul_rn(v[e], inv), kRoundMagic)));
            const int at = c * kV * TPR + lane * A;
#pragma unroll
            for (int k = 0; k < kV / A; ++k) {
                if (at + k * TPR * A >= a.K) continue;
                int8_t *to = y + at + k * TPR * A;
                if (A == 8 && a.vec) *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(o.v);
                else if (A == 4 && a.vec) *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(o.v + k * A);
                else
#pragma unroll
                    for (int e = 0; e < A; ++e) to[e] = o.v[k * A + e];
            }
        });
        return;
    }
    Fp4Row f{static_cast<uint8_t *>(a.Y) + row * a.ldy, a.S + fp4_scale_word(row, 0, a.words), a.K, a.format, a.words, a.vec, 1.f, 0.f};
    if (a.format == SGEMM_FP4_NV) {
        const bool blank = !number || m < kLeastNV;  // a row of zeros: every scale 0
        const float top_value = m < kTinyNV ? m * -kLiftNV : m;
        f.up = blank ? 0.f : __fdiv_rn(2688.f, top_value);
        f.near = blank ? 0.f : __fdiv_rn(448.f, fabsf(top_value));
        if (lane == 0) a.row[i] = !number ? nan : blank ? 0.f : __fmul_rn(__fdiv_rn(m, 2688.f), r);
    } else if (lane == 0 && a.row) {
        // (a row of zeros is one whatever r, which without eps is an infinity)
        a.row[i] = top == 0 && r >= __uint_as_float(kInfBits) ? 0.f : r;
    }
    each([&](int c, const Pack8<T> &p, const Pack8<T> &q) {
        if (c * kV * TPR >= a.K) return;  // (the whole row's threads)
        float v[kV];
        scaled(p, q, v);
        if (f.up <= 0.f) {
#pragma unroll
            for (int e = 0; e < kV; ++e) v[e] = f.up < 0.f ? v[e] * -kLiftNV : 0.f;
        }
        put_fp4<TPR, A>(f, c, lane, v);
    });
}

// Threads a row: enough that it stays in registers (32 elements a thread), and, with
// too few rows to fill the GPU, more of them so that each thread loads less; rows of
// at most eight elements a thread take a kernel of one piece.  (us, BF16 to 8 bits with the
// residual, 8 elements a thread against 32: 32 x 4096 2.05, 2.44; 304 x 2048 2.1, 2.4; 912 x 4096 6.1,
// 4.2; 4864 x 512 7.1, 4.8.  Rows of 8192 have 16 a thread at best and lose by it: 304 of them
// 5.7, 3.3.)
template <class El, int A, bool NORM, int OUT>
cudaError_t row_typed(const RowArgs &a, int num_sms, cudaStream_t stream) {
    const int per = a.M <= 4 * num_sms ? kV : 4 * kV;
    const int want = (a.K + per - 1) / per;
    const int share = want <= 32 ? 32 : want <= 128 ? 128 : want <= 256 ? 256 : 512;
    const bool one = a.K <= kV * share;
#define SG_ROW(TPR)                                                                                              \
    return launch_dependent(one ? row_kernel<El, TPR, A, 1, NORM, OUT> : row_kernel<El, TPR, A, 4, NORM, OUT>,   \
                            dim3(blocks_of(a.M, TPR < 256 ? 256 / TPR : 1)), dim3(TPR < 256 ? 256 : TPR), 0,     \
                            stream, 1, a)
    if (share == 32) SG_ROW(32);
    if (share == 128) SG_ROW(128);
    if (share == 256) SG_ROW(256);
    SG_ROW(512);
#undef SG_ROW
}

// Whether a row of `type`s may be read or written N elements at a time.
template <class T>
bool in_units(const void *p, long long ld, int n) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (n * sizeof(T)) == 0 && ld % n == 0);
}

template <class El, bool NORM, int OUT>
cudaError_t row_for(RowArgs a, int num_sms, cudaStream_t stream) {
    using T = typename El::T;
    constexpr int V = 16 / sizeof(T);
    auto fits = [&](int n) {
        return a.K % n == 0 && in_units<T>(a.X, a.ldx, n) && in_units<T>(a.R, a.ldr, n) && in_units<T>(a.W, 0, n) &&
               in_units<T>(a.H, a.ldh, n) && (OUT != OUT_Y || in_units<T>(a.Y, a.ldy, n));
    };
    const int unit = OUT == OUT_I8 ? V : V / 2;  // bytes of the result that A elements make
    a.vec = in_units<uint8_t>(a.Y, a.ldy, unit);
    if (fits(V)) return row_typed<El, V, NORM, OUT>(a, num_sms, stream);
    if (fits(2)) return row_typed<El, 2, NORM, OUT>(a, num_sms, stream);
    return row_typed<El, 1, NORM, OUT>(a, num_sms, stream);
}

template <bool NORM, int OUT>
cudaError_t row_any(int type, const RowArgs &a, int num_sms, cudaStream_t stream) {
    switch (type) {
        case SGEMM_IN_F32: return row_for<ElF32, NORM, OUT>(a, num_sms, stream);
        case SGEMM_IN_BF16: return row_for<ElBF16, NORM, OUT>(a, num_sms, stream);
        default: return row_for<ElF16, NORM, OUT>(a, num_sms, stream);
    }
}

// ---- 4 bits back -----------------------------------------------------------------
// Y[i][p] = row_i * s_ib * q_ip: the product of code and scale is exact, so there is one
// rounding in FP32 and one to the type.  A elements a thread and step, four steps in
// flight.
template <class El, int A, int FORMAT>
__global__ void __launch_bounds__(256)
dequantize_kernel(const RowArgs a, unsigned across) {
    using T = typename El::T;
    using W = typename AccessOf<static_cast<int>(sizeof(T)) * A>::T;
    constexpr int kSteps = 4;
    griddep_wait();
    griddep_launch_dependents();
    for (unsigned long long b = blockIdx.x; b < static_cast<unsigned long long>(across) * static_cast<unsigned>(a.M); b += gridDim.x) {
        const long long i = static_cast<long long>(b / across);
        const int at = static_cast<int>(b % across) * (256 * A * kSteps) + threadIdx.x * A;
        const uint8_t *q = static_cast<const uint8_t *>(a.X) + i * a.ldx;
        const uint8_t *s = a.S + fp4_scale_word(i, 0, a.words);
        T *y = static_cast<T *>(a.Y) + i * a.ldy;
        uint32_t code[kSteps], scale[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int p = at + k * 256 * A;
            code[k] = scale[k] = 0;
            if (p >= a.K) continue;
            if (A == 8) {
                if (a.vec) code[k] = __ldcg(reinterpret_cast<const uint32_t *>(q + p / 2));
                else
#pragma unroll
                    for (int j = 0; j < 4; ++j) code[k] |= static_cast<uint32_t>(__ldcg(q + p / 2 + j)) << (8 * j);
            } else if (A == 4) {
                if (a.vec) code[k] = __ldcg(reinterpret_cast<const uint16_t *>(q + p / 2));
                else code[k] = __ldcg(q + p / 2) | static_cast<uint32_t>(__ldcg(q + p / 2 + 1)) << 8;
            } else {
                code[k] = __ldcg(q + p / 2) >> (A == 1 && (p & 1) ? 4 : 0);
            }
            const int blk = p / fp4_block(FORMAT);
            scale[k] = __ldca(s + static_cast<long long>(blk / 4) * 512 + (blk & 3));
        }
        const float row = a.row ? __ldca(a.row + i) : 1.f;
        auto put = [&](float less, float row) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const int p = at + k * 256 * A;
                if (p >= a.K) continue;
                uint32_t h[4];
                from_e2m1x8(code[k], h);
                const float f = fp4_scale<FORMAT>(scale[k]) * less;
                alignas(16) T o[A];
#pragma unroll
                for (int e = 0; e < A; ++e) {
                    const float v = __half2float(__ushort_as_half(static_cast<uint16_t>(h[e / 2] >> (16 * (e & 1)))));
                    o[e] = El::down(__fmul_rn(__fmul_rn(v, f), row));
                }
                *reinterpret_cast<W *>(y + p) = *reinterpret_cast<const W *>(o);
            }
        };
        // A code times 2^126 or 2^127 (MX) may pass FP32's range where that times a small row scale does
        // not: such scales are taken at a quarter and the row's four times, both exact.
        const bool large = FORMAT == SGEMM_FP4_MX && max(max(scale[0], scale[1]), max(scale[2], scale[3])) >= 253u;
        if (large && fabsf(row) < 0x1p126f) put(0.25f, row * 4.f);
        else put(1.f, row);
    }
}

template <class El, int A, int FORMAT>
cudaError_t dequantize_typed(const RowArgs &a, int num_sms, cudaStream_t stream) {
    const unsigned across = blocks_of(a.K, 256 * A * 4);
    const unsigned long long blocks = static_cast<unsigned long long>(across) * static_cast<unsigned>(a.M), most = 64ull * num_sms;
    return launch_dependent(dequantize_kernel<El, A, FORMAT>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, stream, 1, a,
                            across);
}

template <class El>
cudaError_t dequantize_for(RowArgs a, int num_sms, cudaStream_t stream) {
    using T = typename El::T;
    constexpr int V = 16 / sizeof(T);
    a.vec = in_units<uint8_t>(a.X, a.ldx, V / 2);
    const bool wide = a.K % V == 0 && in_units<T>(a.Y, a.ldy, V), two = a.K % 2 == 0 && in_units<T>(a.Y, a.ldy, 2);
    if (a.format == SGEMM_FP4_MX)
        return wide ? dequantize_typed<El, V, SGEMM_FP4_MX>(a, num_sms, stream)
                    : two ? dequantize_typed<El, 2, SGEMM_FP4_MX>(a, num_sms, stream) : dequantize_typed<El, 1, SGEMM_FP4_MX>(a, num_sms, stream);
    return wide ? dequantize_typed<El, V, SGEMM_FP4_NV>(a, num_sms, stream)
                : two ? dequantize_typed<El, 2, SGEMM_FP4_NV>(a, num_sms, stream) : dequantize_typed<El, 1, SGEMM_FP4_NV>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_rms_norm(int type, RowOut out, const RowArgs &a, int num_sms, cudaStream_t stream) {
    switch (out) {
        case RowOut::kSame: return row_any<true, OUT_Y>(type, a, num_sms, stream);
        case RowOut::kInt8: return row_any<true, OUT_I8>(type, a, num_sms, stream);
        default: return row_any<true, OUT_F4>(type, a, num_sms, stream);
    }
}

cudaError_t launch_quantize_fp4(int type, const RowArgs &a, int num_sms, cudaStream_t stream) {
    return row_any<false, OUT_F4>(type, a, num_sms, stream);
}

cudaError_t launch_dequantize_fp4(int type, const RowArgs &a, int num_sms, cudaStream_t stream) {
    switch (type) {
        case SGEMM_IN_F32: return dequantize_for<ElF32>(a, num_sms, stream);
        case SGEMM_IN_BF16: return dequantize_for<ElBF16>(a, num_sms, stream);
        default: return dequantize_for<ElF16>(a, num_sms, stream);
    }
}

}  // namespace sg
