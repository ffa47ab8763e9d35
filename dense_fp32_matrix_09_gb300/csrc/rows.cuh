// What the kernels on rows of FP32, BF16 or FP16 share: the element types and
// the accesses by which several threads read or write a row's pieces.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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

// SHARED: through L1, for what several rows' threads read.
template <class T, int TPR, int A, bool SHARED = false>
__device__ __forceinline__ Pack8<T> load8(const T *row, int c, int lane, int width) {
    using W = typename AccessOf<static_cast<int>(sizeof(T)) * A>::T;
    Pack8<T> r;
    const int at = c * kV * TPR + lane * A;
    const W *p = reinterpret_cast<const W *>(row + at);
    W *d = reinterpret_cast<W *>(&r);
#pragma unroll
    for (int i = 0; i < kV / A; ++i)
        d[i] = at + i * TPR * A < width ? (SHARED ? __ldca(p + i * TPR) : __ldcg(p + i * TPR)) : W{};
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

// Blocks of `per` of n > 0 rows (n up to 2^31 - 1).
constexpr unsigned blocks_of(int n, int per) { return static_cast<unsigned>((n - 1) / per + 1); }

}  // namespace
}  // namespace sg
