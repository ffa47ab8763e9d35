// 4-bit floating point (E2M1: sign, two bits of exponent, one of fraction: 0, 0.5,
// 1, 1.5, 2, 3, 4, 6) with a scale a block: what the kernels that write it and
// those that multiply it share.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "sgemm.h"

namespace sg {

// Elements a scale is for.
__host__ __device__ constexpr int fp4_block(int format) { return format == SGEMM_FP4_MX ? 32 : 16; }
// Words of four scales that a row has.
__host__ __device__ constexpr int fp4_words(int format, int K) {
    return (K + 4 * fp4_block(format) - 1) / (4 * fp4_block(format));
}

// Scales lie in tiles of 128 rows x 4 blocks (512 bytes), the layout in which
// the tensor cores take them: a row's four scales are one word, row r's word 16 *
// (r % 32) + 4 * (r / 32) bytes from the tile's start; the tiles of 128 rows follow
// one another along K.
__host__ __device__ __forceinline__ long long fp4_scale_word(long long row, int word, int words) {
    return (row / 128 * words + word) * 512 + row % 32 * 16 + row % 128 / 32 * 4;
}

#ifdef __CUDACC__
// Eight values to their codes, the first in the lowest four bits: nearest, ties to
// the even code, magnitudes above 6 to 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The eight values of a word of codes as four pairs of FP16 (exact).
__device__ __forceinline__ void from_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// A positive value to an E4M3 scale (nearest, ties to even, at most 448), and back.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
    return r & 0xffu;
}
__device__ __forceinline__ float from_e4m3(uint32_t code) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
}

// 2^n for n in [-126, 127].
__device__ __forceinline__ float exp2_of(int n) { return __int_as_float((n + 127) << 23); }

// The value of an E8M0 scale: 2^(code - 127), 255 a NaN (BF16 has all of them).
__device__ __forceinline__ float from_e8m0(uint32_t code) {
    uint32_t b;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(b) : "h"(static_cast<uint16_t>(code)));
    return __uint_as_float(b << 16);
}
template <int FORMAT>
__device__ __forceinline__ float fp4_scale(uint32_t code) {
    return FORMAT == SGEMM_FP4_MX ? from_e8m0(code) : from_e4m3(code);
}
#endif

}  // namespace sg
