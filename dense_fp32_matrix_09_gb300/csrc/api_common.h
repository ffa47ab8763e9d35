// What the entry points on rows, 8- and 4-bit products and experts share: the
// checks that each of them makes and the ends of a call.
#pragma once

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "context.h"
#include "internal.h"
#include "sgemm.h"

namespace {

inline int from_cuda(cudaError_t e) {
    switch (e) {
        case cudaSuccess: return SGEMM_OK;
        case cudaErrorInvalidValue:
        case cudaErrorInvalidConfiguration:
        case cudaErrorLaunchOutOfResources:
        case cudaErrorInvalidDeviceFunction:
        case cudaErrorNoKernelImageForDevice: return SGEMM_ERR_LAUNCH;
        default: return SGEMM_ERR_CUDA;
    }
}

inline bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }
inline bool known_type(int t) { return t == SGEMM_IN_F32 || t == SGEMM_IN_BF16 || t == SGEMM_IN_F16; }
inline int size_of(int t) { return t == SGEMM_IN_F32 ? 4 : 2; }

// Byte range of a buffer that a call reads or writes.
struct Range {
    uintptr_t lo = 0, hi = 0;
    Range() {}
    Range(const void *p, long long rows, long long cols, long long ld, int size)
        : lo(reinterpret_cast<uintptr_t>(p)),
          hi(rows > 0 && cols > 0 ? lo + ((rows - 1) * static_cast<uintptr_t>(ld) + cols) * size : lo) {}
    bool meets(const Range &o) const { return lo < o.hi && o.lo < hi && lo < hi && o.lo < o.hi; }
};

// Rows, channels and elements of a row that the kernels' 32-bit indices reach with
// a tile to spare.
constexpr int kMaxExtent = 1 << 30;

// The checks every call starts with.
inline int enter(sgemm_handle_t h) {
    if (!sg::is_live(h)) return SGEMM_ERR_BAD_HANDLE;
    sg::HandleView v;
    sg::view_of(h, &v);
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != v.device) return SGEMM_ERR_WRONG_DEVICE;
    return SGEMM_OK;
}

// A call that had nothing to do: what the getters report of it.
inline int nothing(sgemm_handle_t h) {
    sg::record_call(h, -1, 1, 0, 0);
    return SGEMM_OK;
}

// The end of a call of one launch: recorded where it was enqueued.
inline int launched(sgemm_handle_t h, cudaError_t e) {
    if (e == cudaSuccess) sg::record_call(h, -1, 1, 1, 0);
    return from_cuda(e);
}

inline int check_row(int type, int width, int ld) {
    return known_type(type) && width >= 0 && width <= kMaxExtent && ld >= std::max(1, width) ? SGEMM_OK : SGEMM_ERR_INVALID_VALUE;
}

}  // namespace
