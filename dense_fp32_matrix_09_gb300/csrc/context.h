// What the entry points in sgemm_ops_api.cu need of a handle, which
// sgemm_api.cu owns, and the tensor-map encoder that it loads.
#pragma once

#include <cstddef>

#include <cuda.h>

#include "sgemm.h"

namespace sg {

struct HandleView {
    int device, num_sms;
    int *d_status;
    float *d_ws;       // stream-K workspace, ws_floats floats
    size_t ws_floats;
    float *d_rl;       // operand re-layout workspace (NULL: none), rl_bytes bytes
    size_t rl_bytes;
    int pinned, relayout_mode, smem_override;
    int i8_tokens, i8_split;  // test hook: the int8 products' token tile and K split (0: chosen)
};

bool is_live(sgemm_handle_t h);
void view_of(sgemm_handle_t h, HandleView *v);
// What sgemm_last_variant, _launches and _relayout report.
void record_call(sgemm_handle_t h, int variant, int splits, int launches, int copied);

enum class MapType { kInt8, kF16 };
// A row-major tensor (planes x rows x cols; dims 2: one plane) as a TMA map with
// the 128-byte swizzle; row and plane strides in bytes, the box in elements.
bool encode_map(CUtensorMap *map, MapType type, int dims, const void *base, long long cols, long long rows,
                long long planes, long long row_bytes, long long plane_bytes, int box_cols, int box_rows);

}  // namespace sg
