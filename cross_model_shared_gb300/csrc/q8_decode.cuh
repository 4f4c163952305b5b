// q8_decode.cuh -- parameters of the stacked-rows attention over the 8-bit
// cache (q8_decode.cu), shared with its host side (q8_host.cu).
#pragma once

#include <stdint.h>

#include "q8.cuh"
#include "shkv_device.cuh"

namespace shkv {

// d: the split plan, the rows' layout (rows: the largest unit's), the outputs
// and the workspace of a decode launch; d.q is read with q_stride.
struct Q8DecodeParams {
    DecodeParams d;
    const uint8_t *scales;           // [num_pages, Hkv, 2, P]
    int64_t q_stride;                // elements from a query token to the next
    int32_t head_dim, causal, has_empty;
    int32_t n_q[SHKV_MAX_BATCH];     // query tokens of each request (see Q8AttnParams)
    int32_t q0[SHKV_MAX_BATCH];
};

}  // namespace shkv
