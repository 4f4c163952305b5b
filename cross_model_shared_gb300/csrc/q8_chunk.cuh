// q8_chunk.cuh -- parameters of the causal chunk attention over the 8-bit
// cache (q8_chunk.cu), shared with its host side (q8_host.cu).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "shkv.h"

namespace shkv {

constexpr int kChunkMaxCtas = 256;
constexpr int kChunkRows = 256;      // query rows of a unit: two MMA tiles

// A unit is two consecutive query tiles of one (request, KV head); units are
// numbered request-major, then by head, then by tile pair.  CTA c takes the
// key stages from (cut_unit[c], cut_stage[c]) up to (cut_unit[c + 1],
// cut_stage[c + 1]).
struct Q8ChunkParams {
    const __nv_bfloat16 *q;          // [query tokens, Hq, D]
    int64_t q_stride;                // elements from a query token to the next
    __nv_bfloat16 *out;              // [query tokens, Hq, D]
    float *lse_out;                  // [query tokens, Hq] or null
    const uint8_t *scales;           // [num_pages, Hkv, 2, P]
    const int32_t *block_table, *seq_lens;
    uint32_t *err;
    float *ws_lse;                   // [2 * CTAs, kChunkRows]
    float *ws_part;                  // [2 * CTAs, 2, D / 4, 128, 4]: four columns of a tile's rows together
    int32_t batch, hq, hkv, group, head_dim, page_size, max_pages, num_pages;
    int32_t tpt;                     // new tokens per tile
    int32_t num_ctas;
    float scale_log2;
    int32_t cut_unit[kChunkMaxCtas + 1];
    int32_t cut_stage[kChunkMaxCtas + 1];
    int32_t units[SHKV_MAX_BATCH + 1];   // units before each request
    int32_t lens[SHKV_MAX_BATCH];
    int32_t n_q[SHKV_MAX_BATCH];
    int32_t q0[SHKV_MAX_BATCH];
};

// Key stages of 128 that tile pair tp of a request attends.
__host__ __device__ inline int chunk_stages(int len, int n, int tpt, int tp)
{
    const int last = (2 * tp + 2) * tpt;
    return (len - n + (last < n ? last : n) + 127) / 128;
}

}  // namespace shkv
