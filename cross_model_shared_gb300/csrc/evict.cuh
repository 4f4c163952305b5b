// evict.cuh -- eviction by accumulated attention weight: parameter blocks of
// the kernels (internal to the library).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "shkv.h"

namespace shkv {

// Masses read and written; `in` may be null (nothing to read).
struct MassIo {
    const float *in;
    float *out;
    int64_t in_request, in_head, out_request, out_head;
};

// A decode step or a chunk: row r = i * G + j of a (request, KV head g) is
// query token i, head g * G + j.  Causal: query token i sits at position
// L_b - n_q + i.
struct MassParams {
    const __nv_bfloat16 *k_pages;    // [num_pages, Hkv, P, D]
    const __nv_bfloat16 *q;          // query token i's rows [Hq, D] at b * q_request + i * q_token
    const float *lse;                // ... and its [Hq]
    int64_t q_request, q_token, lse_request, lse_token;
    MassIo mass;
    const int32_t *block_table, *seq_lens;
    uint32_t *err;
    int32_t batch, n_q, hq, hkv, group, head_dim, page_size, max_pages, num_pages, causal;
    float scale_log2, decay;
    int32_t lens[SHKV_MAX_BATCH];
    int32_t tile0[SHKV_MAX_BATCH + 1];   // 128-token tiles of one KV head before each request
};

struct SelectParams {
    const float *mass;
    int64_t mass_request, mass_head, index_stride;
    int32_t *index;
    const int32_t *seq_lens;
    uint32_t *err;
    int32_t batch, hkv, sink, recent;
    int32_t lens[SHKV_MAX_BATCH];
    int32_t keep[SHKV_MAX_BATCH];
};

// Request b of the moved ones: keep[b] < lens[b].
struct EvictParams {
    uint4 *k_pages, *v_pages;
    const int32_t *index, *table, *new_table;
    int64_t index_stride, table_stride, new_stride;
    MassIo mass;                     // out null: none
    int32_t *block_table, *seq_lens;
    uint32_t *err;
    int32_t batch, hkv, head_dim, page_size, max_pages, num_pages, check_lens;
    int32_t lens[SHKV_MAX_BATCH];
    int32_t keep[SHKV_MAX_BATCH];
    int32_t page0[SHKV_MAX_BATCH + 1];   // new pages before each request
};

// What a row's log-sum-exp takes off its scores, in base 2: +inf for a row
// that attends nothing, so that all its weights are 0.
__device__ __forceinline__ float lse_base2(float lse)
{
    return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
}

}  // namespace shkv
