// evict.cuh -- eviction by accumulated attention weight: parameter blocks of
// the kernels (internal to the library).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "shkv.h"

namespace shkv {

// These kernels may start while the one before them in the stream still writes what
// they read after their wait (log-sum-exps, masses, indexes, tables), so they read
// it by ordinary loads: __ldg wants data that stays as it is for a kernel's lifetime.

// Masses read and written; `in` may be null (nothing to read).
struct MassIo {
    const float *in;
    float *out;
    int64_t in_request, in_head, out_request, out_head;
};

constexpr int kMassMaxCtas = 256;
constexpr int kMassTile = 128;       // tokens of a tile: rows of an MMA
constexpr int kWide = 2 * kMassTile; // tokens of an item with many blocks
constexpr int kMassRows = 128;       // query rows of a block, at most

// Blocks of rows from which rows lie on the MMA's M dimension.  (16 requests of 4K to
// 15K tokens, 8 KV heads of 128, blocks of 32 query tokens: two blocks 76 us with
// tokens on M and 84 with rows on M, three 116 and 104.  By the blocks alone: heads of
// 64 would be 4% faster with tokens on M at three blocks, 97 us against 101, and two
// requests of 3000 tokens a tenth faster with rows on M at two, 12.4 against 14.0.)
inline bool mass_wide(int32_t blocks) { return blocks >= 3; }

// A decode step or a chunk: row r = i * G + j of a (request, KV head g) is
// query token i, head g * G + j.  Causal: query token i sits at position
// L_b - n_q + i.  Blocks of `tpt` query tokens, `blocks` in all; an item is
// kMassTile (few blocks) or kWide consecutive tokens of a (request, KV head), items
// are numbered request-major, then by head.  CTA c takes the blocks from (cut_item[c],
// cut_block[c]) up to (cut_item[c + 1], cut_block[c + 1]); block 0 stands for
// the item's first.
struct MassParams {
    const float *lse;                // query token i's [Hq] at b * lse_request + i * lse_token
    int64_t lse_request, lse_token;
    MassIo mass;
    const int32_t *block_table, *seq_lens;
    uint32_t *err;
    float *pieces;                   // [2 * CTAs, kWide]: sums of a range's first and last, cut item
    int32_t batch, n_q, hkv, group, head_dim, page_size, max_pages, num_pages, causal;
    int32_t tpt, blocks, item_tokens, num_ctas;
    float scale_log2, decay;
    int32_t cut_item[kMassMaxCtas + 1];
    int32_t cut_block[kMassMaxCtas + 1];
    int32_t lens[SHKV_MAX_BATCH];
    int32_t item0[SHKV_MAX_BATCH + 1];   // items before each request
};

// Tokens that every query token of a request sees.
__host__ __device__ inline int mass_past(int len, int n_q, int causal) { return causal ? len - n_q : len; }

// First block with a row that sees token t.
__host__ __device__ inline int mass_block0(int t, int past, int tpt) { return t > past ? (t - past) / tpt : 0; }

// First row of the block of query tokens i0 .. that sees token t of a tile that the
// block sees.  0 where all rows do: the distance to a token far back, times the
// group, would not fit 32 bits (34M tokens and 64 rows).
__host__ __device__ inline int mass_first_row(int t, int past, int i0, int group)
{
    const int tokens = t - past - i0;
    return tokens > 0 ? tokens * group : 0;
}

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
    int32_t at_once;                 // tables and lengths beside the move: it reads neither
    int32_t lens[SHKV_MAX_BATCH];
    int32_t keep[SHKV_MAX_BATCH];
    int32_t page0[SHKV_MAX_BATCH + 1];   // new pages before each request
};

// What is added to a row's scores in base 2: its log-sum-exp off, at most the
// largest number; kRowOut for a row that attends nothing.  Such a row is left out by
// this mark: its scores may be infinite or no number, which adding -inf would not
// make a weight of 0.
constexpr float kRowOut = INFINITY, kLargest = 3.402823466e38f;

__device__ __forceinline__ float lse_offset(float lse)
{
    const float l = lse * -1.4426950408889634f;
    return lse == -INFINITY ? kRowOut : l == INFINITY ? kLargest : l;
}

}  // namespace shkv
