// q8.cuh -- the 8-bit shared KV cache: parameter blocks of its kernels and
// the device pieces they share (internal to the library).
//
// Format.  A (token, KV head) row x[0 .. D) of K or of V is held as D e4m3
// codes q_i and one scale byte s:
//
//   q_i = e4m3(x_i * 2^-e), rounded to nearest even;   x_i ~ q_i * 2^e
//   e = the least integer with max|x_i| <= 448 * 2^e, at least -127; s = e + 127
//
// A power of two loses nothing against any other scale: dividing by it is
// exact and e4m3 is a floating format, so only the 4-bit significands are
// rounded (at most 2^-4 of a value; values under 2^-6 after scaling, 2^-14.8 to
// 2^-13.8 of the row's largest, fall on the subnormal grid).  q_i * 2^e is exact
// in bf16 but at its ends: its smallest subnormals, and a value of 1.9375 * 2^127
// or more, whose code at e = 120 is 256 and which so reads back as an infinity.
// A row that holds an infinity or a NaN has s = 255 and every code 0x7f (NaN); a
// zero row has s = 0.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "shkv.h"

namespace shkv {

// Kernel parameters of append and read: token t of the packed rows
// [tok0[b], tok0[b + 1]) is position start[b] + t - tok0[b] of request b.
struct Q8CacheParams {
    __nv_bfloat16 *k, *v;            // packed rows [tokens, Hkv, D]: read by append, written by read
    int64_t k_stride, v_stride;      // elements from a token's rows to the next one's
    uint8_t *k_pages, *v_pages;      // e4m3 [num_pages, Hkv, P, D]
    uint8_t *scales;                 // [num_pages, Hkv, 2, P]: K's, then V's
    const int32_t *block_table;
    int32_t *seq_lens;
    uint32_t *err;
    int32_t batch, hkv, head_dim, page_size, max_pages, num_pages;
    int32_t tok0[SHKV_MAX_BATCH + 1];
    int32_t start[SHKV_MAX_BATCH];
    int32_t old_len[SHKV_MAX_BATCH]; // host copy of the lengths before the call
};

// An attention call, before its requests are dealt to the kernels.  Request b has n_q[b] query tokens (the
// decoders of a decode step, or the new tokens of a chunk) from packed query
// token q0[b] on; row r = i * G + j of a (request, KV head g) is query token
// i, head g * G + j.
struct Q8AttnParams {
    const __nv_bfloat16 *q;          // [query tokens, Hq, D]
    int64_t q_stride;                // elements from a query token to the next
    __nv_bfloat16 *out;              // [query tokens, Hq, D]
    float *lse_out;                  // [query tokens, Hq] or null
    const uint8_t *scales;
    const int32_t *block_table, *seq_lens;
    uint32_t *err;
    int32_t batch, hq, hkv, group, head_dim, page_size, max_pages, num_pages, causal;
    float scale_log2;
    int32_t lens[SHKV_MAX_BATCH];
    int32_t n_q[SHKV_MAX_BATCH];
    int32_t q0[SHKV_MAX_BATCH];
};

// 2^(byte - 127) in fp32, exact; NaN for byte 255.
__device__ __forceinline__ float q8_scale(uint32_t byte)
{
    return __uint_as_float(byte << 23 | (byte == 0u || byte == 255u ? 1u << 22 : 0u));
}

// The larger of two; NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

}  // namespace shkv
