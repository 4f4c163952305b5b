// host_shared.h -- host-side pieces of shkv_host.cu that the 8-bit cache's
// entry points use as well (internal to the library).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include <initializer_list>

#include "shkv.h"

namespace shkv {

// Device bytes [lo, hi).
struct Span {
    uintptr_t lo, hi;
};

Span span_of(const void *p, size_t bytes);

// What a call's kernels on `stream` read and write: every call that enqueues
// one of the library's kernels records it (a later tails call on the stream
// places its tables clear of these bytes).
void record_stream_use(const void *stream, std::initializer_list<Span> spans);

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The split plan of a decode (build_plan in shkv_host.cu) over requests of
// `lens` tokens, zero allowed, under costs in tokens of one KV head: a range
// pays its stages whole, `seg` a piece, `first` / `last` for an opening /
// closing split piece.  prefix [batch + 1], last_fill [batch], cuts
// [max_ctas + 1].
shkv_status plan_pages(int32_t batch, const int32_t *lens, int32_t page_size, int32_t hkv, int32_t max_ctas,
                       int64_t stage, int64_t seg, int64_t first, int64_t last, int32_t *prefix, uint8_t *last_fill,
                       int32_t *cuts, int64_t *total_chunks, int32_t *num_ctas);

// cuTensorMapEncodeTiled, or null where the driver has none.
EncodeTiledFn encode_tiled_fn();

}  // namespace shkv
