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

// cuTensorMapEncodeTiled, or null where the driver has none.
EncodeTiledFn encode_tiled_fn();

}  // namespace shkv
