// evict.cu -- which tokens of a request stay, and their move into new pages
// (sm_103a).
#include <cuda_runtime.h>
#include <stdint.h>

#include "evict.cuh"
#include "launch.cuh"
#include "shkv_device.cuh"

namespace shkv {

namespace {

constexpr int kSelectThreads = 1024;

// A mass as an unsigned key of the same order: -0 as 0, every NaN on top.
__device__ __forceinline__ uint32_t mass_key(float m)
{
    if (m != m)
        return 0xffffffffu;
    const uint32_t u = __float_as_uint(m == 0.f ? 0.f : m);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

}  // namespace

// A CTA per (request, KV head).  The n-th largest key of the candidates (the
// tokens between the sinks and the recent ones) is found digit by digit, 8 bits
// at a time from the top, by a histogram of the candidates that share the
// digits found so far; then all above it and as many of its equals as still fit
// are written in order of position.
__global__ void __launch_bounds__(kSelectThreads) shkv_select_kernel(const __grid_constant__ SelectParams p)
{
    __shared__ uint32_t hist[256], digit, rest;
    __shared__ uint32_t warp_above[32], warp_equal[32];
    pdl_wait_prior();
    pdl_launch_dependents();
    const int b = blockIdx.x / p.hkv, g = blockIdx.x % p.hkv;
    const int L = p.lens[b], keep = min(p.keep[b], L);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    int32_t *out = p.index + ((int64_t)b * p.hkv + g) * p.index_stride;
    if (g == 0 && threadIdx.x == 0 && p.seq_lens[b] != L)
        atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
    for (int64_t j = keep + threadIdx.x; j < p.index_stride; j += kSelectThreads)
        out[j] = -1;
    if (keep == L) {
        for (int j = threadIdx.x; j < L; j += kSelectThreads)
            out[j] = j;
        return;
    }
    const float *m = p.mass + b * p.mass_request + g * p.mass_head;
    const int lo = p.sink, hi = L - p.recent;
    uint32_t prefix = 0u, need = (uint32_t)(keep - p.sink - p.recent);   // of the keys with this prefix
    for (int shift = 24; shift >= 0 && need; shift -= 8) {
        if (threadIdx.x < 256)
            hist[threadIdx.x] = 0u;
        __syncthreads();
        for (int t = lo + threadIdx.x; t < hi; t += kSelectThreads) {
            const uint32_t u = mass_key(m[t]);
            if (shift == 24 || (u ^ prefix) >> (shift + 8) == 0u)
                atomicAdd(&hist[u >> shift & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int d = 255;
            uint32_t left = need;
            for (; hist[d] < left; --d)
                left -= hist[d];
            digit = (uint32_t)d;
            rest = left;
        }
        __syncthreads();
        prefix |= digit << shift;
        need = rest;
    }
    // `need` of the keys equal to `prefix` stay, all larger ones do
    const bool any = keep - p.sink - p.recent > 0;
    int above0 = 0, equal0 = 0;                          // kept above, equals met, before this pass
    for (int t0 = 0; t0 < L; t0 += kSelectThreads) {
        const int t = t0 + threadIdx.x;
        bool above = false, equal = false;
        if (t < L) {
            if (t < lo || t >= hi) {
                above = true;
            } else if (any) {
                const uint32_t u = mass_key(m[t]);
                above = u > prefix;
                equal = u == prefix;
            }
        }
        const uint32_t ba = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, equal);
        if (lane == 0) {
            warp_above[warp] = (uint32_t)__popc(ba);
            warp_equal[warp] = (uint32_t)__popc(be);
        }
        __syncthreads();
        int a = above0, e = equal0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) {
                a += (int)warp_above[w];
                e += (int)warp_equal[w];
            }
            above0 += (int)warp_above[w];
            equal0 += (int)warp_equal[w];
        }
        const uint32_t before = (1u << lane) - 1u;
        a += __popc(ba & before);
        e += __popc(be & before);
        const int at = a + min(e, (int)need);
        if ((above || (equal && e < (int)need)) && at < keep)   // always, unless masses change under the call
            out[at] = t;
        __syncthreads();
    }
}

cudaError_t launch_select(const SelectParams &p, cudaStream_t stream)
{
    return launch_pdl(shkv_select_kernel, p.batch * p.hkv, kSelectThreads, 0u, stream, p);
}

namespace {
constexpr int kMoveThreads = 256;
}

// The first blocks move masses, a CTA per (request, KV head): a pass reads its
// masses before any is written, and as positions ascend it writes only below
// what later passes read.  The others copy rows, a warp per (new page, KV head).
__global__ void __launch_bounds__(kMoveThreads) shkv_evict_kernel(const __grid_constant__ EvictParams p)
{
    pdl_wait_prior();
    pdl_launch_dependents();
    const int mass_blocks = p.mass.out ? p.batch * p.hkv : 0;
    if ((int)blockIdx.x < mass_blocks) {
        const int b = blockIdx.x / p.hkv, g = blockIdx.x % p.hkv;
        const int L = p.lens[b], keep = p.keep[b];
        if (keep >= L)
            return;
        const int32_t *index = p.index + ((int64_t)b * p.hkv + g) * p.index_stride;
        const float *src = p.mass.in + b * p.mass.in_request + g * p.mass.in_head;
        float *dst = p.mass.out + b * p.mass.out_request + g * p.mass.out_head;
        for (int j0 = 0; j0 < L; j0 += kMoveThreads) {
            const int j = j0 + threadIdx.x;
            float x = 0.f;
            if (j < keep) {
                const int i = index[j];
                if ((uint32_t)i < (uint32_t)L)
                    x = src[i];
            }
            __syncthreads();
            if (j < L)
                dst[j] = x;
        }
        return;
    }
    const int lane = threadIdx.x & 31, vecs = p.head_dim / 8, P = p.page_size;
    const int w = (blockIdx.x - mass_blocks) * (kMoveThreads / 32) + threadIdx.x / 32;
    if (w >= p.page0[p.batch] * p.hkv)
        return;
    const int page = w / p.hkv, g = w % p.hkv;
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.page0[mid] <= page)
            lo = mid;
        else
            hi = mid;
    }
    const int b = lo, j0 = (page - p.page0[b]) * P, n = min(P, p.keep[b] - j0);
    const int to = p.new_table[b * p.new_stride + j0 / P];
    bool ok = (uint32_t)to < (uint32_t)p.num_pages;
    int64_t row = 0;                                     // of the lane's token
    if (!ok) {
        atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
    } else if (lane < n) {
        const int i = p.index[((int64_t)b * p.hkv + g) * p.index_stride + j0 + lane];
        ok = (uint32_t)i < (uint32_t)p.lens[b];
        if (!ok) {
            atomicOr(p.err, SHKV_ERRF_INDEX);
        } else {
            const int from = p.table[b * p.table_stride + i / P];
            ok = (uint32_t)from < (uint32_t)p.num_pages;
            if (!ok)
                atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
            row = ((int64_t)from * p.hkv + g) * P + i % P;
        }
    }
    const uint32_t good = __ballot_sync(0xffffffffu, ok && lane < n);
    const int64_t dst0 = ((int64_t)to * p.hkv + g) * P;
    for (int e = lane; e < 2 * P * vecs; e += 32) {
        const int j = e / (2 * vecs), kv = e / vecs % 2, v = e % vecs;
        const int64_t src = __shfl_sync(0xffffffffu, row, j);
        if (good >> j & 1u) {
            uint4 *pages = kv ? p.v_pages : p.k_pages;
            pages[(dst0 + j) * vecs + v] = pages[src * vecs + v];
        }
    }
}

// After the move: the requests' tables and lengths.  Lets no dependent start
// early: the unit kernel of a decode with tails reads the table without waiting
// for its predecessor.
__global__ void __launch_bounds__(kMoveThreads) shkv_evict_commit_kernel(const __grid_constant__ EvictParams p)
{
    pdl_wait_prior();
    const int b = blockIdx.x;
    const int keep = p.keep[b];
    if (p.check_lens && threadIdx.x == 0 && p.seq_lens[b] != p.lens[b])
        atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
    if (keep >= p.lens[b])
        return;
    for (int i = threadIdx.x; i < p.max_pages; i += kMoveThreads)
        p.block_table[(int64_t)b * p.max_pages + i] = i < p.new_stride ? p.new_table[b * p.new_stride + i] : -1;
    __syncthreads();
    if (threadIdx.x == 0)
        p.seq_lens[b] = keep;
}

cudaError_t launch_evict(const EvictParams &p, cudaStream_t stream)
{
    const int64_t warps = (int64_t)p.page0[p.batch] * p.hkv;
    const int64_t grid = (p.mass.out ? (int64_t)p.batch * p.hkv : 0) + (warps + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
    cudaError_t e = grid ? launch_pdl(shkv_evict_kernel, (int)grid, kMoveThreads, 0u, stream, p) : cudaSuccess;
    if (e == cudaSuccess)
        e = launch_pdl(shkv_evict_commit_kernel, p.batch, kMoveThreads, 0u, stream, p);
    return e;
}

}  // namespace shkv
