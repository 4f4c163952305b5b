// q8_cache.cu -- append to the 8-bit KV cache, quantising as the tokens are
// written, and the read back to bf16 (sm_103a).
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.cuh"
#include "q8.cuh"
#include "shkv_device.cuh"

namespace shkv {

namespace {

constexpr int kCacheThreads = 256;

// Request of packed token t: the last b with tok0[b] <= t.
__device__ __forceinline__ int q8_request(const Q8CacheParams &p, int t)
{
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.tok0[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

constexpr int kVecs = 8;             // vectors of a token that a lane has in flight

// A warp's tokens [t, end) of the packed rows and the slot of the current one.
struct Q8Walk {
    int t, end, b, lim, pos;         // token, last + 1, its request, that request's last token + 1, position
};

// Tokens are dealt to the warps in runs, so that the request is searched once.
__device__ __forceinline__ Q8Walk q8_walk(const Q8CacheParams &p)
{
    const int n = p.tok0[p.batch];
    const int warps = gridDim.x * (kCacheThreads / 32);
    const int per = (n + warps - 1) / warps;
    Q8Walk w;
    w.t = min((int64_t)n, (int64_t)(blockIdx.x * (kCacheThreads / 32) + threadIdx.x / 32) * per);
    w.end = min(n, w.t + per);
    if (w.t < w.end) {
        w.b = q8_request(p, w.t);
        w.lim = p.tok0[w.b + 1];
        w.pos = p.start[w.b] + w.t - p.tok0[w.b];
    }
    return w;
}

__device__ __forceinline__ void q8_next(const Q8CacheParams &p, Q8Walk &w)
{
    ++w.t;
    ++w.pos;
    if (w.t < w.end && w.t == w.lim) {
        do
            ++w.b;
        while (p.tok0[w.b + 1] <= w.t);
        w.lim = p.tok0[w.b + 1];
        w.pos = p.start[w.b] + w.t - p.tok0[w.b];
    }
}

// The token's page, -1 (and flagged) if it lies outside the pool.
__device__ __forceinline__ int q8_page(const Q8CacheParams &p, const Q8Walk &w, int log2P)
{
    const int page = __ldg(p.block_table + (int64_t)w.b * p.max_pages + (w.pos >> log2P));
    if (page >= 0 && page < p.num_pages)
        return page;
    if ((threadIdx.x & 31) == 0)
        atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
    return -1;
}

}  // namespace

// A warp per token, D/8 lanes a row of 8 bf16 values a lane.  The row's
// largest magnitude is an integer maximum of the bf16 bits (their order is
// the values', infinities and NaN above all finite ones).  Bound by bytes; a
// lane's vectors of a token are loaded together so that enough are in flight.
template <int D>
__global__ void __launch_bounds__(kCacheThreads) shkv_q8_append_kernel(const __grid_constant__ Q8CacheParams p)
{
    pdl_wait_prior();
    pdl_launch_dependents();
    constexpr int LR = D / 8, RW = 32 / LR;              // lanes a row, rows a warp's pass
    const int lane = threadIdx.x & (LR - 1), sub = (threadIdx.x & 31) / LR;
    const int log2P = 31 - __clz(p.page_size);
    const int rows = 2 * p.hkv;
    for (Q8Walk w = q8_walk(p); w.t < w.end; q8_next(p, w)) {
        const int page = q8_page(p, w, log2P);
        if (page < 0)
            continue;
        const __nv_bfloat16 *ks = p.k + w.t * p.k_stride, *vs = p.v + w.t * p.v_stride;
        const int64_t unit0 = (int64_t)page * p.hkv;
        const int slot = w.pos & (p.page_size - 1);
        for (int r0 = 0; r0 < rows; r0 += kVecs * RW) {
            uint4 x[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int r = r0 + i * RW + sub;
                x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows)
                    x[i] = __ldg(reinterpret_cast<const uint4 *>((r < p.hkv ? ks + r * D : vs + (r - p.hkv) * D)) + lane);
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int r = r0 + i * RW + sub;
                const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t a = __vmaxu2(__vmaxu2(xs[0] & 0x7fff7fffu, xs[1] & 0x7fff7fffu),
                                      __vmaxu2(xs[2] & 0x7fff7fffu, xs[3] & 0x7fff7fffu));
                a = max(a & 0xffffu, a >> 16);
#pragma unroll
                for (int o = LR / 2; o > 0; o >>= 1)
                    a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
                // 448 = 1.75 * 2^8: one binade more where the significand is above 1.75
                int byte = (int)(a >> 7) - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0);
                byte = byte < 0 ? 0 : byte;
                const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);   // 2^-e
                uint32_t c[4];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    c[v] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(xs[v] << 16) * inv,
                                                                __uint_as_float(xs[v] & 0xffff0000u) * inv),
                                                    __NV_SATFINITE, __NV_E4M3);
                uint2 q = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                if (a >= 0x7f80u) {
                    byte = 255;
                    q.x = q.y = 0x7f7f7f7fu;
                }
                if (r < rows) {
                    const int kv = r >= p.hkv;
                    const int64_t unit = unit0 + r - kv * p.hkv;
                    reinterpret_cast<uint2 *>((kv ? p.v_pages : p.k_pages) + ((unit << log2P) + slot) * D)[lane] = q;
                    if (lane == 0)
                        p.scales[((unit * 2 + kv) << log2P) + slot] = (uint8_t)byte;
                }
            }
        }
    }
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.batch; b += kCacheThreads) {
            if (p.seq_lens[b] != p.old_len[b])
                atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
            p.seq_lens[b] = p.start[b] + p.tok0[b + 1] - p.tok0[b];
        }
}

// The rows of the ranges as bf16, exact (q * 2^e has a 4-bit significand);
// the rows of a page outside the pool are zero.
template <int D>
__global__ void __launch_bounds__(kCacheThreads) shkv_q8_read_kernel(const __grid_constant__ Q8CacheParams p)
{
    pdl_wait_prior();
    pdl_launch_dependents();
    constexpr int LR = D / 8, RW = 32 / LR;
    const int lane = threadIdx.x & (LR - 1), sub = (threadIdx.x & 31) / LR;
    const int log2P = 31 - __clz(p.page_size);
    const int rows = 2 * p.hkv;
    for (Q8Walk w = q8_walk(p); w.t < w.end; q8_next(p, w)) {
        const int page = q8_page(p, w, log2P);
        __nv_bfloat16 *kd = p.k + w.t * p.k_stride, *vd = p.v + w.t * p.v_stride;
        const int64_t unit0 = (int64_t)page * p.hkv;
        const int slot = w.pos & (p.page_size - 1);
        for (int r0 = 0; r0 < rows; r0 += kVecs * RW) {
            uint2 c[kVecs];
            uint32_t s[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int r = r0 + i * RW + sub;
                c[i] = make_uint2(0u, 0u);
                s[i] = 0u;
                if (r < rows && page >= 0) {
                    const int kv = r >= p.hkv;
                    const int64_t unit = unit0 + r - kv * p.hkv;
                    c[i] = __ldg(reinterpret_cast<const uint2 *>((kv ? p.v_pages : p.k_pages) +
                                                                 ((unit << log2P) + slot) * D) + lane);
                    s[i] = __ldg(p.scales + ((unit * 2 + kv) << log2P) + slot);
                }
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int r = r0 + i * RW + sub;
                const float f = q8_scale(s[i]);
                const uint32_t cs[2] = {c[i].x, c[i].y};
                uint32_t o[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float2 x = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
                        (__nv_fp8x2_storage_t)(cs[v >> 1] >> (16 * (v & 1))), __NV_E4M3)));
                    o[v] = pack_bf16x2(x.x * f, x.y * f);
                }
                if (r < rows)
                    reinterpret_cast<uint4 *>(r < p.hkv ? kd + r * D : vd + (r - p.hkv) * D)[lane] =
                        make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.batch; b += kCacheThreads)
            if (p.seq_lens[b] != p.old_len[b])
                atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
}

cudaError_t launch_q8_cache(const Q8CacheParams &p, bool read, int num_sms, cudaStream_t stream)
{
    int64_t blocks = ((int64_t)p.tok0[p.batch] + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
    if (blocks > (int64_t)num_sms * 4)
        blocks = (int64_t)num_sms * 4;
    if (blocks < 1)
        blocks = 1;
    auto kern = read ? (p.head_dim == 64 ? shkv_q8_read_kernel<64> : shkv_q8_read_kernel<128>)
                     : (p.head_dim == 64 ? shkv_q8_append_kernel<64> : shkv_q8_append_kernel<128>);
    return launch_pdl(kern, (int)blocks, kCacheThreads, 0u, stream, p);
}

}  // namespace shkv
