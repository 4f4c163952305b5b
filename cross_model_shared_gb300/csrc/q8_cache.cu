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

// One (token, K or V, head) row of a packed operand, by a group of D/8 lanes.
struct Q8Row {
    bool ok;
    int tok, head, kv;               // packed token, KV head, 0 = K / 1 = V
    int64_t row;                     // (page * Hkv + head) * P + slot
    int64_t scale;                   // its byte in `scales`
};

__device__ __forceinline__ Q8Row q8_row(const Q8CacheParams &p, int64_t r, bool in, bool flag)
{
    Q8Row w;
    w.ok = false;
    w.tok = w.head = w.kv = 0;
    w.row = w.scale = 0;
    if (!in)
        return w;
    const int per_tok = 2 * p.hkv;
    w.tok = (int)(r / per_tok);
    const int rest = (int)(r - (int64_t)w.tok * per_tok);
    w.kv = rest >= p.hkv;
    w.head = rest - w.kv * p.hkv;
    const int b = q8_request(p, w.tok);
    const int pos = p.start[b] + w.tok - p.tok0[b];
    const int log2P = 31 - __clz(p.page_size);
    const int page = __ldg(p.block_table + (int64_t)b * p.max_pages + (pos >> log2P));
    const int slot = pos & (p.page_size - 1);
    if (page < 0 || page >= p.num_pages) {
        if (flag)
            atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
        return w;
    }
    w.ok = true;
    const int64_t unit = (int64_t)page * p.hkv + w.head;
    w.row = (unit << log2P) + slot;
    w.scale = ((unit * 2 + w.kv) << log2P) + slot;
    return w;
}

}  // namespace

// D/8 lanes hold a row, 8 bf16 values each (one 16-byte load).  The row's
// largest magnitude is an integer maximum of the bf16 bits (their order is
// the values', infinities and NaN above all finite ones).
template <int D>
__global__ void __launch_bounds__(kCacheThreads) shkv_q8_append_kernel(const __grid_constant__ Q8CacheParams p)
{
    pdl_wait_prior();
    pdl_launch_dependents();
    constexpr int LR = D / 8;
    const int lane = threadIdx.x & (LR - 1);
    const int64_t rows = (int64_t)p.tok0[p.batch] * 2 * p.hkv;
    const int64_t stride = (int64_t)gridDim.x * (kCacheThreads / LR);
    // a warp's lanes run the loop together (the row maximum is a shuffle)
    const int64_t first = (int64_t)blockIdx.x * (kCacheThreads / LR) + threadIdx.x / LR;
    const int64_t warp_first = first - ((threadIdx.x & 31) / LR);
    for (int64_t wr = warp_first; wr < rows; wr += stride) {
        const int64_t r = wr + (first - warp_first);
        const Q8Row w = q8_row(p, r, r < rows, lane == 0);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (w.ok) {
            const __nv_bfloat16 *src = (w.kv ? p.v + w.tok * p.v_stride : p.k + w.tok * p.k_stride) + w.head * D;
            x = __ldg(reinterpret_cast<const uint4 *>(src) + lane);
        }
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a = __vmaxu2(a, xs[i] & 0x7fff7fffu);
        a = max(a & 0xffffu, a >> 16);
#pragma unroll
        for (int o = LR / 2; o > 0; o >>= 1)
            a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        // 448 = 1.75 * 2^8: one binade more where the significand is above 1.75
        int byte = (int)(a >> 7) - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0);
        byte = byte < 0 ? 0 : byte;
        const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);   // 2^-e
        uint32_t q[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = make_float2(__uint_as_float(xs[i] << 16) * inv,
                                         __uint_as_float(xs[i] & 0xffff0000u) * inv);
            const uint32_t c = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
            q[i >> 1] = (i & 1) ? q[i >> 1] | (c << 16) : c;
        }
        if (a >= 0x7f80u) {
            byte = 255;
            q[0] = q[1] = 0x7f7f7f7fu;
        }
        if (w.ok) {
            reinterpret_cast<uint2 *>((w.kv ? p.v_pages : p.k_pages) + w.row * D)[lane] = make_uint2(q[0], q[1]);
            if (lane == 0)
                p.scales[w.scale] = (uint8_t)byte;
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
// the row of a page outside the pool is zero.
template <int D>
__global__ void __launch_bounds__(kCacheThreads) shkv_q8_read_kernel(const __grid_constant__ Q8CacheParams p)
{
    pdl_wait_prior();
    pdl_launch_dependents();
    constexpr int LR = D / 8;
    const int lane = threadIdx.x & (LR - 1);
    const int64_t rows = (int64_t)p.tok0[p.batch] * 2 * p.hkv;
    for (int64_t r = (int64_t)blockIdx.x * (kCacheThreads / LR) + threadIdx.x / LR; r < rows;
         r += (int64_t)gridDim.x * (kCacheThreads / LR)) {
        const Q8Row w = q8_row(p, r, true, lane == 0);
        uint2 c = make_uint2(0u, 0u);
        float f = 0.f;
        if (w.ok) {
            c = __ldg(reinterpret_cast<const uint2 *>((w.kv ? p.v_pages : p.k_pages) + w.row * D) + lane);
            f = q8_scale(__ldg(p.scales + w.scale));
        }
        const uint32_t cs[2] = {c.x, c.y};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(cs[i >> 1] >> (16 * (i & 1))),
                                                             __NV_E4M3);
            const float2 x = __half22float2(__half2(h));
            o[i] = pack_bf16x2(x.x * f, x.y * f);
        }
        __nv_bfloat16 *dst = (w.kv ? p.v + w.tok * p.v_stride : p.k + w.tok * p.k_stride) + w.head * D;
        reinterpret_cast<uint4 *>(dst)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.batch; b += kCacheThreads)
            if (p.seq_lens[b] != p.old_len[b])
                atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
}

cudaError_t launch_q8_cache(const Q8CacheParams &p, bool read, int num_sms, cudaStream_t stream)
{
    const int64_t threads = (int64_t)p.tok0[p.batch] * 2 * p.hkv * (p.head_dim / 8);
    int64_t blocks = (threads + kCacheThreads - 1) / kCacheThreads;
    if (blocks > (int64_t)num_sms * 8)
        blocks = (int64_t)num_sms * 8;
    if (blocks < 1)
        blocks = 1;
    auto kern = read ? (p.head_dim == 64 ? shkv_q8_read_kernel<64> : shkv_q8_read_kernel<128>)
                     : (p.head_dim == 64 ? shkv_q8_append_kernel<64> : shkv_q8_append_kernel<128>);
    return launch_pdl(kern, (int)blocks, kCacheThreads, 0u, stream, p);
}

}  // namespace shkv
