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

constexpr int kVecs = 4;             // rows of a token that a lane has in flight

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

// The token's table entry (0 behind the warp's last token), and its check.
__device__ __forceinline__ int q8_entry(const Q8CacheParams &p, const Q8Walk &w, int log2P)
{
    return w.t < w.end ? __ldg(p.block_table + (int64_t)w.b * p.max_pages + (w.pos >> log2P)) : 0;
}

__device__ __forceinline__ bool q8_inside(const Q8CacheParams &p, int page)
{
    if ((uint32_t)page < (uint32_t)p.num_pages)
        return true;
    if ((threadIdx.x & 31) == 0)
        atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
    return false;
}

}  // namespace

// A warp per token, D/16 lanes a row: lane l holds values 8l .. 8l+7 and those
// D/2 further on.  The row's largest magnitude is an integer maximum of the
// bf16 bits (their order is the values', infinities and NaN above all finite
// ones).  Bound by bytes and, closely behind, by instructions: two vectors a
// lane halve the shuffles, scales and addresses a value (45k tokens of 8 heads
// of 128: 44 us with one vector a lane).
template <int D>
__global__ void __launch_bounds__(kCacheThreads) shkv_q8_append_kernel(const __grid_constant__ Q8CacheParams p)
{
    pdl_wait_prior();
    pdl_launch_dependents();
    constexpr int LR = D / 16, RW = 32 / LR;             // lanes a row, rows a warp's pass
    const int lane = threadIdx.x & (LR - 1), sub = (threadIdx.x & 31) / LR;
    const int log2P = 31 - __clz(p.page_size);
    const int rows = 2 * p.hkv;
    Q8Walk w = q8_walk(p);
    int page = q8_entry(p, w, log2P);
    while (w.t < w.end) {
        Q8Walk next = w;                                 // the next token's page is read ahead
        q8_next(p, next);
        const int next_page = q8_entry(p, next, log2P);
        const uint4 *ks = reinterpret_cast<const uint4 *>(p.k + w.t * p.k_stride) + lane;
        const uint4 *vs = reinterpret_cast<const uint4 *>(p.v + w.t * p.v_stride) + lane;
        const int64_t unit0 = (int64_t)page * p.hkv;
        const int slot = w.pos & (p.page_size - 1);
        bool inside = false;
        for (int r0 = sub; r0 < rows + sub; r0 += kVecs * RW) {
            uint4 x[kVecs][2];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int r = r0 + i * RW;
                x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) {
                    const uint4 *src = r < p.hkv ? ks + r * (D / 8) : vs + (r - p.hkv) * (D / 8);
                    x[i][0] = __ldg(src);
                    x[i][1] = __ldg(src + LR);
                }
            }
            if (r0 == sub)
                inside = q8_inside(p, page);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int r = r0 + i * RW;
                const uint32_t xs[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                                        x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
                uint32_t a = xs[0] & 0x7fff7fffu;
#pragma unroll
                for (int v = 1; v < 8; ++v)
                    a = __vmaxu2(a, xs[v] & 0x7fff7fffu);
#pragma unroll
                for (int o = LR / 2; o > 0; o >>= 1)
                    a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, o));
                a = max(a & 0xffffu, a >> 16);
                // 448 = 1.75 * 2^8: one binade more where the significand is above 1.75
                int byte = max((int)((a + 0x1fu) >> 7) - 8, 0);
                const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);   // 2^-e
                uint32_t c[8];
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    const float2 f = __fmul2_rn(make_float2(__uint_as_float(xs[v] << 16),
                                                            __uint_as_float(xs[v] & 0xffff0000u)),
                                                make_float2(inv, inv));
                    c[v] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
                }
                uint2 q0 = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                uint2 q1 = make_uint2(c[4] | c[5] << 16, c[6] | c[7] << 16);
                if (a >= 0x7f80u) {
                    byte = 255;
                    q0.x = q0.y = q1.x = q1.y = 0x7f7f7f7fu;
                }
                if (r < rows && inside) {
                    const int kv = r >= p.hkv;
                    const int64_t unit = unit0 + r - kv * p.hkv;
                    uint2 *dst = reinterpret_cast<uint2 *>((kv ? p.v_pages : p.k_pages) + ((unit << log2P) + slot) * D) + lane;
                    dst[0] = q0;
                    dst[LR] = q1;
                    if (lane == 0)
                        p.scales[((unit * 2 + kv) << log2P) + slot] = (uint8_t)byte;
                }
            }
        }
        w = next;
        page = next_page;
    }
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.batch; b += kCacheThreads) {
            if (p.seq_lens[b] != p.old_len[b])
                atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
            p.seq_lens[b] = p.start[b] + p.tok0[b + 1] - p.tok0[b];
        }
}

// Two e4m3 codes of w (the low or the high half) as bf16 pairs times the
// scale: the sign and the seven bits in bf16's places stand for the code's
// value times 2^-120, subnormals too; both products are exact down to bf16's
// own subnormals.
template <bool kHigh>
__device__ __forceinline__ uint32_t q8_bf16x2(uint32_t w, __nv_bfloat162 scale)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(kHigh ? 0xB3A2 : 0x9180));
    r = (r << 4) & 0x87F087F0u;
    const __nv_bfloat162 up = __halves2bfloat162(__ushort_as_bfloat16(0x7B80), __ushort_as_bfloat16(0x7B80));   // 2^120
    const __nv_bfloat162 v = __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&r), up), scale);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The rows of the ranges as bf16, exact (q * 2^e has a 4-bit significand);
// the rows of a page outside the pool are zero.  Lanes as in append.
template <int D>
__global__ void __launch_bounds__(kCacheThreads) shkv_q8_read_kernel(const __grid_constant__ Q8CacheParams p)
{
    pdl_wait_prior();
    pdl_launch_dependents();
    constexpr int LR = D / 16, RW = 32 / LR;
    const int lane = threadIdx.x & (LR - 1), sub = (threadIdx.x & 31) / LR;
    const int log2P = 31 - __clz(p.page_size);
    const int rows = 2 * p.hkv;
    Q8Walk w = q8_walk(p);
    int page = q8_entry(p, w, log2P);
    while (w.t < w.end) {
        Q8Walk next = w;                                 // the next token's page is read ahead
        q8_next(p, next);
        const int next_page = q8_entry(p, next, log2P);
        const bool inside = q8_inside(p, page);
        uint4 *kd = reinterpret_cast<uint4 *>(p.k + w.t * p.k_stride) + lane;
        uint4 *vd = reinterpret_cast<uint4 *>(p.v + w.t * p.v_stride) + lane;
        const int64_t unit0 = (int64_t)page * p.hkv;
        const int slot = w.pos & (p.page_size - 1);
        for (int r0 = sub; r0 < rows; r0 += kVecs * RW) {
            uint2 c[kVecs][2];
            uint32_t s[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int r = r0 + i * RW;
                c[i][0] = c[i][1] = make_uint2(0u, 0u);
                s[i] = 0u;
                if (r < rows && inside) {
                    const int kv = r >= p.hkv;
                    const int64_t unit = unit0 + r - kv * p.hkv;
                    const uint2 *src = reinterpret_cast<const uint2 *>((kv ? p.v_pages : p.k_pages) +
                                                                       ((unit << log2P) + slot) * D) + lane;
                    c[i][0] = __ldg(src);
                    c[i][1] = __ldg(src + LR);
                    s[i] = __ldg(p.scales + ((unit * 2 + kv) << log2P) + slot);
                }
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int r = r0 + i * RW;
                // 2^(s - 127) as bf16, NaN for 255
                const unsigned short sb = (unsigned short)(s[i] << 7 | (s[i] == 0u || s[i] == 255u ? 1u << 6 : 0u));
                const __nv_bfloat162 f = __halves2bfloat162(__ushort_as_bfloat16(sb), __ushort_as_bfloat16(sb));
                if (r < rows) {
                    uint4 *dst = r < p.hkv ? kd + r * (D / 8) : vd + (r - p.hkv) * (D / 8);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        dst[h * LR] = make_uint4(q8_bf16x2<false>(c[i][h].x, f), q8_bf16x2<true>(c[i][h].x, f),
                                                 q8_bf16x2<false>(c[i][h].y, f), q8_bf16x2<true>(c[i][h].y, f));
                }
            }
        }
        w = next;
        page = next_page;
    }
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.batch; b += kCacheThreads)
            if (p.seq_lens[b] != p.old_len[b])
                atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
}

// Takes reported bits out of the error word: atomically, as kernels of other
// streams may be setting others.
__global__ void shkv_q8_clear_errors_kernel(uint32_t *err, uint32_t bits) { atomicAnd(err, ~bits); }

cudaError_t launch_q8_clear_errors(uint32_t *err, uint32_t bits, cudaStream_t stream)
{
    shkv_q8_clear_errors_kernel<<<1, 1, 0, stream>>>(err, bits);
    return cudaGetLastError();
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
