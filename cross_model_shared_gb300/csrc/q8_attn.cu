// q8_attn.cu -- attention over the 8-bit KV cache: eight query rows of one
// (request, KV head) a CTA, fp32 arithmetic, one pass over the keys with a
// running maximum and sum.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "launch.cuh"
#include "q8.cuh"
#include "shkv_device.cuh"

namespace shkv {

namespace {

constexpr int kRows = 8;
constexpr int kKeys = 32;            // keys a step
constexpr int kThreads = 128;

template <int D>
__device__ __forceinline__ void stage(const Q8AttnParams &p, const uint8_t *pages, int kv, int b, int g, int key0,
                                      int last, float (*dst)[D + 1])
{
    const int log2P = 31 - __clz(p.page_size);
    for (int e = threadIdx.x; e < kKeys * (D / 4); e += kThreads) {
        const int t = e / (D / 4), c = e % (D / 4);
        const int key = key0 + t;
        uint32_t code = 0;
        float f = 0.f;
        if (key < last) {
            const int page = __ldg(p.block_table + (int64_t)b * p.max_pages + (key >> log2P));
            if (page >= 0 && page < p.num_pages) {
                const int64_t unit = (int64_t)page * p.hkv + g;
                const int slot = key & (p.page_size - 1);
                code = __ldg(reinterpret_cast<const uint32_t *>(pages + ((unit << log2P) + slot) * D) + c);
                f = q8_scale(__ldg(p.scales + ((unit * 2 + kv) << log2P) + slot));
            } else if (c == 0) {
                atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 x = __half22float2(
                __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(code >> (16 * i)), __NV_E4M3)));
            dst[t][4 * c + 2 * i] = x.x * f;
            dst[t][4 * c + 2 * i + 1] = x.y * f;
        }
    }
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads) shkv_q8_attn_kernel(const __grid_constant__ Q8AttnParams p)
{
    __shared__ float sq[kRows][D], skv[kKeys][D + 1], sp[kRows][kKeys], sm[kRows], sl[kRows], sa[kRows];
    pdl_wait_prior();
    pdl_launch_dependents();
    const int b = blockIdx.z, g = blockIdx.y;
    const int rows = p.n_q[b] * p.group;
    const int r0 = blockIdx.x * kRows;
    if (r0 >= rows)
        return;
    const int L = p.lens[b];
    if (threadIdx.x == 0 && p.seq_lens[b] != L)
        atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
    const int log2P = 31 - __clz(p.page_size);
    auto row_of = [&](int r) -> int64_t { return (int64_t)(p.q0[b] + r / p.group); };
    auto head_of = [&](int r) -> int { return g * p.group + r % p.group; };
    auto limit_of = [&](int r) -> int { return p.causal ? L - p.n_q[b] + r / p.group + 1 : L; };
    for (int e = threadIdx.x; e < kRows * D; e += kThreads) {
        const int r = e / D, d = e % D;
        sq[r][d] = r0 + r < rows ? __bfloat162float(p.q[row_of(r0 + r) * p.q_stride + head_of(r0 + r) * D + d]) : 0.f;
    }
    if (threadIdx.x < kRows) {
        sm[threadIdx.x] = -INFINITY;
        sl[threadIdx.x] = 0.f;
    }
    float acc[kRows * D / kThreads] = {};
    const int last = limit_of(min(r0 + kRows, rows) - 1);
    for (int key0 = 0; key0 < last; key0 += kKeys) {
        __syncthreads();
        stage<D>(p, p.k_pages, 0, b, g, key0, last, skv);
        __syncthreads();
        for (int e = threadIdx.x; e < kRows * kKeys; e += kThreads) {
            const int r = e / kKeys, t = e % kKeys, key = key0 + t;
            float s = 0.f;
            for (int d = 0; d < D; ++d)
                s += sq[r][d] * skv[t][d];
            bool seen = r0 + r < rows && key < limit_of(r0 + r);
            if (seen) {
                const int page = __ldg(p.block_table + (int64_t)b * p.max_pages + (key >> log2P));
                seen = page >= 0 && page < p.num_pages;
            }
            sp[r][t] = seen ? s * p.scale_log2 : -INFINITY;
        }
        __syncthreads();
        if (threadIdx.x < kRows) {
            const int r = threadIdx.x;
            float m = sm[r];
            for (int t = 0; t < kKeys; ++t)
                m = fmaxf(m, sp[r][t]);
            const float mu = m == -INFINITY ? 0.f : m;
            const float alpha = exp2f(sm[r] - mu);
            float l = 0.f;
            for (int t = 0; t < kKeys; ++t) {
                const float x = exp2f(sp[r][t] - mu);
                sp[r][t] = x;
                l += x;
            }
            sl[r] = sl[r] * alpha + l;
            sm[r] = m;
            sa[r] = alpha;
        }
        stage<D>(p, p.v_pages, 1, b, g, key0, last, skv);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRows * D / kThreads; ++i) {
            const int e = threadIdx.x + i * kThreads, r = e / D, d = e % D;
            float a = acc[i] * sa[r];
            for (int t = 0; t < kKeys; ++t)
                a += sp[r][t] != 0.f ? sp[r][t] * skv[t][d] : 0.f;    // a hidden key's NaN has no effect
            acc[i] = a;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows * D / kThreads; ++i) {
        const int e = threadIdx.x + i * kThreads, r = e / D, d = e % D;
        if (r0 + r < rows)
            p.out[(row_of(r0 + r) * p.hq + head_of(r0 + r)) * D + d] =
                __float2bfloat16_rn(sl[r] != 0.f ? acc[i] / sl[r] : 0.f);
    }
    if (threadIdx.x < kRows && r0 + threadIdx.x < rows && p.lse_out)
        p.lse_out[row_of(r0 + threadIdx.x) * p.hq + head_of(r0 + threadIdx.x)] =
            sl[threadIdx.x] != 0.f ? (sm[threadIdx.x] + log2f(sl[threadIdx.x])) * 0.6931471805599453f : -INFINITY;
}

cudaError_t launch_q8_attn(const Q8AttnParams &p, int max_rows, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((max_rows + kRows - 1) / kRows), (unsigned)p.hkv, (unsigned)p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.head_dim == 64 ? shkv_q8_attn_kernel<64> : shkv_q8_attn_kernel<128>, p);
}

}  // namespace shkv
