// mass.cu -- the attention weight that every cached token of a KV head gets
// from the rows of a decode step or of a causal chunk, added to its mass
// (sm_103a).
#include <cuda_runtime.h>
#include <stdint.h>

#include "evict.cuh"
#include "launch.cuh"
#include "shkv_device.cuh"

namespace shkv {

namespace {
constexpr int kTile = 128;           // tokens of a CTA, one a thread
constexpr int kRows = 32;            // rows in shared memory at a time
}  // namespace

// A thread per token holds its row of K; the query rows pass through shared
// memory, 32 at a time.
template <int D>
__global__ void __launch_bounds__(kTile) shkv_mass_kernel(const __grid_constant__ MassParams p)
{
    __shared__ float qs[kRows][D];
    __shared__ float ls[kRows];
    pdl_wait_prior();
    pdl_launch_dependents();
    int lo = 0, hi = p.batch;
    const int tile = blockIdx.x / p.hkv, g = blockIdx.x % p.hkv;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.tile0[mid] <= tile)
            lo = mid;
        else
            hi = mid;
    }
    const int b = lo, L = p.lens[b], t0 = (tile - p.tile0[b]) * kTile, t = t0 + threadIdx.x;
    if (t0 == 0 && g == 0 && threadIdx.x == 0 && p.seq_lens[b] != L)
        atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
    uint32_t k[D / 2];
    bool inside = false;
    if (t < L) {
        const int page = p.block_table[(int64_t)b * p.max_pages + t / p.page_size];
        inside = (uint32_t)page < (uint32_t)p.num_pages;
        if (!inside)
            atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
        const uint4 *src = reinterpret_cast<const uint4 *>(p.k_pages) +
                           (((int64_t)(inside ? page : 0) * p.hkv + g) * p.page_size + t % p.page_size) * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const uint4 x = inside ? src[i] : make_uint4(0u, 0u, 0u, 0u);
            k[4 * i] = x.x, k[4 * i + 1] = x.y, k[4 * i + 2] = x.z, k[4 * i + 3] = x.w;
        }
    }
    const int rows = p.n_q * p.group, past = L - p.n_q;
    const int first = p.causal ? max(0, t0 - past) * p.group : 0;
    float sum = 0.f;
    for (int r0 = first; r0 < rows; r0 += kRows) {
        __syncthreads();
        const int n = min(kRows, rows - r0);
        for (int e = threadIdx.x; e < n * D; e += kTile) {
            const int r = r0 + e / D, i = r / p.group, h = g * p.group + r % p.group;
            qs[e / D][e % D] = __bfloat162float(p.q[b * p.q_request + i * p.q_token + h * D + e % D]);
        }
        if (threadIdx.x < n) {
            const int r = r0 + threadIdx.x;
            ls[threadIdx.x] = lse_base2(p.lse[b * p.lse_request + r / p.group * p.lse_token + g * p.group + r % p.group]);
        }
        __syncthreads();
        if (!inside)
            continue;
        for (int r = 0; r < n; ++r) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < D / 2; ++i) {
                s = fmaf(__uint_as_float(k[i] << 16), qs[r][2 * i], s);
                s = fmaf(__uint_as_float(k[i] & 0xffff0000u), qs[r][2 * i + 1], s);
            }
            if (!p.causal || t <= past + (r0 + r) / p.group)
                sum += ex2_approx(fmaf(s, p.scale_log2, -ls[r]));
        }
    }
    if (t < L) {
        const MassIo &m = p.mass;
        float old = 0.f;
        if (m.in)
            old = p.decay * m.in[b * m.in_request + g * m.in_head + t];
        m.out[b * m.out_request + g * m.out_head + t] = old + sum;
    }
}

cudaError_t launch_mass(const MassParams &p, cudaStream_t stream)
{
    const int grid = p.hkv * p.tile0[p.batch];
    return p.head_dim == 64 ? launch_pdl(shkv_mass_kernel<64>, grid, kTile, 0u, stream, p)
                            : launch_pdl(shkv_mass_kernel<128>, grid, kTile, 0u, stream, p);
}

}  // namespace shkv
