// evict.cu -- which tokens of a request stay, and their move into new pages
// (sm_103a).
#include <cuda_runtime.h>
#include <stdint.h>

#include "evict.cuh"
#include "launch.cuh"
#include "shkv_device.cuh"

namespace shkv {

namespace {

constexpr int kSelectThreads = 512;
constexpr int kBins = 2048;                              // of an 11-bit digit
constexpr int kBinsPerThread = kBins / kSelectThreads;
constexpr int kHistBytes = 2 * kBins * 4;
constexpr int kSelectKeys = 49152;                       // keys of a CTA's slice that it holds in shared memory

// A mass as an unsigned key of the same order: -0 as 0, every NaN on top.
__device__ __forceinline__ uint32_t mass_key(float m)
{
    if (m != m)
        return 0xffffffffu;
    const uint32_t u = __float_as_uint(m == 0.f ? 0.f : m);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Barrier of the row's CTAs; their shared memory is ordered by it.
__device__ __forceinline__ void row_sync(uint32_t ctas)
{
    if (ctas == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t of_rank(const void *p, uint32_t rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

__device__ __forceinline__ uint4 load_of_rank4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint2 load_of_rank2(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

}  // namespace

// A cluster of CTAs per (request, KV head), each with a slice of its positions.
// The n-th largest key of the candidates (the tokens between the sinks and the
// recent ones) is found digit by digit, 11 bits, 11 and 10 from the top: the CTAs
// count the candidates that share the digits found so far in a histogram each,
// read all of them and find the digit, every one for itself.  Then all keys
// above and, by position, as many of the equal ones as still fit are written.
// A slice's keys stay in shared memory between the passes.
__global__ void __launch_bounds__(kSelectThreads) shkv_select_kernel(const __grid_constant__ SelectParams p, int cached)
{
    extern __shared__ __align__(16) uint32_t dyn[];
    __shared__ uint32_t warp_sum[kSelectThreads / 32], found[3][2];      // found: digit and rest of each pass
    __shared__ __align__(8) uint32_t totals[2];
    __shared__ uint2 warp_counts[kSelectThreads / 32];
    uint32_t *const keys = dyn + 2 * kBins;
    uint32_t rank, ctas;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
    pdl_wait_prior();
    pdl_launch_dependents();
    const int row = blockIdx.x / ctas, b = row / p.hkv, g = row % p.hkv;
    const int L = p.lens[b], keep = min(p.keep[b], L);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const int all = rank * kSelectThreads + tid, step = ctas * kSelectThreads;
    int32_t *out = p.index + (int64_t)row * p.index_stride;
    if (g == 0 && all == 0 && p.seq_lens[b] != L)
        atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
    for (int64_t j = keep + all; j < p.index_stride; j += step)
        out[j] = -1;
    if (keep == L) {
        for (int j = all; j < L; j += step)
            out[j] = j;
        return;
    }
    // this CTA's positions, and the candidates among them
    const int per = (L + ctas - 1) / ctas, t0 = min(L, (int)rank * per), t1 = min(L, t0 + per);
    const int lo = max(t0, p.sink), hi = min(t1, L - p.recent);
    const float *m = p.mass + b * p.mass_request + g * p.mass_head;
    const uint32_t zero_key = mass_key(0.f);
    uint32_t prefix = 0u, need = (uint32_t)(keep - p.sink - p.recent);   // of the keys with this prefix
    const bool any = need > 0u;
    if (tid < 6)
        found[tid / 2][tid % 2] = 0u;
    if (any)
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            uint32_t *hist = dyn + (pass & 1) * kBins;
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            reinterpret_cast<uint4 *>(hist)[tid] = make_uint4(0u, 0u, 0u, 0u);
            __syncthreads();
            if (pass == 0) {
                // masses that are exactly 0 are many: counted in a register
                uint32_t zeros = 0u;
                constexpr int kU = 8;
                for (int t = lo + tid; t < hi; t += kU * kSelectThreads) {
                    float x[kU];
#pragma unroll
                    for (int u = 0; u < kU; ++u)
                        x[u] = t + u * kSelectThreads < hi ? __ldg(m + t + u * kSelectThreads) : 0.f;
#pragma unroll
                    for (int u = 0; u < kU; ++u)
                        if (t + u * kSelectThreads < hi) {
                            const uint32_t k = mass_key(x[u]);
                            if (cached)
                                keys[t + u * kSelectThreads - t0] = k;
                            if (k == zero_key)
                                ++zeros;
                            else
                                atomicAdd(hist + (k >> 21), 1u);
                        }
                }
                zeros = __reduce_add_sync(0xffffffffu, zeros);
                if (lane == 0 && zeros)
                    atomicAdd(hist + (zero_key >> 21), zeros);
            } else {
                const int above = shift + bits;
                uint32_t zeros = 0u;
                for (int t = lo + tid; t < hi; t += kSelectThreads) {
                    const uint32_t k = cached ? keys[t - t0] : mass_key(__ldg(m + t));
                    if ((k ^ prefix) >> above == 0u) {
                        if (k == zero_key)
                            ++zeros;
                        else
                            atomicAdd(hist + (k >> shift & ((1u << bits) - 1u)), 1u);
                    }
                }
                zeros = __reduce_add_sync(0xffffffffu, zeros);
                if (lane == 0 && zeros)
                    atomicAdd(hist + (zero_key >> shift & ((1u << bits) - 1u)), zeros);
            }
            row_sync(ctas);
            // thread i: the four bins from the top, over all CTAs
            const int bin = kBins - kBinsPerThread * (tid + 1);
            uint4 n = make_uint4(0u, 0u, 0u, 0u);
            for (uint32_t r = 0; r < ctas; ++r) {
                const uint4 v = ctas == 1 ? *reinterpret_cast<const uint4 *>(hist + bin) : load_of_rank4(of_rank(hist + bin, r));
                n.x += v.x, n.y += v.y, n.z += v.z, n.w += v.w;
            }
            const uint32_t mine = n.x + n.y + n.z + n.w;
            uint32_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                upto += lane >= o ? v : 0u;
            }
            if (lane == 31)
                warp_sum[warp] = upto;
            __syncthreads();
            for (int w = 0; w < warp; ++w)
                upto += warp_sum[w];
            uint32_t before = upto - mine;               // keys in higher bins
            if (before < need && need <= upto) {
                const uint32_t c[4] = {n.w, n.z, n.y, n.x};
                int d = bin + 3;
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (before + c[i] < need && d == bin + 3 - i) {
                        before += c[i];
                        --d;
                    }
                found[pass][0] = (uint32_t)d;
                found[pass][1] = need - before;
            }
            __syncthreads();
            prefix |= found[pass][0] << shift;
            need = found[pass][1];
        }
    // `need` of the keys equal to `prefix` stay, all larger ones do.  A warp takes
    // a run of the slice; first how many of each lie before it.
    const int run = ((t1 - t0 + kSelectThreads - 1) / kSelectThreads) * 32;
    const int w0 = min(t1, t0 + warp * run), w1 = min(t1, w0 + run);
    auto look = [&](int t, bool &above, bool &equal) {
        above = t < lo || t >= hi;                       // the slice's sinks and recent tokens
        equal = false;
        if (!above && any) {
            const uint32_t k = cached ? keys[t - t0] : mass_key(__ldg(m + t));
            above = k > prefix;
            equal = k == prefix;
        }
    };
    uint32_t na = 0u, ne = 0u;
    for (int t = w0 + lane; t < w1; t += 32) {
        bool above, equal;
        look(t, above, equal);
        na += above;
        ne += equal;
    }
    na = __reduce_add_sync(0xffffffffu, na);
    ne = __reduce_add_sync(0xffffffffu, ne);
    if (lane == 0)
        warp_counts[warp] = make_uint2(na, ne);
    __syncthreads();
    uint32_t a = 0u, e = 0u;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
        if (w == warp)
            na = a, ne = e;
        a += warp_counts[w].x;
        e += warp_counts[w].y;
    }
    if (ctas > 1) {
        if (tid == 0)
            totals[0] = a, totals[1] = e;
        row_sync(ctas);
        for (uint32_t r = 0; r < rank; ++r) {
            const uint2 v = load_of_rank2(of_rank(totals, r));
            na += v.x, ne += v.y;
        }
    }
    for (int t = w0 + lane; t - lane < w1; t += 32) {
        bool above = false, equal = false;
        if (t < w1)
            look(t, above, equal);
        const uint32_t ba = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, equal);
        const uint32_t left = (1u << lane) - 1u, ea = ne + __popc(be & left);
        const uint32_t at = na + __popc(ba & left) + min(ea, need);
        if ((above || (equal && ea < need)) && at < (uint32_t)keep)      // always, unless masses change under the call
            out[at] = t;
        na += __popc(ba);
        ne += __popc(be);
    }
    if (ctas > 1)
        row_sync(ctas);                                  // nobody leaves while its counts are read
}

// A row gets more CTAs (a cluster of up to 8) as long as all of them find room
// at once and a slice keeps 4096 tokens.
cudaError_t launch_select(const SelectParams &p, int num_sms, cudaStream_t stream)
{
    int64_t longest = 0;
    for (int b = 0; b < p.batch; ++b)
        if (p.keep[b] < p.lens[b])
            longest = p.lens[b] > longest ? p.lens[b] : longest;
    const int64_t rows = (int64_t)p.batch * p.hkv;
    int ctas = 1;
    while (ctas < 8 && 2 * ctas * rows <= 2 * num_sms && longest > 4096 * ctas)
        ctas *= 2;
    const int64_t slice = (longest + ctas - 1) / ctas;
    const int cached = slice <= kSelectKeys;
    const uint32_t smem = (uint32_t)(kHistBytes + (cached ? slice * 4 : 0));
    cudaError_t e = cudaFuncSetAttribute(shkv_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kHistBytes + kSelectKeys * 4);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * ctas));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, shkv_select_kernel, p, cached);
}

namespace {

constexpr int kMoveThreads = 256;
constexpr int kMassPer = 16;         // masses of a thread and pass
constexpr int kMassZeros = 8;

// Masses of one (request, KV head), a CTA: a pass reads its masses before any is
// written, and as positions ascend it writes only below what later passes read.
__device__ __forceinline__ void move_masses(const EvictParams &p, int row)
{
    const int b = row / p.hkv, g = row % p.hkv;
    const int L = p.lens[b], keep = p.keep[b];
    if (keep >= L)
        return;
    const int32_t *index = p.index + (int64_t)row * p.index_stride;
    const float *src = p.mass.in + b * p.mass.in_request + g * p.mass.in_head;
    float *dst = p.mass.out + b * p.mass.out_request + g * p.mass.out_head;
    for (int j0 = 0; j0 < keep; j0 += kMassPer * kMoveThreads) {
        int i[kMassPer];
        float x[kMassPer];
#pragma unroll
        for (int u = 0; u < kMassPer; ++u) {
            const int j = j0 + u * kMoveThreads + threadIdx.x;
            i[u] = j < keep ? __ldg(index + j) : -1;
        }
#pragma unroll
        for (int u = 0; u < kMassPer; ++u)
            x[u] = (uint32_t)i[u] < (uint32_t)L ? src[i[u]] : 0.f;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kMassPer; ++u) {
            const int j = j0 + u * kMoveThreads + threadIdx.x;
            if (j < keep)
                dst[j] = x[u];
        }
    }
    __syncthreads();
    for (int j0 = keep + threadIdx.x; j0 < L; j0 += kMassZeros * kMoveThreads)
#pragma unroll
        for (int u = 0; u < kMassZeros; ++u)
            if (j0 + u * kMoveThreads < L)
                dst[j0 + u * kMoveThreads] = 0.f;
}

}  // namespace

// The first CTAs move masses.  The others copy rows, a warp per (new page, KV
// head): K's and V's rows of 32 / (2 D / 8) tokens an instruction, eight
// instructions' loads before their stores.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) shkv_evict_kernel(const __grid_constant__ EvictParams p)
{
    constexpr int V = D / 8, kTok = 32 / (2 * V);        // vectors of a row, tokens an instruction
    constexpr int kU = 8;
    pdl_wait_prior();
    pdl_launch_dependents();
    const int mass_blocks = p.mass.out ? p.batch * p.hkv : 0;
    if ((int)blockIdx.x < mass_blocks) {
        move_masses(p, blockIdx.x);
        return;
    }
    const int lane = threadIdx.x & 31, P = p.page_size;
    const int w = (blockIdx.x - mass_blocks) * (kMoveThreads / 32) + threadIdx.x / 32;
    if (w >= p.page0[p.batch] * p.hkv)
        return;
    const int page = w / p.hkv, g = w % p.hkv;
    int b = 0, hi = p.batch;
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (p.page0[mid] <= page)
            b = mid;
        else
            hi = mid;
    }
    const int j0 = (page - p.page0[b]) * P, n = min(P, p.keep[b] - j0);
    const int to = __ldg(p.new_table + b * p.new_stride + j0 / P);
    bool ok = (uint32_t)to < (uint32_t)p.num_pages;
    int row = 0;                                         // of the lane's token (a pool's rows fit 32 bits)
    if (!ok) {
        atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
    } else if (lane < n) {
        const int i = __ldg(p.index + ((int64_t)b * p.hkv + g) * p.index_stride + j0 + lane);
        ok = (uint32_t)i < (uint32_t)p.lens[b];
        if (!ok) {
            atomicOr(p.err, SHKV_ERRF_INDEX);
        } else {
            const int from = __ldg(p.table + b * p.table_stride + i / P);
            ok = (uint32_t)from < (uint32_t)p.num_pages;
            if (!ok)
                atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
            row = (from * p.hkv + g) * P + i % P;
        }
    }
    const uint32_t good = __ballot_sync(0xffffffffu, ok && lane < n);
    const int tok = lane / (2 * V), v = lane % V;
    uint4 *pages = lane / V % 2 ? p.v_pages : p.k_pages;
    uint4 *dst = pages + ((int64_t)to * p.hkv + g) * P * V + v;
    for (int j = 0; j < n; j += kU * kTok) {
        uint4 x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int t = j + u * kTok + tok;
            const int64_t src = __shfl_sync(0xffffffffu, row, t & 31);
            if (t < n && good >> t & 1u)
                x[u] = __ldcs(pages + src * V + v);      // pages that are given up
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int t = j + u * kTok + tok;
            if (t < n && good >> t & 1u)
                dst[(int64_t)t * V] = x[u];
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
    auto kern = p.head_dim == 64 ? shkv_evict_kernel<64> : shkv_evict_kernel<128>;
    cudaError_t e = grid ? launch_pdl(kern, (int)grid, kMoveThreads, 0u, stream, p) : cudaSuccess;
    if (e == cudaSuccess)
        e = launch_pdl(shkv_evict_commit_kernel, p.batch, kMoveThreads, 0u, stream, p);
    return e;
}

}  // namespace shkv
