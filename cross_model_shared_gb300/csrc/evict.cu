// evict.cu -- which tokens of a request stay, and their move into new pages
// (sm_103a).
#include <cuda_runtime.h>
#include <stdint.h>

#include "evict.cuh"
#include "launch.cuh"
#include "shkv_device.cuh"

namespace shkv {

namespace {

constexpr int kBins = 2048, kCoarse = 256;               // of an 11-bit digit, and by its upper 8 bits
constexpr int kHist = kBins + kCoarse;                   // words of a histogram
// Words before the keys: two histograms, then 256 positions a warp.
constexpr int select_front(int threads) { return threads * 8 > 2 * kHist ? threads * 8 : 2 * kHist; }
constexpr int kSelectKeys = 49152;                       // keys of a CTA's slice that it holds in shared memory

// A mass as an unsigned key of the same order: -0 as 0, every NaN on top.  Sinks and
// recent tokens have a key above all, no token the key 0.
constexpr uint32_t kAlways = 0xffffffffu, kNanKey = 0xfffffffeu;

__device__ __forceinline__ uint32_t mass_key(float m)
{
    const uint32_t u = __float_as_uint(m + 0.f);         // -0 + 0 = 0
    return m != m ? kNanKey : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
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

__device__ __forceinline__ uint32_t load_of_rank(const uint32_t *p, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(of_rank(p, rank)));
    return v;
}

}  // namespace

// A cluster of CTAs per (request, KV head), each with a slice of its positions.
// The n-th largest key of the candidates (the tokens between the sinks and the
// recent ones) is found digit by digit, 11 bits, 11 and 10 from the top: the CTAs
// count the candidates that share the digits found so far in a histogram each,
// and every one of them finds the digit from all: first by its upper 8 bits, then
// among 8 bins (reading all 2048 bins of 8 CTAs took 2.5 us a digit).  Then all
// keys above and, by position, as many of the equal ones as still fit are written.
// A slice's keys stay in shared memory between the passes, four of a thread side by
// side.  Bound by the latency of its steps.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    shkv_select_kernel(const __grid_constant__ SelectParams p, int cached)
{
    constexpr int kWarps = kThreads / 32;
    extern __shared__ __align__(16) uint32_t dyn[];
    __shared__ uint32_t warp_sum[kWarps], found[2];            // found: coarse bin, keys in higher ones
    __shared__ uint32_t totals[2];
    __shared__ uint2 warp_counts[kWarps];
    uint32_t *const keys = dyn + select_front(kThreads);
    uint32_t rank, ctas;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
    pdl_wait_prior();
    pdl_launch_dependents();
    const int row = blockIdx.x / ctas, b = row / p.hkv, g = row % p.hkv;
    const int L = p.lens[b], keep = min(p.keep[b], L);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const int all = rank * kThreads + tid, step = ctas * kThreads;
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
    const int per = ((L + (int)ctas - 1) / (int)ctas + 3) & ~3, t0 = min(L, (int)rank * per), t1 = min(L, t0 + per);
    const int lo = max(t0, p.sink), hi = min(t1, L - p.recent);
    const float *m = p.mass + b * p.mass_request + g * p.mass_head;
    const uint32_t zero_key = mass_key(0.f);
    uint32_t prefix = 0u, need = (uint32_t)(keep - p.sink - p.recent);   // of the keys with this prefix
    // keys of positions t .. t + 3, t - t0 a multiple of 4; 0 outside the slice
    auto four = [&](int t) -> uint4 {
        if (cached)
            return *reinterpret_cast<const uint4 *>(keys + (t - t0));
        uint32_t k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            k[i] = t + i >= t1 ? 0u : t + i < lo || t + i >= hi ? kAlways : mass_key(__ldg(m + t + i));
        return make_uint4(k[0], k[1], k[2], k[3]);
    };
    for (int i = tid; i < 2 * kHist / 4; i += kThreads)
        reinterpret_cast<uint4 *>(dyn)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < 2)
        found[tid] = 0u;
    __syncthreads();
    if (need == 0u)
        prefix = kNanKey;                    // no candidate is above, none of the equal ones stays
#pragma unroll 1
    for (int pass = 0; pass < (need ? 3 : 1); ++pass) {
        uint32_t *hist = dyn + (pass & 1) * kHist;
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        // masses that are exactly 0 are many: counted in a register
        uint32_t zeros = 0u;
        if (pass == 0) {
            constexpr int kU = 16;
#pragma unroll 1
            for (int t = t0 + tid; t < t1; t += kU * kThreads) {
                float x[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    x[u] = t + u * kThreads < t1 ? __ldg(m + t + u * kThreads) : 0.f;
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int at = t + u * kThreads;
                    if (at >= t1)
                        break;
                    uint32_t k = mass_key(x[u]);
                    if (at < lo || at >= hi)
                        k = kAlways;
                    else if (k == zero_key)
                        ++zeros;
                    else
                        atomicAdd(hist + (k >> 21), 1u);
                    if (cached)
                        keys[at - t0] = k;
                }
            }
            if (tid < 3 && cached && t1 + tid - t0 < ((t1 - t0 + 3) & ~3))
                keys[t1 + tid - t0] = 0u;
        } else {
            // keys base .. base + width share the digits found (the topmost is kAlways)
            const uint32_t width = min((1u << (pass == 1 ? 21 : 10)) - 1u, kNanKey - prefix);
#pragma unroll 2
            for (int t = t0 + 4 * tid; t < t1; t += 4 * kThreads) {
                const uint4 v = four(t);
                const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                {
                    const bool in = k[i] - prefix <= width, zero = k[i] == zero_key;
                    zeros += in && zero;
                    if (in && !zero)
                        atomicAdd(hist + (k[i] >> shift & mask), 1u);
                }
            }
        }
        zeros = __reduce_add_sync(0xffffffffu, zeros);
        if (lane == 0 && zeros)
            atomicAdd(hist + (zero_key >> shift & mask), zeros);
        __syncthreads();
        if (need == 0u)
            break;                                   // the keys are there, that was all
        if (tid < kCoarse) {
            const uint4 v = reinterpret_cast<const uint4 *>(hist)[2 * tid], x = reinterpret_cast<const uint4 *>(hist)[2 * tid + 1];
            hist[kBins + tid] = (v.x + v.y + v.z + v.w) + (x.x + x.y + x.z + x.w);
        }
        row_sync(ctas);
        // thread i < 256: coarse bin 255 - i of all CTAs
        uint32_t n = 0u;
        if (tid < kCoarse) {
            const uint32_t *bin = hist + kBins + kCoarse - 1 - tid;
            if (ctas == 1)
                n = *bin;
            else
#pragma unroll 4
                for (uint32_t r = 0; r < ctas; ++r)
                    n += load_of_rank(bin, r);
        }
        uint32_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? v : 0u;
        }
        if (lane == 31)
            warp_sum[warp] = upto;
        __syncthreads();
        if (tid < kCoarse) {
#pragma unroll
            for (int w = 0; w < kCoarse / 32; ++w)
                upto += w < warp ? warp_sum[w] : 0u;
            if (upto - n < need && need <= upto) {
                found[0] = (uint32_t)(kCoarse - 1 - tid);
                found[1] = upto - n;              // keys in higher coarse bins
            }
        }
        __syncthreads();
        // every warp finds the digit among the 8 bins: lane = 4 ranks x 8 bins, from the top
        {
            const uint32_t coarse = found[0];
            const uint32_t *bin = hist + coarse * 8u + 7u - (lane & 7);
            uint32_t v = 0u;
            for (uint32_t r = lane >> 3; r < ctas; r += 4)
                v += ctas == 1 ? *bin : load_of_rank(bin, r);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            uint32_t sum = v;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o, 8);
                sum += (lane & 7) >= o ? x : 0u;
            }
            const uint32_t before = found[1] + sum - v;
            const uint32_t here = __ballot_sync(0xffffffffu, before < need && need <= before + v) & 255u;
            const int at = here ? __ffs(here) - 1 : 0;
            need -= __shfl_sync(0xffffffffu, before, at);
            prefix |= (coarse * 8u + 7u - (uint32_t)at) << shift;
        }
        if (pass == 1) {                             // the first histogram serves again: all have read it
            for (int i = tid; i < kHist / 4; i += kThreads)
                reinterpret_cast<uint4 *>(dyn)[i] = make_uint4(0u, 0u, 0u, 0u);
            __syncthreads();
        }
    }
    // `need` of the keys equal to `prefix` stay, all larger ones do.  A warp takes
    // a run of the slice, a lane eight positions at a time; first how many of each lie
    // before it.
    const int run = (((t1 - t0) + 256 * kWarps - 1) / (256 * kWarps)) * 256;
    const int w0 = min(t1, t0 + warp * run), w1 = min(t1, w0 + run);
    uint32_t na = 0u, ne = 0u;
#pragma unroll 2
    for (int t = w0 + 4 * lane; t < w1; t += 128) {
        const uint4 k = four(t);
        na += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
        ne += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
    }
    na = __reduce_add_sync(0xffffffffu, na);
    ne = __reduce_add_sync(0xffffffffu, ne);
    if (lane == 0)
        warp_counts[warp] = make_uint2(na, ne);
    __syncthreads();
    uint32_t a = 0u, e = 0u;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp)
            na = a, ne = e;
        a += warp_counts[w].x;
        e += warp_counts[w].y;
    }
    if (ctas > 1) {
        if (tid == 0)
            totals[0] = a, totals[1] = e;
        row_sync(ctas);
        if (lane < 2) {                                  // lane 0: above, lane 1: equal, of the CTAs before
            uint32_t v = 0u;
#pragma unroll 4
            for (uint32_t r = 0; r < rank; ++r)
                v += load_of_rank(totals + lane, r);
            a = v;
        }
        na += __shfl_sync(0xffffffffu, a, 0);
        ne += __shfl_sync(0xffffffffu, a, 1);
    }
    uint32_t *const stage = dyn + warp * 256;            // the histograms have been read
    for (int t = w0 + 8 * lane; t - 8 * lane < w1; t += 256) {
        const uint4 none = make_uint4(0u, 0u, 0u, 0u), v = t < w1 ? four(t) : none, x = t + 4 < w1 ? four(t + 4) : none;
        const uint32_t k[8] = {v.x, v.y, v.z, v.w, x.x, x.y, x.z, x.w};
        // above in the lower half, equal in the upper half of a word
        uint32_t mine = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            mine += k[i] > prefix ? 1u : k[i] == prefix ? 1u << 16 : 0u;
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? y : 0u;
        }
        const uint32_t sum = __shfl_sync(0xffffffffu, upto, 31);
        // side by side in shared memory first: written from here, a position at a time,
        // they take 6 us of a long row
        const uint32_t base = na + min(ne, need);
        uint32_t pa = na + (upto - mine & 0xffffu), pe = ne + (upto - mine >> 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool up = k[i] > prefix, eq = k[i] == prefix;
            if (up || (eq && pe < need))
                stage[pa + min(pe, need) - base] = t + i;
            pa += up;
            pe += eq;
        }
        na += sum & 0xffffu;
        ne += sum >> 16;
        const uint32_t n = na + min(ne, need) - base;
        __syncwarp();
        for (uint32_t j = lane; j < n; j += 32)
            if (base + j < (uint32_t)keep)               // always, unless masses change under the call
                out[base + j] = (int32_t)stage[j];
        __syncwarp();
    }
    if (ctas > 1)
        row_sync(ctas);                                  // nobody leaves while its counts are read
}

// A row gets more CTAs (a cluster of up to 8) as long as each has an SM to itself and
// a slice keeps 4096 tokens (32 rows of 131584: 2 CTAs 69 us, 4 26 us, 8, two on some
// SMs, 30 us), and where its keys fit no shared memory otherwise (192 rows of 131000:
// 256 us from global memory with a CTA a row).  Long rows and slices have 1024
// threads a CTA, short ones 256: 128 rows of 20K to 40K tokens 41 us with 256, 27 us
// with 1024; 512 rows of 1K to 8K 19 and 30; 1024 rows of 2K to 4K 23 and 53.
cudaError_t launch_select(const SelectParams &p, int num_sms, cudaStream_t stream)
{
    int64_t longest = 0;
    for (int b = 0; b < p.batch; ++b)
        if (p.keep[b] < p.lens[b])
            longest = p.lens[b] > longest ? p.lens[b] : longest;
    const int64_t rows = (int64_t)p.batch * p.hkv;
    int ctas = 1;
    while (ctas < 8 && longest > 4096 * ctas && (2 * ctas * rows <= num_sms || longest > (int64_t)kSelectKeys * ctas))
        ctas *= 2;
    const bool wide = ctas > 1 || longest > 12288;
    const int threads = wide ? 1024 : 256;
    auto kern = wide ? shkv_select_kernel<1024> : shkv_select_kernel<256>;
    const int64_t slice = ((longest + ctas - 1) / ctas + 3) & ~3;
    const int cached = slice <= kSelectKeys;
    const uint32_t front = (uint32_t)select_front(threads) * 4, smem = front + (uint32_t)(cached ? slice * 4 : 0);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)front + kSelectKeys * 4);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * ctas));
    cfg.blockDim = dim3((unsigned)threads);
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
    return cudaLaunchKernelEx(&cfg, kern, p, cached);
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
