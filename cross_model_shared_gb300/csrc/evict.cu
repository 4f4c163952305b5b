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
constexpr int kSelectKeys = 49152;                       // keys of a CTA's slice that it holds in shared memory
constexpr int kSmemSm = 228 * 1024;                      // of an SM, 1 KB a CTA among it
constexpr int kGroup = 128;                              // keys that a warp reads at once, four of a lane

// A mass as an unsigned key of the same order: -0 as 0, every NaN (a sum's result is
// the one with all bits set) on top.
__device__ __forceinline__ uint32_t mass_key(float m)
{
    const uint32_t u = __float_as_uint(m + 0.f);         // -0 + 0 = 0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Barrier of the row's CTAs; their shared memory is ordered by it.  (The cluster's
// is a whole warp's instruction; lanes come from loops of different length.)
__device__ __forceinline__ void row_sync(uint32_t ctas)
{
    if (ctas == 1) {
        __syncthreads();
        return;
    }
    __syncwarp();
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

// A cluster of CTAs per (request, KV head), each with a slice of its candidates, the
// tokens between the sinks and the recent ones; in it every warp has a run.
// The n-th largest key is found digit by digit, 11 bits, 11 and 10 from the top: the
// CTAs count the candidates that share the digits found so far in a histogram each,
// and every one of them finds the digit from all: first by its upper 8 bits, then
// among 8 bins (reading all 2048 bins of 8 CTAs took 2.5 us a digit).  Then all
// keys above and, by position, as many of the equal ones as still fit are written:
// a warp puts its positions side by side where its keys were, and copies them out
// once it knows how many lie before them (written from the scan, a position at a
// time, they took 6 us of a long row).  Candidates behind the row's last, up to a
// whole group, count as -infinity: they come last of all by key and position.
// Bound by instructions (a long row takes about 70 for a key of each lane) and the
// latency of its steps alike: half of the issue slots are taken.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    shkv_select_kernel(const __grid_constant__ SelectParams p, int cached)
{
    constexpr int kWarps = kThreads / 32;
    extern __shared__ __align__(16) uint32_t dyn[];
    __shared__ uint32_t warp_sum[kCoarse / 32], found[2];      // found: coarse bin, keys in higher ones
    __shared__ uint32_t totals[2];
    __shared__ uint2 warp_counts[kWarps];
    uint32_t rank, ctas;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    for (int i = tid; i < 2 * kHist / 4; i += kThreads)
        reinterpret_cast<uint4 *>(dyn)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < 2)
        found[tid] = 0u;
    pdl_wait_prior();
    pdl_launch_dependents();
    const int log_ctas = 31 - __clz((int)ctas);          // a power of two
    const int b = blockIdx.y, g = blockIdx.x >> log_ctas;
    const int L = p.lens[b], keep = min(p.keep[b], L);
    const int all = rank * kThreads + tid, step = ctas * kThreads;
    int32_t *out = p.index + ((int64_t)b * p.hkv + g) * p.index_stride;
    if (g == 0 && all == 0 && p.seq_lens[b] != L)
        atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
#pragma unroll 4
    for (int64_t j = keep + all; j < p.index_stride; j += step)
        out[j] = -1;
    if (keep == L) {
        for (int j = all; j < L; j += step)
            out[j] = j;
        return;
    }
    for (int j = all; j < p.sink + p.recent; j += step) {
        const int from_end = p.sink + p.recent - j;
        out[j < p.sink ? j : keep - from_end] = j < p.sink ? j : L - from_end;
    }
    out += p.sink;
    const uint32_t chosen = (uint32_t)(keep - p.sink - p.recent);
    if (chosen == 0u)
        return;
    const int cand = L - p.sink - p.recent;
    const int per = ((cand + (int)ctas - 1 >> log_ctas) + kGroup - 1) & ~(kGroup - 1);
    const int c0 = min(cand, (int)rank * per), n = min(cand - c0, per);
    const int run = (n + kGroup * kWarps - 1) / (kGroup * kWarps) * kGroup;
    const int w0 = min(n, warp * run), w1 = min(n, w0 + run);
    const float *m = p.mass + b * p.mass_request + g * p.mass_head + p.sink + c0;
    uint32_t *const own = dyn + 2 * kHist + warp * run - w0;   // a run's keys, from w0 on
    // keys t .. t + 3 of the run
    auto four = [&](int t) -> uint4 {
        if (cached)
            return *reinterpret_cast<const uint4 *>(own + t);
        uint32_t k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            k[i] = mass_key(t + i < w1 ? m[t + i] : -INFINITY);
        return make_uint4(k[0], k[1], k[2], k[3]);
    };
    uint32_t prefix = 0u, need = chosen, equal = 0u;     // of the keys with this prefix; keys with all its digits
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        uint32_t *hist = dyn + (pass & 1) * kHist;
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        if (pass == 0) {
            constexpr int kU = 16;
            float x[kU];
            auto load = [&](int t) {
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    x[u] = t + u * 32 + lane < w1 ? m[t + u * 32 + lane] : -INFINITY;
            };
            load(w0);
            __syncthreads();                             // the histograms are empty
#pragma unroll 1
            for (int t = w0; t < w1;) {
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    if (u % 4 == 0 && t + u * 32 >= w1)
                        break;
                    const uint32_t k = mass_key(x[u]);
                    atomicAdd(hist + (k >> 21), 1u);
                    if (cached)
                        own[t + u * 32 + lane] = k;
                }
                t += kU * 32;
                if (t < w1)
                    load(t);
            }
            __syncwarp();
        } else {
            // keys prefix .. prefix + width share the digits found
            const uint32_t width = (1u << (pass == 1 ? 21 : 10)) - 1u;
#pragma unroll 2
            for (int t = w0; t < w1; t += kGroup) {
                const uint4 v = four(t + 4 * lane);
                const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (k[i] - prefix <= width)
                        atomicAdd(hist + (k[i] - prefix >> shift), 1u);
            }
        }
        __syncthreads();
        // thread i < 256: coarse bin 255 - i, of all CTAs
        uint32_t count = 0u;
        if (tid < kCoarse) {
            const uint4 *bin = reinterpret_cast<const uint4 *>(hist) + 2 * (kCoarse - 1 - tid);
            const uint4 v = bin[0], x = bin[1];
            count = (v.x + v.y + v.z + v.w) + (x.x + x.y + x.z + x.w);
        }
        if (ctas > 1) {
            uint32_t *bin = hist + kBins + tid;
            if (tid < kCoarse)
                *bin = count;
            row_sync(ctas);
            if (tid < kCoarse) {
                count = 0u;
#pragma unroll 4
                for (uint32_t r = 0; r < ctas; ++r)
                    count += load_of_rank(bin, r);
            }
        }
        if (pass == 1)                               // the first histogram serves again: all have read it
            for (int i = tid; i < kHist / 4; i += kThreads)
                reinterpret_cast<uint4 *>(dyn)[i] = make_uint4(0u, 0u, 0u, 0u);
        uint32_t upto = count;
        if (tid < kCoarse) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                upto += lane >= o ? v : 0u;
            }
            if (lane == 31)
                warp_sum[warp] = upto;
        }
        __syncthreads();
        if (tid < kCoarse) {
#pragma unroll
            for (int w = 0; w < kCoarse / 32; ++w)
                upto += w < warp ? warp_sum[w] : 0u;
            if (upto - count < need && need <= upto) {
                found[0] = (uint32_t)(kCoarse - 1 - tid);
                found[1] = upto - count;              // keys in higher coarse bins
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
            equal = __shfl_sync(0xffffffffu, v, at);
            prefix |= (coarse * 8u + 7u - (uint32_t)at) << shift;
        }
    }
    // All larger keys stay, and `need` of the `equal` keys that are `prefix`: all of
    // them, as a rule.  Then a run's positions take the place of its keys, four groups
    // at a time, their counts in a byte each (up to 128).
    const bool listed = cached && equal == need;
    uint32_t *const list = own + w0;
    uint32_t some = 0u, same = 0u;                       // that stay; equal ones where not all do
    for (int t = w0; t < w1; t += 4 * kGroup) {
        uint32_t k[16], mine = 0u;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint4 x = t + v * kGroup < w1 ? four(t + v * kGroup + 4 * lane) : make_uint4(0u, 0u, 0u, 0u);
            k[4 * v] = x.x, k[4 * v + 1] = x.y, k[4 * v + 2] = x.z, k[4 * v + 3] = x.w;
#pragma unroll
            for (int i = 4 * v; i < 4 * v + 4; ++i)
                mine += k[i] >= prefix ? 1u << 8 * v : 0u;
        }
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? y : 0u;
        }
        const uint32_t sum = __shfl_sync(0xffffffffu, upto, 31);
        if (listed) {
            upto -= mine;
            __syncwarp();                                // the keys have been read
            uint32_t first = some;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                uint32_t *to = list + first + (upto >> 8 * v & 255u);
#pragma unroll
                for (int i = 4 * v; i < 4 * v + 4; ++i)
                    if (k[i] >= prefix)
                        *to++ = (uint32_t)(t + v * kGroup + 4 * lane + (i & 3));
                first += sum >> 8 * v & 255u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                same += k[i] == prefix;
        }
        some += (sum & 255u) + (sum >> 8 & 255u) + (sum >> 16 & 255u) + (sum >> 24);
    }
    same = __reduce_add_sync(0xffffffffu, same);
    if (lane == 0)
        warp_counts[warp] = make_uint2(some - same, same);
    __syncthreads();
    // those above (and equal ones, where listed) and equal ones: before this warp's, of the CTA
    uint32_t na, ne, a, e;
    {
        const uint2 c = lane < kWarps ? warp_counts[lane] : make_uint2(0u, 0u);
        na = __reduce_add_sync(0xffffffffu, lane < warp ? c.x : 0u);
        ne = __reduce_add_sync(0xffffffffu, lane < warp ? c.y : 0u);
        a = __reduce_add_sync(0xffffffffu, c.x);
        e = __reduce_add_sync(0xffffffffu, c.y);
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
    // (a place of `chosen` and above: only if masses change under the call)
    const int base = p.sink + c0;
    const uint32_t below = (1u << lane) - 1u;
    if (listed) {
        for (uint32_t j = lane; j < some; j += 32)
            if (na + j < chosen)
                out[na + j] = base + (int32_t)list[j];
    } else {
        for (int t0 = w0; t0 < w1; t0 += 32) {
            const int t = t0 + lane;
            const uint32_t k = t >= w1 ? 0u : cached ? own[t] : mass_key(m[t]);
            const bool up = k > prefix, eq = k == prefix;
            const uint32_t ups = __ballot_sync(0xffffffffu, up), eqs = __ballot_sync(0xffffffffu, eq);
            const uint32_t pe = ne + __popc(eqs & below), at = na + __popc(ups & below) + min(pe, need);
            if ((up || (eq && pe < need)) && at < chosen)
                out[at] = base + t;
            na += __popc(ups);
            ne += __popc(eqs);
        }
    }
    if (ctas > 1)
        row_sync(ctas);                                  // nobody leaves while its counts are read
}

// A row gets more CTAs (a cluster of up to 8) as long as a slice keeps 16384 tokens
// and each has an SM to itself (32 rows of 131584: 4 CTAs 17 us, 8, two on some SMs, 45;
// 8 rows of 12000: 1 CTA 9.0 us, 4 10.5; of 40000: 4 CTAs 12.4 us, 8 14.1), and more than
// there are SMs where its keys fit shared memory only then (192 rows of 131000: 4 CTAs
// 105 us, one that reads its masses from global memory in every pass 202).
//
// Threads: as many as make 1024 an SM, by the CTAs that its shared memory takes, 512 a
// row where rows do not fill the SMs.  (256 / 512 / 1024 threads: 512 rows of 1K to 8K
// 13.6 / 15.8 / 22.3 us; 320 rows of 8K to 12K 16.9 / 14.8 / 19.0; 320 of 14K to 16K
// 18.5 / 17.3 / 21.8; 128 of 20K to 40K 26.2 / 19.3 / 18.1; 128 of 8000 9.2 / 7.9 / 9.1.)
cudaError_t launch_select(const SelectParams &p, int num_sms, cudaStream_t stream)
{
    int64_t longest = 0;
    for (int b = 0; b < p.batch; ++b)
        if (p.keep[b] < p.lens[b])
            longest = p.lens[b] > longest ? p.lens[b] : longest;
    const int64_t rows = (int64_t)p.batch * p.hkv;
    int ctas = 1;
    while (ctas < 8 && longest > 16384 * ctas &&
           (2 * ctas * rows <= num_sms || (longest > (int64_t)kSelectKeys * ctas && longest <= 8 * kSelectKeys)))
        ctas *= 2;
    const int64_t room = kSmemSm / (2 * kHist * 4 + 1024 + 4 * longest);
    const int threads = ctas > 1 || room < 2 ? 1024 : room < 4 || (rows <= num_sms && longest > 4096) ? 512 : 256;
    auto kern = threads == 1024  ? shkv_select_kernel<1024>
                : threads == 512 ? shkv_select_kernel<512>
                                 : shkv_select_kernel<256>;
    // runs of whole groups
    const int64_t part = (longest + ctas - 1) / ctas, unit = kGroup * (threads / 32);
    const int64_t slice = (part + unit - 1) / unit * unit;
    const int cached = slice <= kSelectKeys;
    const uint32_t front = 2 * kHist * 4, smem = front + (uint32_t)(cached ? slice * 4 : 0);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)front + kSelectKeys * 4);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.hkv * ctas), (unsigned)p.batch);
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
// written, and as positions ascend it writes only below what later passes read.  A
// token whose row is not copied gets 0: what its slot holds is not its own.  (The
// tables are looked through first, and token by token only if a page is none, in a
// walk of its own: one row of 131072 to half 43 us (d 64) and 40 (d 128), without the
// look 37 and 40; asked in the passes 54, whose 16 masses were then not loaded
// together.)
__device__ __forceinline__ void move_masses(const EvictParams &p, int row)
{
    const int b = row / p.hkv, g = row % p.hkv;
    const int L = p.lens[b], keep = p.keep[b];
    if (keep >= L)
        return;
    const int32_t *index = p.index + (int64_t)row * p.index_stride;
    const float *src = p.mass.in + b * p.mass.in_request + g * p.mass.in_head;
    float *dst = p.mass.out + b * p.mass.out_request + g * p.mass.out_head;
    const int32_t *from = p.table + b * p.table_stride, *to = p.new_table + b * p.new_stride;
    const int shift = p.page_size == 16 ? 4 : 5;
    auto inside = [&](int page) { return (uint32_t)page < (uint32_t)p.num_pages; };
    bool bad = false;
    auto look = [&](const int32_t *pages, int n) {
        for (int i0 = threadIdx.x; i0 < n; i0 += kMassPer * kMoveThreads) {
            int x[kMassPer];
#pragma unroll
            for (int u = 0; u < kMassPer; ++u)
                x[u] = i0 + u * kMoveThreads < n ? pages[i0 + u * kMoveThreads] : 0;
#pragma unroll
            for (int u = 0; u < kMassPer; ++u)
                bad = bad || !inside(x[u]);
        }
    };
    look(from, (L + p.page_size - 1) >> shift);
    look(to, (keep + p.page_size - 1) >> shift);
    bad = __syncthreads_or(bad);
    for (int j0 = 0; j0 < keep; j0 += kMassPer * kMoveThreads) {
        int i[kMassPer];
        float x[kMassPer];
#pragma unroll
        for (int u = 0; u < kMassPer; ++u) {
            const int j = j0 + u * kMoveThreads + threadIdx.x;
            i[u] = j < keep ? index[j] : -1;
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
    if (bad)
        for (int j = threadIdx.x; j < keep; j += kMoveThreads) {
            const int i = index[j];
            if ((uint32_t)i < (uint32_t)L && !(inside(from[i >> shift]) && inside(to[j >> shift])))
                dst[j] = 0.f;
        }
    for (int j0 = keep + threadIdx.x; j0 < L; j0 += kMassZeros * kMoveThreads)
#pragma unroll
        for (int u = 0; u < kMassZeros; ++u)
            if (j0 + u * kMoveThreads < L)
                dst[j0 + u * kMoveThreads] = 0.f;
}

// The request's table row and length, by a CTA.
__device__ __forceinline__ void commit_request(const EvictParams &p, int b)
{
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

}  // namespace

// The first CTAs write tables and lengths, where the move reads a table of the
// caller's (one launch less than from the pool's own: 1 to 2 us of the GPU, up to 2 of
// the host), the next ones move masses.  The others copy rows, a warp per (new page,
// KV head): K's and V's rows of 32 / (2 D / 8) tokens an instruction, eight
// instructions' loads before their stores.  Bound by HBM: 48 requests to half, 491 MB,
// 79 us (93% of a copy's rate).  The eight loads need 72 to 76 registers, three CTAs an
// SM: left to itself the compiler took 56 and loaded fewer at once (104 us; 16 loads of
// a thread 90, 4 and five CTAs 81); stores that stay longer in L2 81 us.
template <int D>
__global__ void __launch_bounds__(kMoveThreads, 3) shkv_evict_kernel(const __grid_constant__ EvictParams p)
{
    constexpr int V = D / 8, kTok = 32 / (2 * V);        // vectors of a row, tokens an instruction
    constexpr int kU = 8;
    pdl_wait_prior();
    if (!p.at_once)                  // as in the kernel below
        pdl_launch_dependents();
    const int commits = p.at_once ? p.batch : 0, mass_blocks = p.mass.out ? p.batch * p.hkv : 0;
    const int block = (int)blockIdx.x - commits - mass_blocks;
    if ((int)blockIdx.x < commits) {
        commit_request(p, blockIdx.x);
        return;
    }
    if (block < 0) {
        move_masses(p, blockIdx.x - commits);
        return;
    }
    const int lane = threadIdx.x & 31, P = p.page_size;
    const int w = block * (kMoveThreads / 32) + threadIdx.x / 32;
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
    const int to = p.new_table[b * p.new_stride + j0 / P];
    bool ok = (uint32_t)to < (uint32_t)p.num_pages;
    int row = 0;                                         // of the lane's token (a pool's rows fit 32 bits)
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
                __stcs(dst + (int64_t)t * V, x[u]);
        }
    }
}

// After a move that read the pool's own table: the requests' tables and lengths.
// Lets no dependent start early: the unit kernel of a decode with tails reads the
// table without waiting for its predecessor.
__global__ void __launch_bounds__(kMoveThreads) shkv_evict_commit_kernel(const __grid_constant__ EvictParams p)
{
    pdl_wait_prior();
    commit_request(p, blockIdx.x);
}

cudaError_t launch_evict(const EvictParams &p, cudaStream_t stream)
{
    const int64_t warps = (int64_t)p.page0[p.batch] * p.hkv;
    const int64_t grid = (p.at_once ? p.batch : 0) + (p.mass.out ? (int64_t)p.batch * p.hkv : 0) + (warps + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
    auto kern = p.head_dim == 64 ? shkv_evict_kernel<64> : shkv_evict_kernel<128>;
    cudaError_t e = grid ? launch_pdl(kern, (int)grid, kMoveThreads, 0u, stream, p) : cudaSuccess;
    if (e == cudaSuccess && !p.at_once)
        e = launch_pdl(shkv_evict_commit_kernel, p.batch, kMoveThreads, 0u, stream, p);
    return e;
}

}  // namespace shkv
