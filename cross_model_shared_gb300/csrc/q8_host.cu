// q8_host.cu -- the C ABI of the 8-bit KV cache: argument checks and kernel
// launches.  Declarations and their contracts are in include/shkv.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <exception>
#include <new>

#include "host_shared.h"
#include "q8.cuh"
#include "q8_chunk.cuh"
#include "q8_decode.cuh"
#include "shkv.h"

namespace shkv {
cudaError_t launch_q8_cache(const Q8CacheParams &p, bool read, int num_sms, cudaStream_t stream);
cudaError_t launch_q8_clear_errors(uint32_t *err, uint32_t bits, cudaStream_t stream);
cudaError_t launch_q8_chunk(const CUtensorMap &tmK, const CUtensorMap &tmV, const Q8ChunkParams &p, bool splits,
                            cudaStream_t stream);
cudaError_t launch_q8_decode(const CUtensorMap &tmK, const CUtensorMap &tmV, const Q8DecodeParams &q,
                             cudaStream_t stream);
}  // namespace shkv

using namespace shkv;

struct shkv_q8_pool {
    shkv_q8_pool_config cfg;
    int device;
    int num_sms;
    CUtensorMap tm_k, tm_v;          // one page of one KV head a box
    int32_t lens[SHKV_MAX_BATCH];    // host copy of seq_lens
};

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

shkv_status status_of(cudaError_t e) { return e == cudaSuccess ? SHKV_OK : SHKV_ERR_CUDA; }

bool on_pool_device(const shkv_q8_pool *pool)
{
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == pool->device;
}

// Calls that wait for their stream cannot be captured into a graph.
bool capturing(cudaStream_t stream)
{
    cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
    return cudaStreamIsCapturing(stream, &s) != cudaSuccess || s != cudaStreamCaptureStatusNone;
}

int64_t capacity(const shkv_q8_pool *pool) { return (int64_t)pool->cfg.max_pages_per_seq * pool->cfg.page_size; }

// Checks and parameters common to append and read.
shkv_status cache_params(const shkv_q8_pool *pool, int32_t batch, const int32_t *start, const int32_t *lens,
                         const void *k, int64_t k_stride, const void *v, int64_t v_stride, Q8CacheParams &p)
{
    const shkv_q8_pool_config &c = pool->cfg;
    const int64_t row = (int64_t)c.num_kv_heads * c.head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8)
        return SHKV_ERR_INVALID_ARG;
    memset(&p, 0, sizeof p);
    int64_t total = 0;
    for (int b = 0; b < batch; ++b) {
        if (lens[b] < 0 || (start && start[b] < 0))
            return SHKV_ERR_INVALID_ARG;
        p.tok0[b] = (int32_t)total;
        p.start[b] = start ? start[b] : pool->lens[b];
        p.old_len[b] = pool->lens[b];
        total += lens[b];
        if (total * 2 * c.num_kv_heads > INT32_MAX)
            return SHKV_ERR_UNSUPPORTED;
    }
    p.tok0[batch] = (int32_t)total;
    if (total > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16)))
        return SHKV_ERR_INVALID_ARG;
    p.k = static_cast<__nv_bfloat16 *>(const_cast<void *>(k));
    p.v = static_cast<__nv_bfloat16 *>(const_cast<void *>(v));
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.k_pages = static_cast<uint8_t *>(c.k_pages);
    p.v_pages = static_cast<uint8_t *>(c.v_pages);
    p.scales = static_cast<uint8_t *>(c.scales);
    p.block_table = c.block_table;
    p.seq_lens = c.seq_lens;
    p.err = c.error_word;
    p.batch = batch;
    p.hkv = c.num_kv_heads;
    p.head_dim = c.head_dim;
    p.page_size = c.page_size;
    p.max_pages = c.max_pages_per_seq;
    p.num_pages = c.num_pages;
    return SHKV_OK;
}

shkv_status launch_cache(shkv_q8_pool *pool, const Q8CacheParams &p, bool read, void *stream)
{
    if (launch_q8_cache(p, read, pool->num_sms, (cudaStream_t)stream) != cudaSuccess)
        return SHKV_ERR_CUDA;
    if (!read)
        for (int b = 0; b < p.batch; ++b)
            pool->lens[b] = p.start[b] + (p.tok0[b + 1] - p.tok0[b]);
    const size_t tokens = (size_t)p.tok0[p.batch];
    const size_t row = (size_t)p.hkv * p.head_dim;
    const size_t kb = tokens ? ((tokens - 1) * p.k_stride + row) * 2 : 0;
    const size_t vb = tokens ? ((tokens - 1) * p.v_stride + row) * 2 : 0;
    record_stream_use(stream, {span_of(p.k, kb), span_of(p.v, vb)});
    return SHKV_OK;
}

// 2-D view of a code pool: dim0 = head_dim bytes, dim1 = the (page, KV head,
// slot) rows.  One box {128, P} with 128-byte swizzle is one page of one KV
// head; at head_dim 64 its upper half lies outside the tensor and is filled
// with zeros, so that the kernels see 128-byte rows.
bool make_map(CUtensorMap *tm, void *base, const shkv_q8_pool_config &c)
{
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc)
        return false;
    cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.num_pages * c.num_kv_heads * c.page_size};
    cuuint64_t strides[1] = {(cuuint64_t)c.head_dim};
    cuuint32_t box[2] = {128u, (cuuint32_t)c.page_size};
    cuuint32_t estr[2] = {1u, 1u};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int32_t kMaxDecodeRows = 64;     // stacked rows per KV head that one decode launch takes

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The workspace: an arrival counter per (request, KV head) of the pool's
// largest batch, then two partials per SM, log-sum-exps and rows, of up to 64
// (stacked) or kChunkRows (chunk) rows.  Nothing else is ever written over the
// counters; the two kernels of a call use the partials one after the other.
size_t count_bytes(const shkv_q8_pool *p) { return align256((size_t)p->cfg.max_batch * p->cfg.num_kv_heads * 4); }
size_t lse_bytes(const shkv_q8_pool *p) { return align256((size_t)2 * p->num_sms * kChunkRows * 4); }
size_t workspace_need(const shkv_q8_pool *p)
{
    return count_bytes(p) + lse_bytes(p) + (size_t)2 * p->num_sms * kChunkRows * p->cfg.head_dim * 4;
}

int max_ctas(const shkv_q8_pool *p) { return std::min(p->num_sms, std::min(kMaxCtas, kChunkMaxCtas)); }

// Up to 64 stacked rows per (request, KV head).
shkv_status launch_stacked(shkv_q8_pool *pool, const Q8AttnParams &a, int max_rows, void *workspace, cudaStream_t stream)
{
    Q8DecodeParams q;
    memset(&q, 0, sizeof q);
    DecodeParams &d = q.d;
    int32_t keys[SHKV_MAX_BATCH];           // of the requests that have rows
    for (int b = 0; b < a.batch; ++b) {
        keys[b] = a.n_q[b] ? a.lens[b] : 0;
        q.n_q[b] = a.n_q[b];
        q.q0[b] = a.q0[b];
        q.has_empty |= a.n_q[b] && !keys[b];
    }
    // fitted over 16 batches of 8, 32 and 40 rows: a piece costs about 5 stages
    // whatever its rows (costs growing with the rows were 6% slower), flat around
    // these values
    const shkv_status st =
        plan_pages(a.batch, keys, a.page_size, a.hkv, max_ctas(pool), 128, 600, 250, 600,
                   d.page_prefix, d.last_fill, d.cta_cut, &d.total_chunks, &d.num_ctas);
    if (st != SHKV_OK)
        return st;
    d.q = a.q;
    d.out = a.out;
    d.lse_out = a.lse_out;
    d.block_table = a.block_table;
    d.seq_lens = a.seq_lens;
    d.err = a.err;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    d.ws_count = reinterpret_cast<uint32_t *>(ws);
    d.ws_lse = reinterpret_cast<float *>(ws + count_bytes(pool));
    d.ws_part = reinterpret_cast<float *>(ws + count_bytes(pool) + lse_bytes(pool));
    d.batch = a.batch;
    d.hq = a.hq;
    d.hkv = a.hkv;
    d.group = a.group;
    d.rows = max_rows;
    d.page_size = a.page_size;
    d.max_pages = a.max_pages;
    d.num_pages = a.num_pages;
    d.scale_log2 = a.scale_log2;
    q.scales = a.scales;
    q.q_stride = a.q_stride;
    q.head_dim = a.head_dim;
    q.causal = a.causal;
    return status_of(launch_q8_decode(pool->tm_k, pool->tm_v, q, stream));
}

// Cuts the units' stages into at most `limit` contiguous ranges so that the
// costliest is as cheap as a greedy fill makes it (bisection over the bound).
// In fifths of a stage of both tiles: a piece pays kPiece for its query rows,
// the pipeline's fill and drain and its output, a stage 5 (3 with one tile).
// (Fitted to the ranges' end times; a piece at 20 was 4 to 7% slower.)
constexpr int64_t kPiece = 30, kPair = 5, kSingle = 3;
constexpr int64_t kMinPiece = 2;            // stages; smaller pieces are not cut off

bool plan_chunks(Q8ChunkParams &p, int limit)
{
    const int hkv = p.hkv, tpt = p.tpt;
    int64_t total = 0, stages = 0;
    for (int b = 0; b < p.batch; ++b) {
        const int tiles = (p.n_q[b] + tpt - 1) / tpt;
        for (int tp = 0; 2 * tp < tiles; ++tp) {
            const int64_t nst = chunk_stages(p.lens[b], p.n_q[b], tpt, tp);
            total += hkv * (kPiece + nst * (2 * tp + 1 < tiles ? kPair : kSingle));
            stages += hkv * nst;
        }
    }
    const int64_t C = std::max<int64_t>(1, std::min<int64_t>(limit, stages / kMinPiece));
    auto fill = [&](int64_t bound, bool out) -> int64_t {
        int64_t acc = 0;
        int c = 0, u = 0;
        for (int b = 0; b < p.batch; ++b) {
            const int tiles = (p.n_q[b] + tpt - 1) / tpt;
            for (int g = 0; g < hkv; ++g)
                for (int tp = 0; 2 * tp < tiles; ++tp, ++u) {
                    const int64_t w = 2 * tp + 1 < tiles ? kPair : kSingle;
                    int64_t rest = chunk_stages(p.lens[b], p.n_q[b], tpt, tp), s = 0;
                    while (acc + kPiece + rest * w > bound) {
                        int64_t m = std::min((bound - acc - kPiece) / w, rest - kMinPiece);
                        if (m < kMinPiece)
                            m = 0;
                        if ((m == 0 && acc == 0) || ++c >= C)
                            return C + 1;
                        s += m;
                        rest -= m;
                        acc = 0;
                        if (out) {
                            p.cut_unit[c] = u;
                            p.cut_stage[c] = (int32_t)s;
                        }
                    }
                    acc += kPiece + rest * w;
                }
        }
        if (out) {
            p.cut_unit[0] = p.cut_stage[0] = 0;
            p.cut_unit[c + 1] = u;
            p.cut_stage[c + 1] = 0;
        }
        return c + 1;
    };
    int64_t lo = total / C - 1, hi = total / C + 2 * kPiece;
    while (fill(hi, false) > C)
        hi += hi - lo;
    const int64_t tol = std::max<int64_t>(1, total / C / 256);
    while (hi - lo > tol) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (fill(mid, false) <= C)
            hi = mid;
        else
            lo = mid;
    }
    p.num_ctas = (int32_t)fill(hi, true);
    for (int c = 1; c < p.num_ctas; ++c)
        if (p.cut_stage[c] > 0)
            return true;
    return false;
}

shkv_status launch_chunk(shkv_q8_pool *pool, const Q8AttnParams &a, void *workspace, cudaStream_t stream)
{
    Q8ChunkParams p;
    memset(&p, 0, sizeof p);
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.out = a.out;
    p.lse_out = a.lse_out;
    p.scales = a.scales;
    p.block_table = a.block_table;
    p.seq_lens = a.seq_lens;
    p.err = a.err;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.ws_lse = reinterpret_cast<float *>(ws + count_bytes(pool));
    p.ws_part = reinterpret_cast<float *>(ws + count_bytes(pool) + lse_bytes(pool));
    p.batch = a.batch;
    p.hq = a.hq;
    p.hkv = a.hkv;
    p.group = a.group;
    p.head_dim = a.head_dim;
    p.page_size = a.page_size;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.tpt = 128 / a.group;
    p.scale_log2 = a.scale_log2;
    int64_t units = 0;
    for (int b = 0; b < a.batch; ++b) {
        p.units[b] = (int32_t)units;
        p.lens[b] = a.lens[b];
        p.n_q[b] = a.n_q[b];
        p.q0[b] = a.q0[b];
        const int tiles = (a.n_q[b] + p.tpt - 1) / p.tpt;
        units += (int64_t)a.hkv * ((tiles + 1) / 2);
        if (units > INT32_MAX)
            return SHKV_ERR_UNSUPPORTED;
    }
    p.units[a.batch] = (int32_t)units;
    const bool splits = plan_chunks(p, max_ctas(pool));
    return status_of(launch_q8_chunk(pool->tm_k, pool->tm_v, p, splits, stream));
}

// Both attentions: n_q query tokens of request b start at query token q0[b].
shkv_status attention(shkv_q8_pool *pool, Q8AttnParams &p, int32_t hq, const void *q, int64_t q_stride, float scale,
                      void *out, float *lse_out, void *workspace, size_t ws_bytes, void *stream)
{
    const shkv_q8_pool_config &c = pool->cfg;
    const float scale_log2 = (float)((double)scale * 1.4426950408889634);
    if (!q || !out || !workspace || !aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(lse_out, 4) || q_stride < (int64_t)hq * c.head_dim || q_stride % 8 || !isfinite(scale_log2) ||
        ws_bytes < workspace_need(pool))
        return SHKV_ERR_INVALID_ARG;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_stride = q_stride;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse_out = lse_out;
    p.scales = static_cast<const uint8_t *>(c.scales);
    p.block_table = c.block_table;
    p.seq_lens = c.seq_lens;
    p.err = c.error_word;
    p.hq = hq;
    p.hkv = c.num_kv_heads;
    p.group = hq / c.num_kv_heads;
    p.head_dim = c.head_dim;
    p.page_size = c.page_size;
    p.max_pages = c.max_pages_per_seq;
    p.num_pages = c.num_pages;
    p.scale_log2 = scale_log2;
    // requests of up to kMaxDecodeRows rows per KV head go to the stacked
    // kernel, which reads a page once for all of them (16 requests of 4000
    // tokens, 8 KV heads: 64 rows 51 us; the chunk kernel takes 69 us for 68 to
    // 128 rows: one tile, nothing to overlap its chain with, so 68 rows cost a
    // third more than 64), the others to the chunk kernel; a few small requests
    // beside large ones go along with them, where that costs a CTA less than the
    // second launch (about 12 us, the time of 6 stages; a mixed batch of 9
    // requests took 41 us with it, 24 without)
    int max_rows = 0;
    int64_t tokens = 0, small_cost = 0;
    Q8AttnParams large = p;
    bool any_large = false;
    for (int b = 0; b < p.batch; ++b) {
        tokens += p.n_q[b];
        if ((int64_t)p.n_q[b] * p.group > kMaxDecodeRows) {
            any_large = true;
        } else if (p.n_q[b]) {
            max_rows = std::max(max_rows, p.n_q[b] * p.group);
            small_cost += p.hkv * (kPiece + (int64_t)(p.lens[b] + 127) / 128 * kSingle);
        }
    }
    if (any_large && small_cost <= 6 * kPair * (int64_t)pool->num_sms)
        max_rows = 0;                        // all to the chunk kernel
    else
        for (int b = 0; b < p.batch; ++b)
            ((int64_t)p.n_q[b] * p.group > kMaxDecodeRows ? p : large).n_q[b] = 0;
    shkv_status st = SHKV_OK;
    if (any_large)
        st = launch_chunk(pool, large, workspace, (cudaStream_t)stream);
    if (st == SHKV_OK && max_rows > 0)
        st = launch_stacked(pool, p, max_rows, workspace, (cudaStream_t)stream);
    if (st != SHKV_OK)
        return st;
    const size_t row = (size_t)hq * c.head_dim;
    record_stream_use(stream, {span_of(workspace, workspace_need(pool)),
                               span_of(q, ((size_t)(tokens - 1) * q_stride + row) * 2),
                               span_of(out, (size_t)tokens * row * 2), span_of(lse_out, (size_t)tokens * hq * 4)});
    return SHKV_OK;
}

}  // namespace

extern "C" {

shkv_status shkv_q8_pool_create(const shkv_q8_pool_config *cfg, shkv_q8_pool **out)
{
    if (!cfg || !out)
        return SHKV_ERR_INVALID_ARG;
    *out = nullptr;
    const shkv_q8_pool_config &c = *cfg;
    if (c.num_pages <= 0 || c.num_kv_heads <= 0 || c.max_batch <= 0 || c.max_pages_per_seq <= 0 || !c.k_pages ||
        !c.v_pages || !c.scales || !c.block_table || !c.seq_lens || !c.error_word)
        return SHKV_ERR_INVALID_ARG;
    if (!aligned(c.k_pages, 16) || !aligned(c.v_pages, 16) || !aligned(c.scales, 16) || !aligned(c.block_table, 4) ||
        !aligned(c.seq_lens, 4) || !aligned(c.error_word, 4))
        return SHKV_ERR_INVALID_ARG;
    if ((c.page_size != 16 && c.page_size != 32) || (c.head_dim != 64 && c.head_dim != 128) ||
        c.max_batch > SHKV_MAX_BATCH || (int64_t)c.num_pages * c.num_kv_heads * c.page_size > INT32_MAX ||
        (int64_t)c.max_pages_per_seq * c.page_size > INT32_MAX)
        return SHKV_ERR_UNSUPPORTED;
    if (c.initial_seq_lens)
        for (int b = 0; b < c.max_batch; ++b)
            if (c.initial_seq_lens[b] < 0 ||
                (int64_t)c.initial_seq_lens[b] > (int64_t)c.max_pages_per_seq * c.page_size)
                return SHKV_ERR_CAPACITY;
    shkv_q8_pool *pool = new (std::nothrow) shkv_q8_pool();
    if (!pool)
        return SHKV_ERR_INVALID_ARG;
    pool->cfg = c;
    pool->cfg.initial_seq_lens = nullptr;
    memset(pool->lens, 0, sizeof pool->lens);
    if (c.initial_seq_lens)
        memcpy(pool->lens, c.initial_seq_lens, sizeof(int32_t) * c.max_batch);
    if (cudaGetDevice(&pool->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&pool->num_sms, cudaDevAttrMultiProcessorCount, pool->device) != cudaSuccess ||
        !make_map(&pool->tm_k, c.k_pages, c) || !make_map(&pool->tm_v, c.v_pages, c) ||
        cudaMemcpy(c.seq_lens, pool->lens, sizeof(int32_t) * c.max_batch, cudaMemcpyHostToDevice) !=
            cudaSuccess ||
        cudaMemset(c.error_word, 0, sizeof(uint32_t)) != cudaSuccess) {
        delete pool;
        return SHKV_ERR_CUDA;
    }
    *out = pool;
    return SHKV_OK;
}

shkv_status shkv_q8_pool_destroy(shkv_q8_pool *pool)
{
    if (!pool)
        return SHKV_ERR_INVALID_ARG;
    delete pool;
    return SHKV_OK;
}

shkv_status shkv_q8_pool_set_seq_lens(shkv_q8_pool *pool, int32_t batch, const int32_t *lens, void *stream)
{
    if (!pool || !lens || batch < 0 || batch > pool->cfg.max_batch || !on_pool_device(pool))
        return SHKV_ERR_INVALID_ARG;
    for (int b = 0; b < batch; ++b)
        if (lens[b] < 0 || lens[b] > capacity(pool))
            return SHKV_ERR_CAPACITY;
    if (batch == 0)
        return SHKV_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (capturing(st))
        return SHKV_ERR_INVALID_ARG;
    memcpy(pool->lens, lens, sizeof(int32_t) * batch);
    cudaError_t e =
        cudaMemcpyAsync(pool->cfg.seq_lens, pool->lens, sizeof(int32_t) * batch, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    return status_of(e);
}

shkv_status shkv_q8_pool_get_seq_lens(const shkv_q8_pool *pool, int32_t batch, int32_t *lens)
{
    if (!pool || !lens || batch < 0 || batch > pool->cfg.max_batch)
        return SHKV_ERR_INVALID_ARG;
    memcpy(lens, pool->lens, sizeof(int32_t) * batch);
    return SHKV_OK;
}

shkv_status shkv_q8_append_kv(shkv_q8_pool *pool, int32_t batch, const int32_t *start, const int32_t *new_lens,
                              const void *k_new, int64_t k_stride, const void *v_new, int64_t v_stride, void *stream)
try {
    if (!pool || !new_lens || batch < 0 || batch > pool->cfg.max_batch || !on_pool_device(pool))
        return SHKV_ERR_INVALID_ARG;
    Q8CacheParams p;
    const shkv_status st = cache_params(pool, batch, start, new_lens, k_new, k_stride, v_new, v_stride, p);
    if (st != SHKV_OK)
        return st;
    bool moves = false;
    for (int b = 0; b < batch; ++b) {
        if (p.start[b] > pool->lens[b])
            return SHKV_ERR_INVALID_ARG;     // would leave a gap of unwritten tokens
        if ((int64_t)p.start[b] + new_lens[b] > capacity(pool))
            return SHKV_ERR_CAPACITY;
        moves = moves || p.start[b] != pool->lens[b] || new_lens[b] > 0;
    }
    if (!moves)
        return SHKV_OK;
    return launch_cache(pool, p, false, stream);
} catch (const std::exception &) {
    return SHKV_ERR_CUDA;                // no host memory for the plan
}

shkv_status shkv_q8_read_kv(shkv_q8_pool *pool, int32_t batch, const int32_t *start, const int32_t *lens, void *k_out,
                            int64_t k_stride, void *v_out, int64_t v_stride, void *stream)
try {
    if (!pool || !start || !lens || batch < 0 || batch > pool->cfg.max_batch || !on_pool_device(pool))
        return SHKV_ERR_INVALID_ARG;
    Q8CacheParams p;
    const shkv_status st = cache_params(pool, batch, start, lens, k_out, k_stride, v_out, v_stride, p);
    if (st != SHKV_OK)
        return st;
    for (int b = 0; b < batch; ++b)
        if ((int64_t)start[b] + lens[b] > pool->lens[b])
            return SHKV_ERR_INVALID_ARG;
    if (p.tok0[batch] == 0)
        return SHKV_OK;
    return launch_cache(pool, p, true, stream);
} catch (const std::exception &) {
    return SHKV_ERR_CUDA;                // no host memory for the plan
}

shkv_status shkv_q8_workspace_size(const shkv_q8_pool *pool, size_t *bytes, size_t *zero_bytes)
{
    if (!pool || !bytes || !zero_bytes)
        return SHKV_ERR_INVALID_ARG;
    *bytes = workspace_need(pool);
    *zero_bytes = count_bytes(pool);
    return SHKV_OK;
}

shkv_status shkv_q8_decode_attention(shkv_q8_pool *pool, int32_t batch, int32_t n_models, int32_t hq_per_model,
                                     const void *q, float scale, void *out, float *lse_out, void *workspace,
                                     size_t workspace_bytes, void *stream)
try {
    if (!pool || batch < 1 || batch > pool->cfg.max_batch || n_models < 1 || hq_per_model < 1 ||
        !on_pool_device(pool))
        return SHKV_ERR_INVALID_ARG;
    const int32_t hkv = pool->cfg.num_kv_heads;
    if (hq_per_model % hkv || (int64_t)n_models * (hq_per_model / hkv) > kMaxDecodeRows)
        return SHKV_ERR_UNSUPPORTED;
    Q8AttnParams p;
    memset(&p, 0, sizeof p);
    p.batch = batch;
    p.causal = 0;
    for (int b = 0; b < batch; ++b) {
        p.lens[b] = pool->lens[b];
        p.n_q[b] = n_models;
        p.q0[b] = b * n_models;
    }
    return attention(pool, p, hq_per_model, q, (int64_t)hq_per_model * pool->cfg.head_dim, scale, out, lse_out,
                     workspace, workspace_bytes, stream);
} catch (const std::exception &) {
    return SHKV_ERR_CUDA;                // no host memory for the plan
}

shkv_status shkv_q8_chunk_attention(shkv_q8_pool *pool, int32_t batch, const int32_t *new_lens, int32_t hq,
                                    const void *q, int64_t q_stride, float scale, void *out, float *lse_out,
                                    void *workspace, size_t workspace_bytes, void *stream)
try {
    if (!pool || !new_lens || batch < 1 || batch > pool->cfg.max_batch || hq < 1 || !on_pool_device(pool))
        return SHKV_ERR_INVALID_ARG;
    const int32_t hkv = pool->cfg.num_kv_heads;
    if (hq % hkv || hq / hkv > 128)
        return SHKV_ERR_UNSUPPORTED;
    Q8AttnParams p;
    memset(&p, 0, sizeof p);
    p.batch = batch;
    p.causal = 1;
    int64_t tokens = 0;
    for (int b = 0; b < batch; ++b) {
        if (new_lens[b] < 0 || new_lens[b] > pool->lens[b])
            return SHKV_ERR_INVALID_ARG;     // the new tokens must already be in the pool
        p.lens[b] = pool->lens[b];
        p.n_q[b] = new_lens[b];
        p.q0[b] = (int32_t)tokens;
        tokens += new_lens[b];
        if (tokens * hq > INT32_MAX)
            return SHKV_ERR_UNSUPPORTED;
    }
    if (tokens == 0)
        return SHKV_OK;
    return attention(pool, p, hq, q, q_stride, scale, out, lse_out, workspace, workspace_bytes, stream);
} catch (const std::exception &) {
    return SHKV_ERR_CUDA;                // no host memory for the plan
}

shkv_status shkv_q8_check_errors(shkv_q8_pool *pool, void *stream, uint32_t *flags)
{
    if (!pool || !flags || !on_pool_device(pool))
        return SHKV_ERR_INVALID_ARG;
    *flags = 0;
    cudaStream_t st = (cudaStream_t)stream;
    if (capturing(st))
        return SHKV_ERR_INVALID_ARG;
    uint32_t v = 0;
    if (cudaMemcpyAsync(&v, pool->cfg.error_word, sizeof v, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return SHKV_ERR_CUDA;
    // only what is reported is cleared, and before the call returns: a bit that
    // a kernel of another stream sets in the meantime stays for the next check
    if (v && (launch_q8_clear_errors(pool->cfg.error_word, v, st) != cudaSuccess ||
              cudaStreamSynchronize(st) != cudaSuccess))
        return SHKV_ERR_CUDA;
    *flags = v;
    return v ? SHKV_ERR_DEVICE : SHKV_OK;
}

}  // extern "C"
