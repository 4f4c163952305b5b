// evict_host.cu -- the C ABI of eviction by accumulated attention weight:
// argument checks and kernel launches.  Declarations and their contracts are in
// include/shkv.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <exception>

#include "evict.cuh"
#include "host_shared.h"
#include "shkv.h"

namespace shkv {
cudaError_t launch_mass(const CUtensorMap &tm_k, const CUtensorMap &tm_q, const MassParams &p, bool pieces,
                        cudaStream_t stream);
cudaError_t launch_select(const SelectParams &p, int num_sms, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams &p, cudaStream_t stream);
}  // namespace shkv

using namespace shkv;

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// A pool, a batch that it takes, and its device current.
bool callable(const shkv_pool *pool, int32_t batch)
{
    int dev = -1;
    return pool && batch >= 0 && batch <= pool->cfg.max_batch && batch <= SHKV_MAX_BATCH &&
           cudaGetDevice(&dev) == cudaSuccess && dev == pool->device;
}

bool capturing(void *stream)
{
    cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing((cudaStream_t)stream, &s) == cudaSuccess)
        return s == cudaStreamCaptureStatusActive;
    cudaGetLastError();                  // the default stream beside a capture: no error of this call's
    return false;
}

int64_t longest(int32_t batch, const int32_t *lens)
{
    int64_t n = 0;
    for (int b = 0; b < batch; ++b)
        n = std::max<int64_t>(n, lens[b]);
    return n;
}

constexpr int32_t kMaxTokens = 1 << 30;   // of a request: the kernels step past its end in 32 bits

// Masses of up to `len` tokens that a call reads; of none they may be anywhere.
bool readable(const shkv_mass *m, int64_t len)
{
    return m && (len == 0 || (m->data && aligned(m->data, 4))) && m->request_stride >= 0 && m->head_stride >= 0 &&
           m->length >= len;
}

// Masses that a call writes: the rows of `len` must not overlap, whichever of
// requests and heads lies outside.
bool writable(const shkv_mass *m, int32_t batch, int32_t hkv, int64_t len)
{
    if (!readable(m, len))
        return false;
    const int64_t r = m->request_stride, h = m->head_stride;
    if (batch == 1 || hkv == 1)
        return batch * hkv == 1 || (batch == 1 ? h : r) >= len;
    return (h >= len && r >= h * (hkv - 1) + len) || (r >= len && h >= r * (batch - 1) + len);
}

// The same masses have the same strides (those that are used).
bool same_layout(const shkv_mass *a, const shkv_mass *b, int32_t batch, int32_t hkv)
{
    return a->data != b->data || ((batch == 1 || a->request_stride == b->request_stride) &&
                                  (hkv == 1 || a->head_stride == b->head_stride));
}

Span mass_span(const float *data, int64_t request_stride, int64_t head_stride, int32_t batch, int32_t hkv, int64_t len)
{
    return span_of(data, (size_t)((batch - 1) * request_stride + (hkv - 1) * head_stride + len) * 4);
}

// Rows of a call: dim0 = head_dim, dim1 = heads, dim2 = query tokens of a
// request, dim3 = requests.  A box {64, G, tpt, 1} is a column half of a block's
// rows of one KV head, 128-byte swizzled; query tokens behind a request's last
// are zeros.
bool make_q_map(CUtensorMap *tm, const void *q, const shkv_pool_config &c, int32_t batch, int32_t n_q, int32_t hq,
                int64_t q_request, int64_t q_token, int32_t tpt)
{
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc)
        return false;
    cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)hq, (cuuint64_t)n_q, (cuuint64_t)batch};
    cuuint64_t strides[3] = {(cuuint64_t)c.head_dim * 2, (cuuint64_t)q_token * 2, (cuuint64_t)q_request * 2};
    cuuint32_t box[4] = {64u, (cuuint32_t)(hq / c.num_kv_heads), (cuuint32_t)tpt, 1u};
    cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Bytes of the cut items' sums.
size_t piece_bytes(const shkv_pool *pool)
{
    return (size_t)2 * std::min(pool->num_sms, kMassMaxCtas) * kWide * sizeof(float);
}

// Cuts the items into at most `limit` ranges of about equal cost, counted in
// products of a tile and a block of rows (0.3 us); an item costs kItemCost more (its
// K's copy, the join of its threads' sums).  A compromise: at 1 and 4 a document takes
// 2 and 1% more; at 12 and 16 it takes 1 and 2% less (573, 566, 560 us at 8, 12, 16),
// as do a few requests of 8K (29.2, 28.0, 27.4), but chunks without much before them
// up to 6% more (283 tokens 11.6, 12.3, 12.3; 1889 tokens 16.0, 16.5, 16.6); ten drawn
// chunks are the same in the mean.  An item of many
// blocks may be cut between two of them, but not into pieces of under kMinPiece
// blocks.  (Leaving items whole where a cut seemed dearer than the second kernel
// gained nothing: 24.2 us.)  True if an item is cut.
constexpr int64_t kItemCost = 8, kMinPiece = 2;

bool plan_mass(MassParams &p, int limit)
{
    const int tokens = p.item_tokens;
    // cost of item `at` of a request's head, and of all of the head's
    auto cost = [&](int L, int at) -> int64_t {
        const int past = mass_past(L, p.n_q, p.causal);
        int64_t k = kItemCost;
        for (int t = at * tokens; t < std::min(L, (at + 1) * tokens); t += kMassTile)
            k += p.blocks - mass_block0(t, past, p.tpt);
        return k;
    };
    // the first `even` items take part in every block
    auto even = [&](int L) -> int64_t { return std::max(0, std::min(L, mass_past(L, p.n_q, p.causal)) / tokens); };
    const int64_t full = kItemCost + (int64_t)(tokens / kMassTile) * p.blocks;
    auto head = [&](int L) -> int64_t {
        int64_t k = even(L) * full;
        for (int at = (int)even(L); at * tokens < L; ++at)
            k += cost(L, at);
        return k;
    };
    int64_t total = 0;
    for (int b = 0; b < p.batch; ++b)
        total += p.hkv * head(p.lens[b]);
    const int64_t C = std::max<int64_t>(
        1, std::min<int64_t>(limit, mass_wide(p.blocks) ? total / (2 * kMinPiece) : p.item0[p.batch]));
    int n = 0, b = 0;
    int64_t before = 0, h = head(p.lens[0]);
    bool cut = false;
    p.cut_item[0] = p.cut_block[0] = 0;
    for (int64_t c = 1; c < C; ++c) {
        const int64_t target = total * c / C;
        while (h == 0 || target >= before + p.hkv * h) {
            before += p.hkv * h;
            h = head(p.lens[++b]);
        }
        const int L = p.lens[b], g = (int)((target - before) / h);
        int64_t rest = (target - before) % h;
        int at = (int)std::min(rest / full, even(L));
        rest -= at * full;
        int64_t k = cost(L, at);
        while (rest >= k) {
            rest -= k;
            k = cost(L, ++at);
        }
        int item = p.item0[b] + g * ((L + tokens - 1) / tokens) + at;
        const int block0 = mass_block0(at * tokens, mass_past(L, p.n_q, p.causal), p.tpt);
        const int64_t steps = p.blocks - block0, done = steps * rest / k;
        int block = 0;
        if (steps >= 2 * kMinPiece && done >= kMinPiece && steps - done >= kMinPiece)
            block = block0 + (int)done;
        else if (2 * done >= steps)
            ++item;
        if (item > p.cut_item[n] || (item == p.cut_item[n] && block > p.cut_block[n])) {
            if (item >= p.item0[p.batch])
                break;
            ++n;
            p.cut_item[n] = item;
            p.cut_block[n] = block;
            cut = cut || block > 0;
        }
    }
    p.num_ctas = n + 1;
    p.cut_item[n + 1] = p.item0[p.batch];
    p.cut_block[n + 1] = 0;
    return cut;
}

// Both forms: the n_q query tokens of every request.
shkv_status add_mass(shkv_pool *pool, int32_t batch, int32_t n_q, int32_t hq, const void *q, int64_t q_request,
                     int64_t q_token, float scale, const float *lse, int64_t lse_request, int64_t lse_token,
                     float decay, const shkv_mass *mass, const shkv_mass *out, bool causal, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    const shkv_pool_config &c = pool->cfg;
    const int64_t row = (int64_t)hq * c.head_dim;
    if (n_q == 1)                        // a stride that no step is taken along: one that divides the requests'
        q_token = c.head_dim, lse_token = 0;
    if (q_token >= (int64_t)1 << 39)     // a tensor map's strides are below 2^40 bytes
        return SHKV_ERR_UNSUPPORTED;
    if (batch == 1)
        q_request = n_q * q_token, lse_request = 0;
    const float scale_log2 = (float)((double)scale * 1.4426950408889634);
    const int64_t len = longest(batch, pool->lens.data());
    if (!q || !aligned(q, 16) || !lse || !aligned(lse, 4) || (n_q > 1 && q_token < row) || q_token % c.head_dim ||
        q_request <= 0 || q_request % q_token || lse_request < 0 || lse_token < 0 || !isfinite(scale_log2) ||
        !isfinite(decay) || !writable(out, batch, c.num_kv_heads, len) ||
        (mass && (!readable(mass, len) || (len > 0 && !same_layout(mass, out, batch, c.num_kv_heads)))))
        return SHKV_ERR_INVALID_ARG;
    if (q_request >= (int64_t)1 << 39 || len > kMaxTokens)
        return SHKV_ERR_UNSUPPORTED;
    MassParams p;
    memset(&p, 0, sizeof p);
    p.group = hq / c.num_kv_heads;
    p.tpt = std::min(kMassRows / p.group, n_q);
    p.blocks = (n_q + p.tpt - 1) / p.tpt;
    const int ctas = std::min(pool->num_sms, kMassMaxCtas);
    p.item_tokens = mass_wide(p.blocks) ? kWide : kMassTile;
    int64_t items = 0;
    for (int b = 0; b < batch; ++b) {
        p.lens[b] = pool->lens[b];
        p.item0[b] = (int32_t)items;
        items += ((int64_t)pool->lens[b] + p.item_tokens - 1) / p.item_tokens * c.num_kv_heads;
        if (items > INT32_MAX)
            return SHKV_ERR_UNSUPPORTED;
    }
    p.item0[batch] = (int32_t)items;     // 0: one CTA that looks at the lengths
    p.lse = lse;
    p.lse_request = lse_request;
    p.lse_token = lse_token;
    if (mass && decay != 0.f) {
        p.mass.in = mass->data;
        p.mass.in_request = mass->request_stride;
        p.mass.in_head = mass->head_stride;
    }
    p.mass.out = out->data;
    p.mass.out_request = out->request_stride;
    p.mass.out_head = out->head_stride;
    p.block_table = c.block_table;
    p.seq_lens = c.seq_lens;
    p.err = c.error_word;
    p.pieces = static_cast<float *>(workspace);
    p.batch = batch;
    p.n_q = n_q;
    p.hkv = c.num_kv_heads;
    p.head_dim = c.head_dim;
    p.page_size = c.page_size;
    p.max_pages = c.max_pages_per_seq;
    p.num_pages = c.num_pages;
    p.causal = causal;
    p.scale_log2 = scale_log2;
    p.decay = decay;
    CUtensorMap tm_q;
    if (!make_q_map(&tm_q, q, c, batch, n_q, hq, q_request, q_token, p.tpt))
        return SHKV_ERR_CUDA;
    const bool pieces = plan_mass(p, ctas);
    if (launch_mass(pool->tm_k2, tm_q, p, pieces, (cudaStream_t)stream) != cudaSuccess)
        return SHKV_ERR_CUDA;
    record_stream_use(stream,
                      {span_of(q, (size_t)((batch - 1) * q_request + (n_q - 1) * q_token + row) * 2),
                       span_of(lse, (size_t)((batch - 1) * lse_request + (n_q - 1) * lse_token + hq) * 4),
                       span_of(workspace, workspace_bytes),
                       mass_span(p.mass.in, p.mass.in_request, p.mass.in_head, batch, c.num_kv_heads, len),
                       mass_span(p.mass.out, p.mass.out_request, p.mass.out_head, batch, c.num_kv_heads, len)});
    return SHKV_OK;
}

}  // namespace

extern "C" {

shkv_status shkv_prefill_mass_workspace_size(const shkv_pool *pool, size_t *bytes)
{
    if (!pool || !bytes)
        return SHKV_ERR_INVALID_ARG;
    *bytes = piece_bytes(pool);
    return SHKV_OK;
}

shkv_status shkv_decode_mass(shkv_pool *pool, int32_t batch, int32_t n_models, int32_t hq_per_model, const void *q,
                             float scale, const float *lse, float decay, const shkv_mass *mass, const shkv_mass *out,
                             void *stream)
try {
    if (!callable(pool, batch) || batch < 1 || n_models < 1 || hq_per_model < 1)
        return SHKV_ERR_INVALID_ARG;
    const int32_t hkv = pool->cfg.num_kv_heads;
    if (hq_per_model % hkv || (int64_t)n_models * (hq_per_model / hkv) > 64)
        return SHKV_ERR_UNSUPPORTED;
    const int64_t row = (int64_t)hq_per_model * pool->cfg.head_dim;
    return add_mass(pool, batch, n_models, hq_per_model, q, n_models * row, row, scale, lse,
                    (int64_t)n_models * hq_per_model, hq_per_model, decay, mass, out, false, nullptr, 0, stream);
} catch (const std::exception &) {
    return SHKV_ERR_CUDA;                // no host memory
}

shkv_status shkv_prefill_mass(shkv_pool *pool, int32_t batch, int32_t n_new, int32_t hq_per_model, const void *q,
                              int64_t q_request_stride, int64_t q_token_stride, float scale, const float *lse,
                              int64_t lse_request_stride, int64_t lse_token_stride, float decay,
                              const shkv_mass *mass, const shkv_mass *out, void *workspace, size_t workspace_bytes,
                              void *stream)
try {
    if (!callable(pool, batch) || batch < 1 || n_new < 1 || hq_per_model < 1 || !workspace ||
        !aligned(workspace, 16) || workspace_bytes < piece_bytes(pool))
        return SHKV_ERR_INVALID_ARG;
    const int32_t hkv = pool->cfg.num_kv_heads;
    if (hq_per_model % hkv || hq_per_model / hkv > 128)
        return SHKV_ERR_UNSUPPORTED;
    for (int b = 0; b < batch; ++b)
        if (pool->lens[b] < n_new)
            return SHKV_ERR_INVALID_ARG;     // the new tokens must already be in the pool
    return add_mass(pool, batch, n_new, hq_per_model, q, q_request_stride, q_token_stride, scale, lse,
                    lse_request_stride, lse_token_stride, decay, mass, out, true, workspace, workspace_bytes, stream);
} catch (const std::exception &) {
    return SHKV_ERR_CUDA;                // no host memory
}

shkv_status shkv_select_tokens(shkv_pool *pool, int32_t batch, const shkv_mass *mass, const int32_t *keep,
                               int32_t sink, int32_t recent, int32_t *index, int64_t index_stride, void *stream)
try {
    if (!callable(pool, batch) || !keep || sink < 0 || recent < 0)
        return SHKV_ERR_INVALID_ARG;
    if (batch == 0)
        return SHKV_OK;
    const int64_t len = longest(batch, pool->lens.data());
    if (!readable(mass, len) || !index || !aligned(index, 4) || index_stride < 1)
        return SHKV_ERR_INVALID_ARG;
    const int32_t hkv = pool->cfg.num_kv_heads;
    SelectParams p;
    memset(&p, 0, sizeof p);
    for (int b = 0; b < batch; ++b) {
        const int32_t L = pool->lens[b];
        if (keep[b] < 0 || std::min(keep[b], L) > index_stride ||
            (keep[b] < L && (int64_t)sink + recent > keep[b]))
            return SHKV_ERR_INVALID_ARG;
        p.lens[b] = L;
        p.keep[b] = keep[b];
    }
    if ((int64_t)batch * hkv * 8 > INT32_MAX || len > kMaxTokens)
        return SHKV_ERR_UNSUPPORTED;
    p.mass = mass->data;
    p.mass_request = mass->request_stride;
    p.mass_head = mass->head_stride;
    p.index = index;
    p.index_stride = index_stride;
    p.seq_lens = pool->cfg.seq_lens;
    p.err = pool->cfg.error_word;
    p.batch = batch;
    p.hkv = hkv;
    p.sink = sink;
    p.recent = recent;
    if (launch_select(p, pool->num_sms, (cudaStream_t)stream) != cudaSuccess)
        return SHKV_ERR_CUDA;
    record_stream_use(stream, {mass_span(p.mass, p.mass_request, p.mass_head, batch, hkv, len),
                               span_of(index, (size_t)batch * hkv * index_stride * 4)});
    return SHKV_OK;
} catch (const std::exception &) {
    return SHKV_ERR_CUDA;                // no host memory
}

shkv_status shkv_select_width(const shkv_pool *pool, int32_t batch, const int32_t *keep, int32_t *width)
{
    if (!pool || !width || batch < 0 || batch > pool->cfg.max_batch || (batch > 0 && !keep))
        return SHKV_ERR_INVALID_ARG;
    *width = 0;
    for (int b = 0; b < batch; ++b)
        *width = std::max(*width, std::min(keep[b], pool->lens[b]));
    return SHKV_OK;
}

shkv_status shkv_evict_tokens(shkv_pool *pool, int32_t batch, const int32_t *keep, const int32_t *index,
                              int64_t index_stride, const int32_t *new_table, int64_t new_table_stride,
                              const int32_t *table, int64_t table_stride, const int32_t *lens, const shkv_mass *mass,
                              const shkv_mass *out, void *stream)
try {
    if (!callable(pool, batch) || !keep || !table != !lens || !mass != !out)
        return SHKV_ERR_INVALID_ARG;
    const shkv_pool_config &c = pool->cfg;
    EvictParams p;
    memset(&p, 0, sizeof p);
    int64_t pages = 0, len = 0;
    bool moves = false;
    if (!table)
        table_stride = c.max_pages_per_seq;
    for (int b = 0; b < batch; ++b) {
        const int32_t L = lens ? lens[b] : pool->lens[b];
        if (keep[b] < 0 || L < 0 || (int64_t)L > table_stride * c.page_size)
            return SHKV_ERR_INVALID_ARG;
        p.lens[b] = L;
        p.keep[b] = keep[b];
        p.page0[b] = (int32_t)pages;
        if (keep[b] >= L)
            continue;
        moves = true;
        len = std::max<int64_t>(len, L);
        const int64_t n = ((int64_t)keep[b] + c.page_size - 1) / c.page_size;
        if (n > c.max_pages_per_seq)
            return SHKV_ERR_CAPACITY;
        if (n > new_table_stride || keep[b] > index_stride)
            return SHKV_ERR_INVALID_ARG;
        pages += n;
    }
    p.page0[batch] = (int32_t)pages;     // at most SHKV_MAX_BATCH * max_pages_per_seq; checked below
    p.block_table = c.block_table;
    p.seq_lens = c.seq_lens;
    p.err = c.error_word;
    p.batch = batch;
    p.hkv = c.num_kv_heads;
    p.head_dim = c.head_dim;
    p.page_size = c.page_size;
    p.max_pages = c.max_pages_per_seq;
    p.num_pages = c.num_pages;
    p.check_lens = !lens;
    if (!moves) {
        // nothing to launch, but a replay has to find out about lengths that it was not captured with
        if (batch == 0 || lens || !capturing(stream))
            return SHKV_OK;
        return launch_evict(p, (cudaStream_t)stream) == cudaSuccess ? SHKV_OK : SHKV_ERR_CUDA;
    }
    // the pool's table is written from new_table: no byte of one may be the other's
    const Span own = span_of(c.block_table, (size_t)c.max_batch * c.max_pages_per_seq * 4);
    const Span given = span_of(new_table, (size_t)batch * new_table_stride * 4);
    if (!new_table || !aligned(new_table, 4) || (given.lo < own.hi && own.lo < given.hi) ||
        (pages > 0 && (!index || !aligned(index, 4))))
        return SHKV_ERR_INVALID_ARG;
    if (table && !aligned(table, 4))
        return SHKV_ERR_INVALID_ARG;
    if (out && (!readable(mass, len) || !writable(out, batch, c.num_kv_heads, len) ||
                !same_layout(mass, out, batch, c.num_kv_heads)))
        return SHKV_ERR_INVALID_ARG;
    if ((pages + batch) * c.num_kv_heads > INT32_MAX - 64 - batch || len > kMaxTokens)   // warps, whole CTAs of them
        return SHKV_ERR_UNSUPPORTED;
    p.k_pages = static_cast<uint4 *>(c.k_pages);
    p.v_pages = static_cast<uint4 *>(c.v_pages);
    p.index = index;
    p.index_stride = index_stride;
    p.new_table = new_table;
    p.new_stride = new_table_stride;
    p.table = table ? table : c.block_table;
    p.table_stride = table_stride;
    if (out) {
        p.mass.in = mass->data;
        p.mass.in_request = mass->request_stride;
        p.mass.in_head = mass->head_stride;
        p.mass.out = out->data;
        p.mass.out_request = out->request_stride;
        p.mass.out_head = out->head_stride;
    }
    // a source of the caller's that is no part of the pool's own table
    const Span source = span_of(table, (size_t)batch * table_stride * 4);
    p.at_once = table && (source.hi <= own.lo || own.hi <= source.lo);
    if (launch_evict(p, (cudaStream_t)stream) != cudaSuccess)
        return SHKV_ERR_CUDA;
    for (int b = 0; b < batch; ++b)
        if (p.keep[b] < p.lens[b])
            pool->lens[b] = p.keep[b];
    // the pool's table has changed: a decode with tails right behind this call
    // has to wait for it, as it does where no byte is free
    record_stream_use(stream, {Span{0, UINTPTR_MAX}});
    return SHKV_OK;
} catch (const std::exception &) {
    return SHKV_ERR_CUDA;                // no host memory
}

}  // extern "C"
