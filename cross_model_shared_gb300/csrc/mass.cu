// mass.cu -- the attention weight that every cached token of a KV head gets
// from the rows of a decode step or of a causal chunk, added to its mass
// (tcgen05, sm_103a).
//
//   mass'[t] = decay * mass[t] + sum_r exp2(c <q_r, k_t> - l_r),
//
// c = scale * log2(e), l_r = lse_r * log2(e).  The rows' log-sum-exps are given,
// so there is no running maximum and nothing to rescale: a weight is final as
// soon as its score is there.
//
// Tokens lie on the MMA's M dimension, S[t, r] = K Q^T with M = 128 tokens and
// N = up to 128 rows in a TMEM buffer, so that a thread owns a token (its TMEM
// lane) and adds up its row of weights in a register, without a word between
// threads: no atomics, the same bits every time.  K is read once per call; the
// rows of a decode step stay in shared memory while a CTA walks along the tokens
// of a head, those of a chunk stream past the two K tiles of an item (a Q block
// of 32 KB feeds two MMAs of 128 x 128 x D).
//
// Warps 0-3 and 4-7 take the weights of the item's first and second tile, each
// with two S buffers; warp 8 copies K, warp 9 Q (and the log-sum-exps), one lane
// of warp 10 issues the MMAs.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "evict.cuh"
#include "launch.cuh"
#include "q8_wait.cuh"
#include "shkv_device.cuh"

namespace shkv {

namespace {

constexpr int kThreads = 352;
constexpr int kKWarp = 8, kQWarp = 9, kMmaWarp = 10;
constexpr uint32_t kTmemCols = 512;          // S[tile][buffer], 128 columns each
constexpr uint32_t kHalfBytes = 128u * 128u; // 64 columns of 128 tokens or rows

// Ring slots: at D = 128 seven of 32 KB fill shared memory (K four, a decode's
// 128 KB in flight).
template <int D>
struct Ring {
    static constexpr int kK = D == 128 ? 4 : 8, kQ = D == 128 ? 3 : 5;
    static constexpr uint32_t kSlot = (uint32_t)(D / 64) * kHalfBytes;
    // barriers: K full, K empty, Q full, Q empty, S full [tile][buffer], S empty, fin
    static constexpr int kBars = 2 * kK + 2 * kQ + 9;
    static constexpr uint32_t kQ0 = kK * kSlot, kLse = kQ0 + kQ * kSlot, kBar0 = kLse + kQ * kMassRows * 4,
                              kMisc = kBar0 + 8 * kBars, kBytes = kMisc + 16 + 1024;
};
static_assert(Ring<128>::kBytes <= kSmemLimit && Ring<64>::kBytes <= kSmemLimit, "shared memory");

template <int D>
struct Ctx {
    uint8_t *smem;
    uint32_t base;
    volatile uint32_t *abort_flag;
    uint32_t *err;
    __device__ uint32_t bar(int i) const { return base + Ring<D>::kBar0 + 8u * (uint32_t)i; }
    __device__ uint32_t k_full(int s) const { return bar(s); }
    __device__ uint32_t k_empty(int s) const { return bar(Ring<D>::kK + s); }
    __device__ uint32_t q_full(int s) const { return bar(2 * Ring<D>::kK + s); }
    __device__ uint32_t q_empty(int s) const { return bar(2 * Ring<D>::kK + Ring<D>::kQ + s); }
    __device__ uint32_t s_full(int x, int i) const { return bar(2 * Ring<D>::kK + 2 * Ring<D>::kQ + 2 * x + i); }
    __device__ uint32_t s_empty(int x, int i) const { return s_full(x, i) + 32u; }
    __device__ uint32_t fin() const { return s_full(0, 0) + 64u; }
    __device__ uint32_t k_slot(int s) const { return base + (uint32_t)s * Ring<D>::kSlot; }
    __device__ uint32_t q_slot(int s) const { return base + Ring<D>::kQ0 + (uint32_t)s * Ring<D>::kSlot; }
    __device__ float *lse(int s) const { return reinterpret_cast<float *>(smem + Ring<D>::kLse) + s * kMassRows; }
    __device__ bool wait(uint32_t b, uint32_t parity) const { return q8_wait<true>(b, parity, abort_flag, err); }
};

// Position in a ring of n slots.
struct Turn {
    int slot = 0;
    uint32_t parity = 0;
    __device__ void next(int n)
    {
        if (++slot == n) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// The items of a CTA's range, one after another; every role walks them alike.
struct Walk {
    int item, last, b, g, pair, pairs;   // `last`: one past the range's last item
    int L, past, t0;
    int begin, end;                      // blocks of this item in the range
    int block0[2];                       // first block that a tile takes part in; beyond all if it is empty
    bool fresh;                          // another (request, KV head) than the item before
};

__device__ __forceinline__ void walk_request(const MassParams &p, Walk &w)
{
    w.L = p.lens[w.b];
    w.past = mass_past(w.L, p.n_q, p.causal);
    w.pairs = (w.L + kMassItem - 1) / kMassItem;
}

__device__ __forceinline__ void walk_item(const MassParams &p, Walk &w)
{
    w.t0 = w.pair * kMassItem;
    w.block0[0] = mass_block0(w.t0, w.past, p.tpt);
    w.block0[1] = w.t0 + kMassTile < w.L ? mass_block0(w.t0 + kMassTile, w.past, p.tpt) : INT32_MAX;
    w.begin = w.block0[0];
    if (w.item == p.cut_item[blockIdx.x])
        w.begin = max(w.begin, p.cut_block[blockIdx.x]);
    w.end = w.item == p.cut_item[blockIdx.x + 1] ? p.cut_block[blockIdx.x + 1] : p.blocks;
}

// Whether the CTA has an item at all.
__device__ __forceinline__ bool walk_first(const MassParams &p, Walk &w)
{
    w.item = p.cut_item[blockIdx.x];
    w.last = p.cut_item[blockIdx.x + 1] + (p.cut_block[blockIdx.x + 1] > 0);
    if (w.item >= w.last)
        return false;
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.item0[mid] <= w.item)
            lo = mid;
        else
            hi = mid;
    }
    w.b = lo;
    walk_request(p, w);
    w.g = (w.item - p.item0[lo]) / w.pairs;
    w.pair = (w.item - p.item0[lo]) % w.pairs;
    w.fresh = true;
    walk_item(p, w);
    return true;
}

__device__ __forceinline__ bool walk_next(const MassParams &p, Walk &w)
{
    if (++w.item >= w.last)
        return false;
    w.fresh = false;
    if (++w.pair == w.pairs) {
        w.pair = 0;
        w.fresh = true;
        if (++w.g == p.hkv) {
            w.g = 0;
            do
                ++w.b;
            while (p.lens[w.b] == 0);
            walk_request(p, w);
        }
    }
    walk_item(p, w);
    return true;
}

// A block of rows is copied again for every item, unless it is a head's only one.
__device__ __forceinline__ bool new_rows(const MassParams &p, const Walk &w) { return p.blocks > 1 || w.fresh; }

// K tiles: a lane per (column half, page) of a tile.  A page outside the pool
// is left out and flagged; the tile's threads look at their table entries
// themselves.
template <int D>
__device__ void copy_k(const CUtensorMap *tm, const MassParams &p, const Ctx<D> &c)
{
    const int lane = threadIdx.x & 31, P = p.page_size, RB = kMassTile / P;
    const int half = lane / RB, rb = lane % RB;
    const bool copier = half < D / 64;
    const uint64_t pol = l2_evict_first_policy();
    Walk w;
    Turn turn;
    bool alive = true;
    int issued = 0;
    if (!walk_first(p, w))
        return;
    do {
        const int32_t *row = p.block_table + (int64_t)w.b * p.max_pages;
        if (lane == 0 && w.fresh && w.pair == 0 && w.g == 0 && __ldg(p.seq_lens + w.b) != w.L)
            atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
        const int pages = (w.L + P - 1) / P;
        int id[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int pg = (w.t0 + x * kMassTile) / P + rb;
            id[x] = copier && pg < pages ? __ldg(row + pg) : -1;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int pg = (w.t0 + x * kMassTile) / P + rb;
            if (w.t0 + x * kMassTile >= w.L)
                break;
            bool ok = true;
            if (alive && lane == 0)
                ok = c.wait(c.k_empty(turn.slot), turn.parity ^ 1u);
            alive = alive && __all_sync(0xffffffffu, ok);
            const bool inside = copier && (uint32_t)id[x] < (uint32_t)p.num_pages;
            if (copier && pg < pages && !inside)
                atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
            const uint32_t mask = __ballot_sync(0xffffffffu, inside);
            if (alive && lane == 0)
                mbar_arrive_expect_tx(c.k_full(turn.slot), (uint32_t)__popc(mask) * (uint32_t)P * 128u);
            __syncwarp();
            if (alive && inside)
                tma_load_2d(c.k_slot(turn.slot) + (uint32_t)half * kHalfBytes + (uint32_t)(rb * P) * 128u, tm, half * 64,
                            (id[x] * p.hkv + w.g) * P, c.k_full(turn.slot), pol);
            if (alive) {
                ++issued;
                turn.next(Ring<D>::kK);
            }
        }
    } while (walk_next(p, w));
    if (!alive && lane == 0)                 // wait for the copies in flight
        for (int i = max(0, issued - Ring<D>::kK); i < issued; ++i)
            mbar_drain_bounded(c.k_full(i % Ring<D>::kK), (uint32_t)(i / Ring<D>::kK) & 1u);
}

// Q blocks and what their rows' log-sum-exps take off the scores; a row beyond
// the block's, or one that attends nothing, gets -inf and so weighs nothing.
template <int D>
__device__ void copy_q(const CUtensorMap *tm, const MassParams &p, const Ctx<D> &c)
{
    const int lane = threadIdx.x & 31;
    const uint32_t bytes = (uint32_t)(p.tpt * p.group * D * 2);
    Walk w;
    Turn turn;
    bool alive = true;
    int issued = 0;
    if (!walk_first(p, w))
        return;
    do {
        if (!new_rows(p, w))
            continue;
        for (int k = w.begin; k < w.end; ++k) {
            const int i0 = k * p.tpt, rows = min(p.tpt, p.n_q - i0) * p.group;
            const float *src = p.lse + w.b * p.lse_request + w.g * p.group;
            float off[kMassRows / 32];
#pragma unroll
            for (int j = 0; j < kMassRows / 32; ++j) {
                const int r = lane + 32 * j;
                off[j] = INFINITY;
                if (r < rows)
                    off[j] = lse_base2(__ldg(src + (i0 + r / p.group) * p.lse_token + r % p.group));
            }
            bool ok = true;
            if (alive && lane == 0)
                ok = c.wait(c.q_empty(turn.slot), turn.parity ^ 1u);
            alive = alive && __all_sync(0xffffffffu, ok);
            if (!alive)
                continue;
#pragma unroll
            for (int j = 0; j < kMassRows / 32; ++j)
                c.lse(turn.slot)[lane + 32 * j] = -off[j];
            __syncwarp();
            if (lane == 0)
                mbar_arrive_expect_tx(c.q_full(turn.slot), bytes);
            __syncwarp();
            if (lane < D / 64)
                asm volatile(
                    "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                    " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(c.q_slot(turn.slot) + (uint32_t)lane * kHalfBytes),
                    "l"(reinterpret_cast<uint64_t>(tm)), "r"(lane * 64), "r"(w.g * p.group), "r"(i0), "r"(w.b),
                    "r"(c.q_full(turn.slot))
                    : "memory");
            ++issued;
            turn.next(Ring<D>::kQ);
        }
    } while (walk_next(p, w));
    if (!alive && lane == 0)
        for (int i = max(0, issued - Ring<D>::kQ); i < issued; ++i)
            mbar_drain_bounded(c.q_full(i % Ring<D>::kQ), (uint32_t)(i / Ring<D>::kQ) & 1u);
}

// S = K Q^T for every (block, tile) of the range.  A slot of K is free after the
// item's last block, one of Q when the next block's rows are needed.
template <int D>
__device__ void issue(const MassParams &p, const Ctx<D> &c, uint32_t tmem)
{
    const uint64_t kd0 = umma_sdesc_sw128(c.k_slot(0), 16u, 1024u), qd0 = umma_sdesc_sw128(c.q_slot(0), 16u, 1024u);
    Walk w;
    Turn kt, qt, st[2];
    bool alive = true, rows_in = false;
    if (!walk_first(p, w))
        return;
    do {
        bool k_in[2] = {false, false};
        int kslot[2];
        uint32_t kpar[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            kslot[x] = kt.slot;
            kpar[x] = kt.parity;
            if (w.block0[x] < INT32_MAX)
                kt.next(Ring<D>::kK);
        }
        for (int k = w.begin; k < w.end; ++k) {
            if (new_rows(p, w)) {
                if (rows_in) {
                    umma_commit(c.q_empty(qt.slot));
                    qt.next(Ring<D>::kQ);
                }
                rows_in = true;
                if (alive)
                    alive = c.wait(c.q_full(qt.slot), qt.parity);
            }
            const int rows = min(p.tpt, p.n_q - k * p.tpt) * p.group;
            const uint32_t idesc = umma_idesc_bf16(kMassTile, (rows + 15) & ~15, false, false);
            const uint64_t qd = qd0 + (((uint32_t)qt.slot * Ring<D>::kSlot) >> 4);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (k < w.block0[x])
                    continue;
                if (alive && !k_in[x])
                    alive = c.wait(c.k_full(kslot[x]), kpar[x]);
                k_in[x] = true;
                if (alive)
                    alive = c.wait(c.s_empty(x, st[x].slot), st[x].parity ^ 1u);
                if (alive) {
                    tc_fence_after();
                    const uint64_t kd = kd0 + (((uint32_t)kslot[x] * Ring<D>::kSlot) >> 4);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t off = ((uint32_t)(i >> 2) * kHalfBytes + (uint32_t)(i & 3) * 32u) >> 4;
                        umma_bf16(tmem + (uint32_t)(2 * x + st[x].slot) * 128u, kd + off, qd + off, idesc, i ? 1u : 0u);
                    }
                }
                umma_commit(c.s_full(x, st[x].slot));
                st[x].next(2);
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (w.block0[x] < INT32_MAX) {
                if (alive && !k_in[x])       // a range that ends before the tile's first block
                    alive = c.wait(c.k_full(kslot[x]), kpar[x]);
                umma_commit(c.k_empty(kslot[x]));
            }
    } while (walk_next(p, w));
    umma_commit(c.fin());
    mbar_drain_bounded(c.fin(), 0u);
}

// Waits for the columns of S that were asked for.
__device__ __forceinline__ void landed(uint32_t (&r)[64])
{
    // the operands keep the compiler from using a register before the wait
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 64; i += 16)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                     "+r"(r[i + 6]), "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]),
                     "+r"(r[i + 12]), "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15]));
}

// The weights of columns c0 .. c0 + 15 into four partial sums, two values an
// instruction where there is one for it.
template <bool kMasked>
__device__ __forceinline__ void weigh16(const uint32_t *s, const float *lse, int c0, int rows, int first, float c,
                                        float2 (&sum)[2])
{
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(lse + c0 + j);
        float2 x0 = __ffma2_rn(make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), make_float2(c, c),
                               make_float2(l.x, l.y));
        float2 x1 = __ffma2_rn(make_float2(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3])), make_float2(c, c),
                               make_float2(l.z, l.w));
        if (kMasked) {
            const int i = c0 + j;
            x0.x = i >= first && i < rows ? x0.x : -INFINITY;
            x0.y = i + 1 >= first && i + 1 < rows ? x0.y : -INFINITY;
            x1.x = i + 2 >= first && i + 2 < rows ? x1.x : -INFINITY;
            x1.y = i + 3 >= first && i + 3 < rows ? x1.y : -INFINITY;
        }
        sum[0] = __fadd2_rn(sum[0], make_float2(ex2_approx(x0.x), ex2_approx(x0.y)));
        sum[1] = __fadd2_rn(sum[1], make_float2(ex2_approx(x1.x), ex2_approx(x1.y)));
    }
}

// Sum of a thread's weights over the columns [first, rows) of S at taddr.  The
// columns that the MMA rounds rows up to are zero queries, whose product with an
// infinite key is no number; `latest` is the warp's largest `first`.  S is in
// registers half a buffer at a time; `empty` is arrived on as soon as all of it
// is, so that the next product into the buffer runs beside the exponentials.
__device__ __forceinline__ float weigh(uint32_t taddr, const float *lse, int rows, int first, int latest, float c,
                                       uint32_t empty)
{
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint32_t s[2][64];
    tmem_ld32_nowait(taddr, s[0]);
    if (rows > 32)
        tmem_ld32_nowait(taddr + 32u, s[0] + 32);
    landed(s[0]);
    if (rows > 64)
        tmem_ld32_nowait(taddr + 64u, s[1]);
    if (rows > 96)
        tmem_ld32_nowait(taddr + 96u, s[1] + 32);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h)
            landed(s[1]);
        if (h || rows <= 64) {
            tc_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0)
                mbar_arrive(empty);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c0 = 64 * h + 16 * i;
            if (c0 >= rows)
                break;
            if (c0 < latest || c0 + 16 > rows)
                weigh16<true>(s[h] + 16 * i, lse, c0, rows, first, c, sum);
            else
                weigh16<false>(s[h] + 16 * i, lse, c0, rows, first, c, sum);
        }
        if (rows <= 64)
            break;
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The weights of tile x of every item, and its masses.
template <int D>
__device__ void add_up(const MassParams &p, const Ctx<D> &c, uint32_t tmem, int x)
{
    const int lane = threadIdx.x & 31;
    const uint32_t taddr = tmem + (uint32_t)x * 256u + ((uint32_t)(threadIdx.x & 96) << 16);
    Walk w;
    Turn qt, st;
    bool alive = true, rows_in = false;
    if (!walk_first(p, w))
        return;
    do {
        const int t = w.t0 + x * kMassTile + (threadIdx.x & 127);
        const bool whole = w.begin == w.block0[0] && w.end == p.blocks;
        const int64_t at = w.b * p.mass.in_request + w.g * p.mass.in_head + t;
        float old = 0.f;
        bool inside = false;
        if (t < w.L) {
            inside = (uint32_t)__ldg(p.block_table + (int64_t)w.b * p.max_pages + t / p.page_size) < (uint32_t)p.num_pages;
            if (whole && p.mass.in)
                old = p.mass.in[at];
        }
        float sum = 0.f;
        for (int k = w.begin; k < w.end; ++k) {
            if (new_rows(p, w)) {
                if (rows_in) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(c.q_empty(qt.slot));
                    qt.next(Ring<D>::kQ);
                }
                rows_in = true;
                if (alive)
                    alive = c.wait(c.q_full(qt.slot), qt.parity);
            }
            if (k < w.block0[x])
                continue;
            if (alive)
                alive = c.wait(c.s_full(x, st.slot), st.parity);
            alive = __all_sync(0xffffffffu, alive);
            const int i0 = k * p.tpt, rows = min(p.tpt, p.n_q - i0) * p.group;
            if (alive) {
                tc_fence_after();
                // query tokens before t - past do not see the thread's token
                const int first = t - w.past - i0, latest = first + 31 - lane;
                sum += weigh(taddr + (uint32_t)st.slot * 128u, c.lse(qt.slot), rows, first * p.group, latest * p.group,
                             p.scale_log2, c.s_empty(x, st.slot));
            } else if (lane == 0) {
                mbar_arrive(c.s_empty(x, st.slot));
            }
            st.next(2);
        }
        if (!inside)
            sum = 0.f;
        if (!whole) {
            // of a range's cut items the first has its end cut off or both, the last its beginning left
            const int i = 2 * blockIdx.x + (w.item != p.cut_item[blockIdx.x] || p.cut_block[blockIdx.x] == 0);
            p.pieces[(int64_t)i * kMassItem + threadIdx.x] = sum;
        } else if (t < w.L) {
            p.mass.out[w.b * p.mass.out_request + w.g * p.mass.out_head + t] = p.mass.in ? fmaf(p.decay, old, sum) : sum;
        }
    } while (walk_next(p, w));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    shkv_mass_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ MassParams p)
{
    extern __shared__ uint8_t raw[];
    Ctx<D> c;
    const uint32_t at = smem_u32(raw);
    c.base = align_up(at, 1024u);
    c.smem = raw + (c.base - at);
    c.abort_flag = reinterpret_cast<volatile uint32_t *>(c.smem + Ring<D>::kMisc);
    c.err = p.err;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < Ring<D>::kK; ++s) {
            mbar_init(c.k_full(s), 1u);
            mbar_init(c.k_empty(s), 1u);
        }
        for (int s = 0; s < Ring<D>::kQ; ++s) {
            mbar_init(c.q_full(s), 1u);
            mbar_init(c.q_empty(s), 9u);     // the MMAs and the eight warps that read the log-sum-exps
        }
        for (int x = 0; x < 2; ++x)
            for (int i = 0; i < 2; ++i) {
                mbar_init(c.s_full(x, i), 1u);
                mbar_init(c.s_empty(x, i), 4u);
            }
        mbar_init(c.fin(), 1u);
        *c.abort_flag = 0u;
        fence_barrier_init();
    }
    // rows that no copy of a block writes: zeros, for good
    const int used = p.tpt * p.group;
    for (int e = threadIdx.x; e < Ring<D>::kQ * (D / 64) * (kMassRows - used) * 8; e += kThreads) {
        const int v = e & 7, r = (e >> 3) % (kMassRows - used), h = (e >> 3) / (kMassRows - used);
        st_shared_zero16(c.q_slot(0) + (uint32_t)h * kHalfBytes + (uint32_t)(used + r) * 128u + (uint32_t)v * 16u);
    }
    fence_proxy_async_smem();
    if (warp == kMmaWarp)
        tmem_alloc(c.base + Ring<D>::kMisc + 4u, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(c.smem + Ring<D>::kMisc + 4u);
    pdl_wait_prior();
    pdl_launch_dependents();
    if (warp == kKWarp)
        copy_k<D>(&tm_k, p, c);
    else if (warp == kQWarp)
        copy_q<D>(&tm_q, p, c);
    else if (warp == kMmaWarp) {
        if ((threadIdx.x & 31) == 0)
            issue<D>(p, c, tmem);
    } else
        add_up<D>(p, c, tmem, warp / 4);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        tmem_dealloc(tmem, kTmemCols);
}

// Items that ranges cut: the sums of the pieces, in the order of the blocks.
// CTA c looks at the cut before range c and does an item's first.
__global__ void __launch_bounds__(kMassItem) shkv_mass_join_kernel(const __grid_constant__ MassParams p)
{
    pdl_wait_prior();
    pdl_launch_dependents();
    const int c = blockIdx.x + 1, item = p.cut_item[c];
    if (p.cut_block[c] == 0 || (p.cut_item[c - 1] == item && p.cut_block[c - 1] > 0))
        return;
    float sum = p.pieces[(int64_t)(2 * (c - 1) + 1) * kMassItem + threadIdx.x];
    for (int i = c; i < p.num_ctas && p.cut_item[i] == item; ++i)
        sum += p.pieces[(int64_t)(2 * i) * kMassItem + threadIdx.x];
    int b = 0;
    while (p.item0[b + 1] <= item)
        ++b;
    const int pairs = (p.lens[b] + kMassItem - 1) / kMassItem;
    const int g = (item - p.item0[b]) / pairs, t = (item - p.item0[b]) % pairs * kMassItem + threadIdx.x;
    if (t < p.lens[b])
        p.mass.out[b * p.mass.out_request + g * p.mass.out_head + t] =
            p.mass.in ? fmaf(p.decay, p.mass.in[b * p.mass.in_request + g * p.mass.in_head + t], sum) : sum;
}

}  // namespace

// tm_k: a column half of one page of one KV head; tm_q: a column half of a block's rows.
cudaError_t launch_mass(const CUtensorMap &tm_k, const CUtensorMap &tm_q, const MassParams &p, bool pieces,
                        cudaStream_t stream)
{
    auto kern = p.head_dim == 64 ? shkv_mass_kernel<64> : shkv_mass_kernel<128>;
    const uint32_t smem = p.head_dim == 64 ? Ring<64>::kBytes : Ring<128>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = launch_pdl(kern, p.num_ctas, kThreads, smem, stream, tm_k, tm_q, p);
    if (e == cudaSuccess && pieces)
        e = launch_pdl(shkv_mass_join_kernel, p.num_ctas - 1, kMassItem, 0u, stream, p);
    return e;
}

}  // namespace shkv
