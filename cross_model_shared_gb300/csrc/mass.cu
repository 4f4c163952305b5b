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
// of a head, those of a chunk stream past the K tiles of an item (a Q block of
// 32 KB feeds up to four MMAs of 128 x 128 x D).
//
// Warps 0-15 take the weights, warp 16 copies K, warp 17 Q (and the log-sum-exps),
// warps 18 and 19 issue the MMAs of an item's even and odd tiles (one issuer alone
// needs 1150 cycles a product, twice the product's time), in one of two ways:
//
// * few blocks (a decode step, a short window): both operands from shared memory,
//   four warps a tile of an item, four S buffers.  Bound by the bytes of K.
// * many blocks: at M = N = 128 two operands from shared memory take 120 of its 128
//   bytes a cycle and leave none for the log-sum-exps, so an item's K goes from
//   shared memory to TMEM (64 columns a tile) once, and two S buffers remain, one
//   for the even tiles and one for the odd ones, each emptied into the registers
//   of eight warps, 64 columns a thread, before the exponentials begin.  Bound by
//   the tensor cores and the exponentials alike (512 cycles a product each).
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "evict.cuh"
#include "launch.cuh"
#include "q8_wait.cuh"
#include "shkv_device.cuh"

namespace shkv {

namespace {

constexpr int kThreads = 640;
constexpr int kKWarp = 16, kQWarp = 17, kMmaWarp = 18;
constexpr uint32_t kTmemCols = 512;          // four S buffers of 128 columns
constexpr uint32_t kHalfBytes = 128u * 128u; // 64 columns of 128 tokens or rows

// Ring slots: at D = 128 seven of 32 KB fill shared memory (K four, a decode's
// 128 KB in flight).
template <int D>
struct Ring {
    static constexpr int kK = D == 128 ? 4 : 8, kQ = D == 128 ? 3 : 5;
    static constexpr uint32_t kSlot = (uint32_t)(D / 64) * kHalfBytes;
    // barriers: K full, K empty, Q full, Q empty, S full, S empty, K in TMEM, fin
    static constexpr int kBars = 2 * kK + 2 * kQ + 14;
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
    __device__ uint32_t s_full(int i) const { return bar(2 * Ring<D>::kK + 2 * Ring<D>::kQ + i); }
    __device__ uint32_t s_empty(int i) const { return s_full(i) + 32u; }
    __device__ uint32_t k_in_tmem(int x) const { return s_full(x) + 64u; }
    __device__ uint32_t fin(int odd) const { return s_full(0) + 96u + 8u * (uint32_t)odd; }
    __device__ uint32_t k_slot(int s) const { return base + (uint32_t)s * Ring<D>::kSlot; }
    __device__ uint32_t q_slot(int s) const { return base + Ring<D>::kQ0 + (uint32_t)s * Ring<D>::kSlot; }
    __device__ uint32_t lse(int s) const { return base + Ring<D>::kLse + (uint32_t)(s * kMassRows * 4); }
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

// A ring of n slots dealt to the tiles of an item: tile x uses x, x + span, ... in
// turn, whatever the other tiles do.  So a slot is waited for by the same role every
// time, in order: with slots handed round in one ring, an item of fewer tiles would
// shift them, and a role that runs ahead could wait for a phase while the one before
// is still open, which a parity wait takes for the phase before that.  Four bits a
// tile count its uses, modulo twice its slots.
struct TileRing {
    uint32_t counts = 0u;
    int span, log2n;
    __device__ TileRing(int span_, int n) : span(span_), log2n(n >= 8 * span_ ? 3 : n >= 4 * span_ ? 2 : n >= 2 * span_) {}
    __device__ int slot(int x) const { return x + span * (int)(counts >> 4 * x & ((1u << log2n) - 1u)); }
    __device__ uint32_t parity(int x) const { return counts >> (4 * x + log2n) & 1u; }
    __device__ void next(int x)
    {
        const uint32_t n = ((counts >> 4 * x & 15u) + 1u) & ((2u << log2n) - 1u);
        counts = (counts & ~(15u << 4 * x)) | n << 4 * x;
    }
};

// The items of a CTA's range, one after another; every role walks them alike.
struct Walk {
    int item, last, b, g, at, items;     // `last`: one past the range's last item; item `at` of the head's `items`
    int L, past, t0;
    int begin, end;                      // blocks of this item in the range
    bool fresh;                          // another (request, KV head) than the item before
    // whether block k has a row that sees a token of tile x
    __device__ bool sees(const MassParams &p, int k, int x) const
    {
        return t0 + x * kMassTile - past < min((k + 1) * p.tpt, p.n_q);
    }
    __device__ bool whole(const MassParams &p) const { return begin == mass_block0(t0, past, p.tpt) && end == p.blocks; }
};

__device__ __forceinline__ void walk_request(const MassParams &p, Walk &w)
{
    w.L = p.lens[w.b];
    w.past = mass_past(w.L, p.n_q, p.causal);
    w.items = (w.L + p.span * kMassTile - 1) / (p.span * kMassTile);
}

__device__ __forceinline__ void walk_item(const MassParams &p, Walk &w)
{
    w.t0 = w.at * p.span * kMassTile;
    w.begin = mass_block0(w.t0, w.past, p.tpt);
    if (w.item == p.cut_item[blockIdx.x])
        w.begin = max(w.begin, p.cut_block[blockIdx.x]);
    w.end = w.item == p.cut_item[blockIdx.x + 1] ? p.cut_block[blockIdx.x + 1] : p.blocks;
}

// Where the sums of a cut item go: of a range's cut items the first has its
// beginning in the range before, the last only its end cut off.
__device__ __forceinline__ int piece_of(const MassParams &p, const Walk &w)
{
    return 2 * blockIdx.x + (w.item != p.cut_item[blockIdx.x] || p.cut_block[blockIdx.x] == 0);
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
    w.g = (w.item - p.item0[lo]) / w.items;
    w.at = (w.item - p.item0[lo]) % w.items;
    w.fresh = true;
    walk_item(p, w);
    return true;
}

__device__ __forceinline__ bool walk_next(const MassParams &p, Walk &w)
{
    if (++w.item >= w.last)
        return false;
    w.fresh = false;
    if (++w.at == w.items) {
        w.at = 0;
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

// K tiles, a lane per (column half, page) of a tile.  A lane also holds one of the
// item's table entries, read an item ahead.  A page outside the pool is left out
// and flagged; the tile's threads look at their table entries themselves.
template <int D>
__device__ void copy_k(const CUtensorMap *tm, const MassParams &p, const Ctx<D> &c)
{
    const int lane = threadIdx.x & 31, P = p.page_size, RB = kMassTile / P;
    const int half = lane / RB, rb = lane % RB;
    const bool copier = half < D / 64;
    const uint64_t pol = l2_evict_first_policy();
    auto entry = [&](const Walk &w) {
        const int pg = w.t0 / P + lane;
        return lane < p.span * RB && pg * P < w.L ? __ldg(p.block_table + (int64_t)w.b * p.max_pages + pg) : -1;
    };
    Walk w;
    TileRing kt(p.span, Ring<D>::kK);
    bool alive = true, more = walk_first(p, w);
    uint32_t armed = 0u, armed_parity = 0u;  // slots with a copy, and of which phase
    int id = more ? entry(w) : -1;
    while (more) {
        Walk next = w;
        more = walk_next(p, next);
        const int next_id = more ? entry(next) : -1;
        if (lane == 0 && w.fresh && w.at == 0 && w.g == 0 && __ldg(p.seq_lens + w.b) != w.L)
            atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
#pragma unroll 1
        for (int x = 0; x < p.span && w.t0 + x * kMassTile < w.L; ++x) {
            const int page = __shfl_sync(0xffffffffu, id, (x * RB + rb) & 31);
            const bool there = copier && w.t0 + x * kMassTile + rb * P < w.L;
            const bool inside = there && (uint32_t)page < (uint32_t)p.num_pages;
            if (there && !inside)
                atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
            const uint32_t mask = __ballot_sync(0xffffffffu, inside);
            const int slot = kt.slot(x);
            bool ok = true;
            if (alive && lane == 0) {
                ok = c.wait(c.k_empty(slot), kt.parity(x) ^ 1u);
                if (ok)
                    mbar_arrive_expect_tx(c.k_full(slot), (uint32_t)__popc(mask) * (uint32_t)P * 128u);
            }
            alive = __all_sync(0xffffffffu, alive && ok);
            if (!alive)
                continue;
            if (inside)
                tma_load_2d(c.k_slot(slot) + (uint32_t)half * kHalfBytes + (uint32_t)(rb * P) * 128u, tm, half * 64,
                            (page * p.hkv + w.g) * P, c.k_full(slot), pol);
            armed |= 1u << slot;
            armed_parity = (armed_parity & ~(1u << slot)) | kt.parity(x) << slot;
            kt.next(x);
        }
        w = next;
        id = next_id;
    }
    if (!alive && lane == 0)                 // wait for the copies in flight
        for (int s = 0; s < Ring<D>::kK; ++s)
            if (armed >> s & 1u)
                mbar_drain_bounded(c.k_full(s), armed_parity >> s & 1u);
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
    int tok[kMassRows / 32], head[kMassRows / 32];       // of the lane's rows in a block
#pragma unroll
    for (int j = 0; j < kMassRows / 32; ++j) {
        tok[j] = (lane + 32 * j) / p.group;
        head[j] = lane + 32 * j - tok[j] * p.group;
    }
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
                    off[j] = lse_base2(__ldg(src + (i0 + tok[j]) * p.lse_token + head[j]));
            }
            bool ok = true;
            if (alive && lane == 0)
                ok = c.wait(c.q_empty(turn.slot), turn.parity ^ 1u);
            alive = alive && __all_sync(0xffffffffu, ok);
            if (!alive)
                continue;
#pragma unroll
            for (int j = 0; j < kMassRows / 32; ++j)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(c.lse(turn.slot) + 4u * (uint32_t)(lane + 32 * j)), "f"(-off[j])
                             : "memory");
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

// The issuers' warps run converged, so that addresses and descriptors stay in
// uniform registers; one lane issues.
template <int D>
__device__ __forceinline__ bool issuer_wait(const Ctx<D> &c, uint32_t bar, uint32_t parity, bool alive)
{
    return __all_sync(0xffffffffu, alive && c.wait(bar, parity));
}

// S = K Q^T for every block of the range and every tile of one parity.  A slot of K
// is free after the item's last block, one of Q when the next block's rows are
// needed.  (Loops are kept rolled: the roles of an SM sub-partition share its
// instruction cache.)
template <int D>
__device__ void issue(const MassParams &p, const Ctx<D> &c, uint32_t tmem, int odd)
{
    const uint64_t kd0 = umma_sdesc_sw128(c.k_slot(0), 16u, 1024u), qd0 = umma_sdesc_sw128(c.q_slot(0), 16u, 1024u);
    const bool one = (threadIdx.x & 31) == 0;
    Walk w;
    Turn qt;
    TileRing kt(p.span, Ring<D>::kK), st(p.span, 4);
    bool alive = true, rows_in = false;
    if (!walk_first(p, w))
        return;
    do {
        const int tiles = min(p.span, (w.L - w.t0 + kMassTile - 1) / kMassTile);
        uint32_t k_in = 0u;                  // tiles whose K has been waited for
#pragma unroll 1
        for (int k = w.begin; k < w.end; ++k) {
            if (new_rows(p, w)) {
                if (rows_in) {
                    if (one)
                        umma_commit(c.q_empty(qt.slot));
                    qt.next(Ring<D>::kQ);
                }
                rows_in = true;
                alive = issuer_wait(c, c.q_full(qt.slot), qt.parity, alive);
            }
            const int rows = min(p.tpt, p.n_q - k * p.tpt) * p.group;
            const uint32_t idesc = umma_idesc_bf16(kMassTile, (rows + 15) & ~15, false, false);
            const uint64_t qd = qd0 + (((uint32_t)qt.slot * Ring<D>::kSlot) >> 4);
#pragma unroll 1
            for (int x = odd; x < tiles; x += 2) {
                if (!w.sees(p, k, x))
                    break;
                const int s = st.slot(x), slot = kt.slot(x);
                if (!(k_in >> x & 1u))
                    alive = issuer_wait(c, c.k_full(slot), kt.parity(x), alive);
                k_in |= 1u << x;
                alive = issuer_wait(c, c.s_empty(s), st.parity(x) ^ 1u, alive);
                tc_fence_after();
                const uint64_t kd = kd0 + (((uint32_t)slot * Ring<D>::kSlot) >> 4);
                if (one) {
                    if (alive) {
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint32_t off = ((uint32_t)(i >> 2) * kHalfBytes + (uint32_t)(i & 3) * 32u) >> 4;
                            umma_bf16(tmem + (uint32_t)s * 128u, kd + off, qd + off, idesc, i ? 1u : 0u);
                        }
                    }
                    umma_commit(c.s_full(s));
                    if (k == w.end - 1)
                        umma_commit(c.k_empty(slot));
                }
                __syncwarp();
                st.next(x);
            }
        }
        for (int x = odd; x < tiles; x += 2) {
            if (!(k_in >> x & 1u)) {         // a range that ends before the tile's first block
                alive = issuer_wait(c, c.k_full(kt.slot(x)), kt.parity(x), alive);
                if (one)
                    umma_commit(c.k_empty(kt.slot(x)));
            }
            kt.next(x);
        }
    } while (walk_next(p, w));
    if (one) {
        umma_commit(c.fin(odd));
        mbar_drain_bounded(c.fin(odd), 0u);
    }
}

__device__ __forceinline__ float4 load_shared4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// The weights of 16 columns into partial sums, two values an instruction where
// there is one for it; kMasked: of the columns [first, end) of them.
template <bool kMasked>
__device__ __forceinline__ void weigh16(const uint32_t *s, uint32_t lse, int first, int end, float c, float2 (&sum)[2])
{
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        const float4 l = load_shared4(lse + 4u * j);
        float2 x0 = __ffma2_rn(make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), make_float2(c, c),
                               make_float2(l.x, l.y));
        float2 x1 = __ffma2_rn(make_float2(__uint_as_float(s[j + 2]), __uint_as_float(s[j + 3])), make_float2(c, c),
                               make_float2(l.z, l.w));
        if (kMasked) {
            x0.x = j >= first && j < end ? x0.x : -INFINITY;
            x0.y = j + 1 >= first && j + 1 < end ? x0.y : -INFINITY;
            x1.x = j + 2 >= first && j + 2 < end ? x1.x : -INFINITY;
            x1.y = j + 3 >= first && j + 3 < end ? x1.y : -INFINITY;
        }
        sum[0] = __fadd2_rn(sum[0], make_float2(ex2_approx(x0.x), ex2_approx(x0.y)));
        sum[1] = __fadd2_rn(sum[1], make_float2(ex2_approx(x1.x), ex2_approx(x1.y)));
    }
}

// A warp has read an S buffer to its end.
__device__ __forceinline__ void leave(uint32_t empty)
{
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(empty);
}

// Sum of a thread's weights over columns [first, n) of S at taddr, n <= 64;
// `latest` is the warp's largest `first`.  The columns that the MMA rounds rows up
// to are zero queries, whose product with an infinite key is no number, so they
// are left out.  `last`: the buffer is arrived on as empty as soon as its values
// are in registers, and the next product into it runs beside the exponentials.
// (No use of a score can move before its wait: it needs a log-sum-exp that is read
// after it.)
__device__ __forceinline__ float weigh(uint32_t taddr, uint32_t lse, int n, int first, int latest, float c, bool last,
                                       uint32_t empty)
{
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (n > 48 && latest <= 0) {             // nearly all blocks of a chunk: straight code
        uint32_t s[64];
        tmem_ld32_nowait(taddr, s);
        tmem_ld32_nowait(taddr + 32u, s + 32);
        tmem_wait_ld();
        if (last)
            leave(empty);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            weigh16<false>(s + 16 * i, lse + 64u * i, 0, 16, c, sum);
        if (n < 64)
            weigh16<true>(s + 48, lse + 192u, 0, n - 48, c, sum);
        else
            weigh16<false>(s + 48, lse + 192u, 0, 16, c, sum);
    } else {
#pragma unroll 1
        for (int i = 0; i < n; i += 16) {
            uint32_t s[16];
            tmem_ld16_nowait(taddr + (uint32_t)i, s);
            tmem_wait_ld();
            if (i < latest || i + 16 > n)
                weigh16<true>(s, lse + 4u * i, first - i, n - i, c, sum);
            else
                weigh16<false>(s, lse + 4u * i, 0, 16, c, sum);
        }
        if (last)
            leave(empty);
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The weights of tile x of every item, and its masses.
template <int D>
__device__ void add_up(const MassParams &p, const Ctx<D> &c, uint32_t tmem, int x)
{
    const int lane = threadIdx.x & 31, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(threadIdx.x & 96) << 16;
    Walk w;
    Turn qt;
    TileRing st(p.span, 4);
    bool alive = true, rows_in = false;
    if (!walk_first(p, w))
        return;
    do {
        const bool whole = w.whole(p), mine = x < p.span && w.t0 + x * kMassTile < w.L;
        const int t = w.t0 + x * kMassTile + row;
        float old = 0.f, sum = 0.f;
        bool inside = false;
        if (mine && t < w.L) {
            inside = (uint32_t)__ldg(p.block_table + (int64_t)w.b * p.max_pages + t / p.page_size) < (uint32_t)p.num_pages;
            if (whole && p.mass.in)
                old = p.mass.in[w.b * p.mass.in_request + w.g * p.mass.in_head + t];
        }
#pragma unroll 1
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
            if (!mine || !w.sees(p, k, x))
                continue;
            const int i0 = k * p.tpt, rows = min(p.tpt, p.n_q - i0) * p.group;
            const int s = st.slot(x);
            if (alive)
                alive = c.wait(c.s_full(s), st.parity(x));
            alive = __all_sync(0xffffffffu, alive);
            if (alive) {
                tc_fence_after();
                // query tokens before t - past do not see the thread's token
                const int first = (t - w.past - i0) * p.group, latest = first + (31 - lane) * p.group;
                const uint32_t taddr = tmem + lanes + (uint32_t)s * 128u;
#pragma unroll 1
                for (int h = 0; h < rows; h += 64)
                    sum += weigh(taddr + (uint32_t)h, c.lse(qt.slot) + 4u * h, min(64, rows - h), first - h, latest - h,
                                 p.scale_log2, h + 64 >= rows, c.s_empty(s));
            } else if (lane == 0) {
                mbar_arrive(c.s_empty(s));
            }
            st.next(x);
        }
        if (!mine || t >= w.L)
            continue;
        if (!inside)
            sum = 0.f;
        if (!whole)
            p.pieces[(int64_t)piece_of(p, w) * (kMassSpan * kMassTile) + t - w.t0] = sum;
        else
            p.mass.out[w.b * p.mass.out_request + w.g * p.mass.out_head + t] =
                p.mass.in ? fmaf(p.decay, old, sum) : sum;
    } while (walk_next(p, w));
}

// ---------------------------------------------------------------------------
// many blocks: K in TMEM
// ---------------------------------------------------------------------------
constexpr uint32_t kStreamS = 256u;          // first column of the two S buffers; tile x's K is at 64 x

template <int D>
__device__ void issue_stream(const MassParams &p, const Ctx<D> &c, uint32_t tmem, int odd)
{
    const uint64_t qd0 = umma_sdesc_sw128(c.q_slot(0), 16u, 1024u);
    const uint32_t d = tmem + kStreamS + (uint32_t)odd * 128u, empty = c.s_empty(odd), full = c.s_full(odd);
    const bool one = (threadIdx.x & 31) == 0;
    Walk w;
    Turn qt;
    uint32_t s_par = 1u, k_par = 0u;         // of the S buffer's next wait; of the tiles' (odd, odd + 2), a bit each
    bool alive = true, rows_in = false;
    if (!walk_first(p, w))
        return;
    do {
        const int tiles = min(p.span, (w.L - w.t0 + kMassTile - 1) / kMassTile);
        uint32_t k_in = 0u;                  // tiles whose K has been waited for
#pragma unroll 1
        for (int k = w.begin; k < w.end; ++k) {
            if (rows_in) {
                if (one)
                    umma_commit(c.q_empty(qt.slot));
                qt.next(Ring<D>::kQ);
            }
            rows_in = true;
            const int rows = min(p.tpt, p.n_q - k * p.tpt) * p.group;
            const uint32_t idesc = umma_idesc_bf16(kMassTile, (rows + 15) & ~15, false, false);
            const uint64_t qd = qd0 + (((uint32_t)qt.slot * Ring<D>::kSlot) >> 4);
            alive = issuer_wait(c, c.q_full(qt.slot), qt.parity, alive);
#pragma unroll 1
            for (int x = odd; x < tiles; x += 2) {
                if (!w.sees(p, k, x))
                    break;
                const uint32_t a = tmem + (uint32_t)(x * 64);
                if (!(k_in >> x & 1u))
                    alive = issuer_wait(c, c.k_in_tmem(x), k_par >> x & 1u, alive);
                k_in |= 1u << x;
                alive = issuer_wait(c, empty, s_par, alive);
                tc_fence_after();
                if (one) {
                    if (alive) {
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint32_t off = ((uint32_t)(i >> 2) * kHalfBytes + (uint32_t)(i & 3) * 32u) >> 4;
                            umma_bf16_ts(d, a + (uint32_t)(i * 8), qd + off, idesc, i ? 1u : 0u);
                        }
                    }
                    umma_commit(full);
                }
                __syncwarp();
                s_par ^= 1u;
            }
        }
        for (int x = odd; x < tiles; x += 2) // a range that ends before the tile's first block
            if (!(k_in >> x & 1u))
                alive = issuer_wait(c, c.k_in_tmem(x), k_par >> x & 1u, alive);
        k_par ^= (1u << tiles) - 1u;
    } while (walk_next(p, w));
    if (one) {
        umma_commit(c.fin(odd));
        mbar_drain_bounded(c.fin(odd), 0u);
    }
}

// K of an item's tiles into TMEM, a tile of four warps each; the weights of the
// even tiles by warps 0-7, of the odd ones by warps 8-15, each four warps of
// them taking half of the columns; the halves joined, the masses.
template <int D>
__device__ void add_up_stream(const MassParams &p, const Ctx<D> &c, uint32_t tmem, int four)
{
    const int lane = threadIdx.x & 31, row = threadIdx.x & 127, odd = four / 2, half = four % 2;
    const uint32_t lanes = (uint32_t)(threadIdx.x & 96) << 16;
    // this warp's columns of its S buffer; and the barrier of the two warps of the same tokens
    const uint32_t s_mine = tmem + kStreamS + lanes + (uint32_t)(128 * odd + 64 * half);
    const uint32_t pair_bar = 1u + (uint32_t)(4 * odd + row / 32);
    Walk w;
    Turn qt;
    TileRing kt(p.span, Ring<D>::kK);
    const int own = 2 * half + odd;          // the tile that this warp takes to TMEM
    uint32_t s_par = 0u;
    bool alive = true, rows_in = false;
    if (!walk_first(p, w))
        return;
    do {
        const int tiles = min(p.span, (w.L - w.t0 + kMassTile - 1) / kMassTile);
        // every product that read the tile's last K is done: the warps of its parity
        // have waited for all of them
        if (own < tiles) {
            const int slot = kt.slot(own);
            if (alive)
                alive = c.wait(c.k_full(slot), kt.parity(own));
            alive = __all_sync(0xffffffffu, alive);
            if (alive) {
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    uint32_t v[32];
                    const uint32_t src = c.k_slot(slot) + (uint32_t)h * kHalfBytes + (uint32_t)row * 128u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 f = load_shared4(src + (uint32_t)((i ^ (row & 7)) << 4));
                        v[4 * i] = __float_as_uint(f.x), v[4 * i + 1] = __float_as_uint(f.y);
                        v[4 * i + 2] = __float_as_uint(f.z), v[4 * i + 3] = __float_as_uint(f.w);
                    }
                    tmem_st32(tmem + lanes + (uint32_t)(own * 64 + h * 32), v);
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(c.k_in_tmem(own));
                mbar_arrive(c.k_empty(slot));
            }
            kt.next(own);
        }
        float sum[2] = {0.f, 0.f};           // tiles odd and odd + 2
#pragma unroll 1
        for (int k = w.begin; k < w.end; ++k) {
            if (rows_in) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(c.q_empty(qt.slot));
                qt.next(Ring<D>::kQ);
            }
            rows_in = true;
            if (alive)
                alive = c.wait(c.q_full(qt.slot), qt.parity);
            const int i0 = k * p.tpt, n = min(min(p.tpt, p.n_q - i0) * p.group - 64 * half, 64);
#pragma unroll 1
            for (int x = odd; x < tiles; x += 2) {
                if (!w.sees(p, k, x))
                    break;
                if (alive)
                    alive = c.wait(c.s_full(odd), s_par);
                alive = __all_sync(0xffffffffu, alive);
                if (alive) {
                    tc_fence_after();
                    // query tokens before t - past do not see token t
                    const int first = (w.t0 + x * kMassTile + row - w.past - i0) * p.group - 64 * half;
                    const float v = weigh(s_mine, c.lse(qt.slot) + 256u * half, n, first, first + (31 - lane) * p.group,
                                          p.scale_log2, true, c.s_empty(odd));
                    sum[0] += x < 2 ? v : 0.f;
                    sum[1] += x < 2 ? 0.f : v;
                } else if (lane == 0) {
                    mbar_arrive(c.s_empty(odd));
                }
                s_par ^= 1u;
            }
        }
        // the upper half's sums by way of its own columns of S, which no product
        // writes before the next item's K is in TMEM
        if (half) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __float_as_uint(sum[i & 1]);
            tmem_st8_nowait(s_mine, v);
            tmem_wait_st();
            tc_fence_before();
        }
        named_barrier(pair_bar, 64u);
        if (half == 0) {
            uint32_t v[8];
            tc_fence_after();
            tmem_ld8_nowait(s_mine + 64u, v);
            tmem_wait_ld();
            tc_fence_before();
            const bool whole = w.whole(p);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int x = 2 * i + odd, t = w.t0 + x * kMassTile + row;
                if (x >= tiles || t >= w.L)
                    continue;
                const bool inside = (uint32_t)__ldg(p.block_table + (int64_t)w.b * p.max_pages + t / p.page_size) <
                                    (uint32_t)p.num_pages;
                const float total = inside ? sum[i] + __uint_as_float(v[i]) : 0.f;
                if (!whole)
                    p.pieces[(int64_t)piece_of(p, w) * (kMassSpan * kMassTile) + t - w.t0] = total;
                else
                    p.mass.out[w.b * p.mass.out_request + w.g * p.mass.out_head + t] =
                        p.mass.in ? fmaf(p.decay, p.mass.in[w.b * p.mass.in_request + w.g * p.mass.in_head + t], total)
                                  : total;
            }
        }
    } while (walk_next(p, w));
}

template <int D, bool kStream>
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
            mbar_init(c.k_empty(s), kStream ? 4u : 1u);   // the warps that take it to TMEM, or the MMAs
        }
        for (int s = 0; s < Ring<D>::kQ; ++s) {
            mbar_init(c.q_full(s), 1u);
            mbar_init(c.q_empty(s), 18u);    // both issuers' MMAs and the warps that read the log-sum-exps
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(c.s_full(i), 1u);
            mbar_init(c.s_empty(i), kStream ? 8u : 4u);
            mbar_init(c.k_in_tmem(i), 4u);
        }
        mbar_init(c.fin(0), 1u);
        mbar_init(c.fin(1), 1u);
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
    else if (warp >= kMmaWarp) {
        if (kStream)
            issue_stream<D>(p, c, tmem, warp - kMmaWarp);
        else
            issue<D>(p, c, tmem, warp - kMmaWarp);
    } else if (kStream)
        add_up_stream<D>(p, c, tmem, warp / 4);
    else
        add_up<D>(p, c, tmem, warp / 4);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        tmem_dealloc(tmem, kTmemCols);
}

// Items that ranges cut: the sums of the pieces, in the order of the blocks.
// CTA c looks at the cut before range c and does an item's first.
__global__ void __launch_bounds__(kMassSpan *kMassTile) shkv_mass_join_kernel(const __grid_constant__ MassParams p)
{
    pdl_wait_prior();
    pdl_launch_dependents();
    const int c = blockIdx.x + 1, item = p.cut_item[c], u = threadIdx.x;
    if (p.cut_block[c] == 0 || (p.cut_item[c - 1] == item && p.cut_block[c - 1] > 0))
        return;
    int b = 0, hi = p.batch;
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (p.item0[mid] <= item)
            b = mid;
        else
            hi = mid;
    }
    const int tokens = p.span * kMassTile, items = (p.lens[b] + tokens - 1) / tokens;
    const int g = (item - p.item0[b]) / items, t = (item - p.item0[b]) % items * tokens + u;
    if (u >= tokens || t >= p.lens[b])
        return;
    float sum = p.pieces[(int64_t)(2 * (c - 1) + 1) * (kMassSpan * kMassTile) + u];
    for (int i = c; i < p.num_ctas && p.cut_item[i] == item; ++i)
        sum += p.pieces[(int64_t)(2 * i) * (kMassSpan * kMassTile) + u];
    p.mass.out[b * p.mass.out_request + g * p.mass.out_head + t] =
        p.mass.in ? fmaf(p.decay, p.mass.in[b * p.mass.in_request + g * p.mass.in_head + t], sum) : sum;
}

}  // namespace

// tm_k: a column half of one page of one KV head; tm_q: a column half of a block's rows.
cudaError_t launch_mass(const CUtensorMap &tm_k, const CUtensorMap &tm_q, const MassParams &p, bool pieces,
                        cudaStream_t stream)
{
    const bool many = p.blocks >= kMassStream;
    auto kern = p.head_dim == 64 ? (many ? shkv_mass_kernel<64, true> : shkv_mass_kernel<64, false>)
                                 : (many ? shkv_mass_kernel<128, true> : shkv_mass_kernel<128, false>);
    const uint32_t smem = p.head_dim == 64 ? Ring<64>::kBytes : Ring<128>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = launch_pdl(kern, p.num_ctas, kThreads, smem, stream, tm_k, tm_q, p);
    if (e == cudaSuccess && pieces)
        e = launch_pdl(shkv_mass_join_kernel, p.num_ctas - 1, kMassSpan * kMassTile, 0u, stream, p);
    return e;
}

}  // namespace shkv
