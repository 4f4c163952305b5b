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
// K is read once per call.  Nothing is added across threads but in a fixed order:
// no atomics, the same bits every time.  Two ways:
//
// * Few blocks of rows (a decode step, a short window): tokens on the MMA's M
//   dimension, S[t, r] = K Q^T with M = 128 tokens and N = up to 128 rows in one of
//   four TMEM buffers.  A thread owns a token (its TMEM lane) and adds up its row of
//   weights in a register.  The rows stay in shared memory while a CTA walks along
//   the tokens of a head.  Bound by the bytes of K.
// * Many blocks: rows on M, S[r, t] = Q K^T with N = the 256 tokens of an item, whose
//   K stays while the blocks stream past.  A thread owns a row and 64 tokens, for
//   which it adds up the weights of its row in every block in 64 registers; the
//   threads' sums are joined at the item's end.  A row's log-sum-exp is one register
//   then: with tokens on M every weight needs one from shared memory, and at 512
//   cycles a product of 128 x 128 those reads alone take as long as the product
//   (2048 new tokens of 40 heads behind 38k: 774 us).  Bound by the tensor cores and
//   the exponentials alike, 512 cycles each.
//
// Warps 0-15 take the weights, warp 16 copies K, warp 17 Q (and the log-sum-exps),
// warps 18 and 19 issue the MMAs: of the even and of the odd tiles with few blocks
// (one issuer alone needs about 1150 cycles a product), warp 18 all with many.
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
constexpr uint32_t kTmemCols = 512;          // four S buffers of 128 columns, or two of 256
// Registers a thread, many blocks (setmaxnreg): 112 * 512 + 32 * 128 = 96 * 640.  (At
// 104 for the weights their inner loop spills: half as fast again.)
constexpr uint32_t kLaunchRegs = 96, kWeightRegs = 112, kOtherRegs = 32;
static_assert(kWeightRegs * 512 + kOtherRegs * 128 == kLaunchRegs * kThreads, "register split");
constexpr uint32_t kHalfBytes = 128u * 128u; // 64 columns of 128 tokens or rows

// Ring slots: at D = 128 seven of 32 KB fill shared memory (K four, a decode's
// 128 KB in flight).
template <int D>
struct Ring {
    static constexpr int kK = D == 128 ? 4 : 8, kQ = D == 128 ? 3 : 5;
    static constexpr uint32_t kSlot = (uint32_t)(D / 64) * kHalfBytes;
    // barriers: K full, K empty, Q full, Q empty, S full, S empty, fin
    static constexpr int kBars = 2 * kK + 2 * kQ + 10;
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
    __device__ uint32_t fin(int odd) const { return s_full(0) + 64u + 8u * (uint32_t)odd; }
    __device__ uint32_t k_slot(int s) const { return base + (uint32_t)s * Ring<D>::kSlot; }
    __device__ uint32_t q_slot(int s) const { return base + Ring<D>::kQ0 + (uint32_t)s * Ring<D>::kSlot; }
    __device__ uint32_t lse(int s) const { return base + Ring<D>::kLse + (uint32_t)(s * kMassRows * 4); }
    // a byte: whether a row of the block in slot s attends nothing
    __device__ uint32_t outs(int s) const { return base + Ring<D>::kMisc + 8u + (uint32_t)s; }
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
    int item, last, b, g, at, items;     // `last`: one past the range's last item; item `at` of the head's `items`
    int step;                            // items taken together: with few blocks up to four tiles of a head
    int L, past, t0;
    int begin, end;                      // blocks of this item in the range
    bool fresh;                          // another (request, KV head) than the item before
    // whether block k has a row that sees a token of the step's tile x
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
    w.items = (w.L + p.item_tokens - 1) / (p.item_tokens);
}

__device__ __forceinline__ void walk_item(const MassParams &p, Walk &w)
{
    w.t0 = w.at * p.item_tokens;
    w.step = p.item_tokens == kWide ? 1 : min(4, min(w.items - w.at, w.last - w.item));
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
    w.item += w.step;
    if (w.item >= w.last)
        return false;
    w.fresh = false;
    w.at += w.step;
    if (w.at == w.items) {
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

// ---------------------------------------------------------------------------
// few blocks: tokens on M, an item is a tile, up to four are taken together
// ---------------------------------------------------------------------------
// Tile n of a range (n = 0, 1, ..) uses K slot n mod kK, S buffer n mod 4, and belongs
// to issuer n mod 2 and to the four warps n mod 4.  As kK is a multiple of 4, a slot
// is waited for by the same role every time, in order: a role that waited only for
// some of a slot's phases could look at the slot while the phase before is still
// open, and a parity wait takes that for the phase before it, which is over.
__device__ __forceinline__ int tile_of(const MassParams &p, const Walk &w) { return w.item - p.cut_item[blockIdx.x]; }

// Every request's length against the device's, requests without a token among them (in
// the warp that copies K, behind its copies).
__device__ __forceinline__ void check_lens(const MassParams &p)
{
    for (int b = 32 * blockIdx.x + (threadIdx.x & 31); b < p.batch; b += 32 * gridDim.x)
        if (p.seq_lens[b] != p.lens[b])
            atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
}

// K tiles, a lane per (column half, page) of a tile.  A lane also holds one of the
// table entries of up to four tiles, read four tiles ahead.  A page outside the pool
// is left out and flagged; the tile's threads look at their table entries themselves.
template <int D>
__device__ void copy_k(const CUtensorMap *tm, const MassParams &p, const Ctx<D> &c)
{
    const int lane = threadIdx.x & 31, P = p.page_size, RB = kMassTile / P;
    const int half = lane / RB, rb = lane % RB;
    const bool copier = half < D / 64;
    const uint64_t pol = l2_evict_first_policy();
    auto entry = [&](const Walk &w) {
        const int pg = w.t0 / P + lane;
        return lane < w.step * RB && pg * P < w.L ? p.block_table[(int64_t)w.b * p.max_pages + pg] : -1;
    };
    Walk w;
    bool alive = true, more = walk_first(p, w);
    int issued = 0, id = more ? entry(w) : -1;
#pragma unroll 1
    while (more) {
        Walk next = w;
        more = walk_next(p, next);
        const int next_id = more ? entry(next) : -1;
#pragma unroll 1
        for (int x = 0; x < w.step; ++x) {
            const int slot = issued % Ring<D>::kK, page = __shfl_sync(0xffffffffu, id, (x * RB + rb) & 31);
            const bool there = copier && w.t0 + x * kMassTile + rb * P < w.L;
            const bool inside = there && (uint32_t)page < (uint32_t)p.num_pages;
            if (there && !inside)
                atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
            const uint32_t mask = __ballot_sync(0xffffffffu, inside);
            bool ok = true;
            if (alive && lane == 0) {
                ok = c.wait(c.k_empty(slot), ((uint32_t)(issued / Ring<D>::kK) & 1u) ^ 1u);
                if (ok)
                    mbar_arrive_expect_tx(c.k_full(slot), (uint32_t)__popc(mask) * (uint32_t)P * 128u);
            }
            alive = __all_sync(0xffffffffu, alive && ok);
            if (!alive)
                continue;
            if (inside)
                tma_load_2d(c.k_slot(slot) + (uint32_t)half * kHalfBytes + (uint32_t)(rb * P) * 128u, tm, half * 64,
                            (page * p.hkv + w.g) * P, c.k_full(slot), pol);
            ++issued;
        }
        w = next;
        id = next_id;
    }
    if (!alive && lane == 0)                 // wait for the copies in flight
        for (int i = max(0, issued - Ring<D>::kK); i < issued; ++i)
            mbar_drain_bounded(c.k_full(i % Ring<D>::kK), (uint32_t)(i / Ring<D>::kK) & 1u);
}

// Block k of the rows of an item's head into a Q slot.
template <int D>
__device__ __forceinline__ void copy_block(const CUtensorMap *tm, const MassParams &p, const Ctx<D> &c, const Walk &w, int k,
                                           int slot)
{
    const int lane = threadIdx.x & 31;
    if (lane == 0)
        mbar_arrive_expect_tx(c.q_full(slot), (uint32_t)(p.tpt * p.group * D * 2));
    __syncwarp();
    if (lane < D / 64)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(c.q_slot(slot) + (uint32_t)lane * kHalfBytes),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(lane * 64), "r"(w.g * p.group), "r"(k * p.tpt), "r"(w.b),
            "r"(c.q_full(slot))
            : "memory");
}

// The blocks of every head that the range comes to, what their rows' log-sum-exps
// add to the scores, and whether one of the rows attends nothing.
template <int D>
__device__ void copy_q(const CUtensorMap *tm, const MassParams &p, const Ctx<D> &c)
{
    const int lane = threadIdx.x & 31;
    Walk w;
    Turn turn;
    bool alive = true;
    int issued = 0;
    if (!walk_first(p, w))
        return;
    do {
        if (!w.fresh)
            continue;
        const float *src = p.lse + w.b * p.lse_request + w.g * p.group;
#pragma unroll 1
        for (int k = 0; k < p.blocks; ++k) {
            const int i0 = k * p.tpt, rows = min(p.tpt, p.n_q - i0) * p.group;
            float l[kMassRows / 32];
            bool out = false;
#pragma unroll
            for (int j = 0; j < kMassRows / 32; ++j) {
                const int r = lane + 32 * j;
                l[j] = r < rows ? lse_offset(src[(i0 + r / p.group) * p.lse_token + r % p.group]) : 0.f;
                out = out || l[j] == kRowOut;
            }
            out = __any_sync(0xffffffffu, out);
            bool ok = true;
            if (alive && lane == 0)
                ok = c.wait(c.q_empty(turn.slot), turn.parity ^ 1u);
            alive = alive && __all_sync(0xffffffffu, ok);
            if (!alive)
                continue;
#pragma unroll
            for (int j = 0; j < kMassRows / 32; ++j)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(c.lse(turn.slot) + 4u * (uint32_t)(lane + 32 * j)), "f"(l[j])
                             : "memory");
            if (lane == 0)
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(c.outs(turn.slot)), "r"((uint32_t)out) : "memory");
            __syncwarp();
            copy_block<D>(tm, p, c, w, k, turn.slot);
            ++issued;
            turn.next(Ring<D>::kQ);
        }
    } while (walk_next(p, w));
    if (!alive && lane == 0)
        for (int i = max(0, issued - Ring<D>::kQ); i < issued; ++i)
            mbar_drain_bounded(c.q_full(i % Ring<D>::kQ), (uint32_t)(i / Ring<D>::kQ) & 1u);
}

// The next head's blocks: leaves the last one's (`done` on each of their slots) and
// waits for these.  `turn` is the first one's.
template <int D, typename Done>
__device__ __forceinline__ bool next_blocks(const MassParams &p, const Ctx<D> &c, Turn &turn, bool first, bool alive, Done done)
{
    if (!first)
#pragma unroll 1
        for (int k = 0; k < p.blocks; ++k) {
            done(turn.slot);
            turn.next(Ring<D>::kQ);
        }
    Turn t = turn;
#pragma unroll 1
    for (int k = 0; k < p.blocks; ++k) {
        alive = __all_sync(0xffffffffu, alive && c.wait(c.q_full(t.slot), t.parity));
        t.next(Ring<D>::kQ);
    }
    return alive;
}

// The issuers' warps run converged, so that addresses and descriptors stay in
// uniform registers; one lane issues.
template <int D>
__device__ __forceinline__ bool issuer_wait(const Ctx<D> &c, uint32_t bar, uint32_t parity, bool alive)
{
    return __all_sync(0xffffffffu, alive && c.wait(bar, parity));
}

// S = K Q^T for the range's tiles of one parity and every block that sees them.
template <int D>
__device__ void issue(const MassParams &p, const Ctx<D> &c, uint32_t tmem, int odd)
{
    const uint64_t kd0 = umma_sdesc_sw128(c.k_slot(0), 16u, 1024u), qd0 = umma_sdesc_sw128(c.q_slot(0), 16u, 1024u);
    const bool one = (threadIdx.x & 31) == 0;
    Walk w;
    Turn qt;
    uint32_t s_par = 0xfu;                   // of the S buffers' next waits
    bool alive = true, first = true;
    if (!walk_first(p, w))
        return;
    do {
        if (w.fresh) {
            alive = next_blocks<D>(p, c, qt, first, alive, [&](int slot) {
                if (one)
                    umma_commit(c.q_empty(slot));
            });
            first = false;
        }
        const int n0 = tile_of(p, w);
#pragma unroll 1
        for (int x = (n0 ^ odd) & 1; x < w.step; x += 2) {
            const int n = n0 + x, s = n & 3, slot = n % Ring<D>::kK;
            const uint64_t kd = kd0 + (((uint32_t)slot * Ring<D>::kSlot) >> 4);
            alive = issuer_wait(c, c.k_full(slot), (uint32_t)(n / Ring<D>::kK) & 1u, alive);
            Turn t = qt;
#pragma unroll 1
            for (int k = 0; k < p.blocks; ++k, t.next(Ring<D>::kQ)) {
                if (!w.sees(p, k, x))
                    continue;
                const int rows = min(p.tpt, p.n_q - k * p.tpt) * p.group;
                const uint32_t idesc = umma_idesc_bf16(kMassTile, (rows + 15) & ~15, false, false);
                const uint64_t qd = qd0 + (((uint32_t)t.slot * Ring<D>::kSlot) >> 4);
                alive = issuer_wait(c, c.s_empty(s), s_par >> s & 1u, alive);
                s_par ^= 1u << s;
                tc_fence_after();
                if (one) {
                    if (alive) {
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint32_t off = ((uint32_t)(i >> 2) * kHalfBytes + (uint32_t)(i & 3) * 32u) >> 4;
                            umma_bf16(tmem + (uint32_t)s * 128u, kd + off, qd + off, idesc, i ? 1u : 0u);
                        }
                    }
                    umma_commit(c.s_full(s));
                    if (k == p.blocks - 1)
                        umma_commit(c.k_empty(slot));
                }
                __syncwarp();
            }
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
// there is one for it; kMasked: of the columns [first, end) of them; kOuts: of those
// whose rows are not out.
template <bool kMasked, bool kOuts = false>
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
        if (kOuts) {
            x0.x = l.x != kRowOut ? x0.x : -INFINITY;
            x0.y = l.y != kRowOut ? x0.y : -INFINITY;
            x1.x = l.z != kRowOut ? x1.x : -INFINITY;
            x1.y = l.w != kRowOut ? x1.y : -INFINITY;
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
// are left out, as are rows that attend nothing where there are some (`outs`: 128
// rows with a quarter out 41 us, 28 with all in).
// `last`: the buffer is arrived on as empty as soon as its values are in registers,
// and the next product into it runs beside the exponentials.  (No use of a score can
// move before its wait: it needs a log-sum-exp that is read after it.)
__device__ __forceinline__ float weigh(uint32_t taddr, uint32_t lse, int n, int first, int latest, float c, bool outs,
                                       bool last, uint32_t empty)
{
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (n > 48 && latest <= 0 && !outs) {    // nearly all blocks of a chunk: straight code
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
            if (outs)
                weigh16<true, true>(s, lse + 4u * i, first - i, n - i, c, sum);
            else if (i < latest || i + 16 > n)
                weigh16<true>(s, lse + 4u * i, first - i, n - i, c, sum);
            else
                weigh16<false>(s, lse + 4u * i, 0, 16, c, sum);
        }
        if (last)
            leave(empty);
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The weights of every fourth tile, and its masses.
template <int D>
__device__ void add_up(const MassParams &p, const Ctx<D> &c, uint32_t tmem, int four)
{
    const int lane = threadIdx.x & 31;
    const uint32_t taddr = tmem + ((uint32_t)(threadIdx.x & 96) << 16) + 128u * (uint32_t)four;
    Walk w;
    Turn qt;
    uint32_t s_par = 0u;
    bool alive = true, first = true;
    if (!walk_first(p, w))
        return;
    do {
        if (w.fresh) {
            alive = next_blocks<D>(p, c, qt, first, alive, [&](int slot) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(c.q_empty(slot));
            });
            first = false;
        }
        const int x = (four - tile_of(p, w)) & 3;
        if (x >= w.step)
            continue;
        const int t = w.t0 + x * kMassTile + (threadIdx.x & 127);
        float old = 0.f, sum = 0.f;
        int page = -1;
        if (t < w.L) {                       // looked at when the sum is there
            page = p.block_table[(int64_t)w.b * p.max_pages + t / p.page_size];
            if (p.mass.in)
                old = p.mass.in[w.b * p.mass.in_request + w.g * p.mass.in_head + t];
        }
        Turn q = qt;
#pragma unroll 1
        for (int k = 0; k < p.blocks; ++k, q.next(Ring<D>::kQ)) {
            if (!w.sees(p, k, x))
                continue;
            const int i0 = k * p.tpt, rows = min(p.tpt, p.n_q - i0) * p.group;
            uint32_t outs;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(outs) : "r"(c.outs(q.slot)));
            alive = __all_sync(0xffffffffu, alive && c.wait(c.s_full(four), s_par));
            s_par ^= 1u;
            if (alive) {
                tc_fence_after();
                // of the thread's token, and of the warp's last
                const int first_row = mass_first_row(t, w.past, i0, p.group);
                const int latest = mass_first_row(t + 31 - lane, w.past, i0, p.group);
#pragma unroll 1
                for (int h = 0; h < rows; h += 64)
                    sum += weigh(taddr + (uint32_t)h, c.lse(q.slot) + 4u * h, min(64, rows - h), first_row - h, latest - h,
                                 p.scale_log2, outs != 0u, h + 64 >= rows, c.s_empty(four));
            } else if (lane == 0) {
                mbar_arrive(c.s_empty(four));
            }
        }
        if (t >= w.L)
            continue;
        if ((uint32_t)page >= (uint32_t)p.num_pages)
            sum = 0.f;
        p.mass.out[w.b * p.mass.out_request + w.g * p.mass.out_head + t] = p.mass.in ? fmaf(p.decay, old, sum) : sum;
    } while (walk_next(p, w));
}

// ---------------------------------------------------------------------------
// many blocks: rows on M, 256 tokens on N
// ---------------------------------------------------------------------------

// An item's K, [column half][256 tokens][128 B], a lane per (half, page); pages as
// in copy_k().
template <int D>
__device__ void copy_k_wide(const CUtensorMap *tm, const MassParams &p, const Ctx<D> &c)
{
    constexpr int kSlots = Ring<D>::kK / 2;
    const int lane = threadIdx.x & 31, P = p.page_size, RB = kWide / P;
    const uint64_t pol = l2_evict_first_policy();
    auto entry = [&](const Walk &w) {
        const int pg = w.t0 / P + lane;
        return lane < RB && pg * P < w.L ? p.block_table[(int64_t)w.b * p.max_pages + pg] : -1;
    };
    Walk w;
    Turn turn;
    bool alive = true, more = walk_first(p, w);
    int issued = 0, id = more ? entry(w) : -1;
    while (more) {
        Walk next = w;
        more = walk_next(p, next);
        const int next_id = more ? entry(next) : -1;
        const bool there = lane < RB && w.t0 + lane * P < w.L, inside = there && (uint32_t)id < (uint32_t)p.num_pages;
        if (there && !inside)
            atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
        const uint32_t mask = __ballot_sync(0xffffffffu, inside);
        bool ok = true;
        if (alive && lane == 0) {
            ok = c.wait(c.k_empty(turn.slot), turn.parity ^ 1u);
            if (ok)
                mbar_arrive_expect_tx(c.k_full(turn.slot), (uint32_t)(__popc(mask) * P * D * 2));
        }
        alive = __all_sync(0xffffffffu, alive && ok);
        if (alive) {
            if (inside)
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    tma_load_2d(c.k_slot(2 * turn.slot) + (uint32_t)(h * kWide + lane * P) * 128u, tm, h * 64,
                                (id * p.hkv + w.g) * P, c.k_full(turn.slot), pol);
            ++issued;
            turn.next(kSlots);
        }
        w = next;
        id = next_id;
    }
    if (!alive && lane == 0)
        for (int i = max(0, issued - kSlots); i < issued; ++i)
            mbar_drain_bounded(c.k_full(i % kSlots), (uint32_t)(i / kSlots) & 1u);
}

template <int D>
__device__ void copy_q_wide(const CUtensorMap *tm, const MassParams &p, const Ctx<D> &c)
{
    Walk w;
    Turn turn;
    bool alive = true;
    int issued = 0;
    if (!walk_first(p, w))
        return;
    do {
#pragma unroll 1
        for (int k = w.begin; k < w.end; ++k) {
            alive = issuer_wait(c, c.q_empty(turn.slot), turn.parity ^ 1u, alive);
            if (!alive)
                continue;
            copy_block<D>(tm, p, c, w, k, turn.slot);
            ++issued;
            turn.next(Ring<D>::kQ);
        }
    } while (walk_next(p, w));
    if (!alive && (threadIdx.x & 31) == 0)
        for (int i = max(0, issued - Ring<D>::kQ); i < issued; ++i)
            mbar_drain_bounded(c.q_full(i % Ring<D>::kQ), (uint32_t)(i / Ring<D>::kQ) & 1u);
}

template <int D>
__device__ void issue_wide(const MassParams &p, const Ctx<D> &c, uint32_t tmem)
{
    const uint64_t kd0 = umma_sdesc_sw128(c.k_slot(0), 16u, 1024u), qd0 = umma_sdesc_sw128(c.q_slot(0), 16u, 1024u);
    const bool one = (threadIdx.x & 31) == 0;
    Walk w;
    Turn kt, qt, st;
    bool alive = true;
    if (!walk_first(p, w))
        return;
    do {
        const uint32_t idesc = umma_idesc_bf16(128, w.t0 + kMassTile < w.L ? kWide : kMassTile, false, false);
        const uint64_t kd = kd0 + ((2u * (uint32_t)kt.slot * Ring<D>::kSlot) >> 4);
        alive = issuer_wait(c, c.k_full(kt.slot), kt.parity, alive);
#pragma unroll 1
        for (int k = w.begin; k < w.end; ++k) {
            const uint64_t qd = qd0 + (((uint32_t)qt.slot * Ring<D>::kSlot) >> 4);
            alive = issuer_wait(c, c.q_full(qt.slot), qt.parity, alive);
            alive = issuer_wait(c, c.s_empty(st.slot), st.parity ^ 1u, alive);
            tc_fence_after();
            if (one) {
                if (alive) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t in = (uint32_t)(i & 3) * 32u;
                        umma_bf16(tmem + (uint32_t)st.slot * 256u, qd + (((uint32_t)(i >> 2) * kHalfBytes + in) >> 4),
                                  kd + (((uint32_t)(i >> 2) * 2u * kHalfBytes + in) >> 4), idesc, i ? 1u : 0u);
                    }
                }
                umma_commit(c.s_full(st.slot));
                umma_commit(c.q_empty(qt.slot));
            }
            __syncwarp();
            st.next(2);
            qt.next(Ring<D>::kQ);
        }
        kt.next(Ring<D>::kK / 2);
    } while (walk_next(p, w));
    if (one) {
        umma_commit(c.fin(0));
        mbar_drain_bounded(c.fin(0), 0u);
    }
}

// Adds to acc the weights of 32 tokens for the thread's row; kMasked: of the first
// `seen` ones.
template <bool kMasked>
__device__ __forceinline__ void weigh_row32(const uint32_t *s, float c, float l, int seen, float2 *acc)
{
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), make_float2(c, c),
                              make_float2(l, l));
        if (kMasked) {
            x.x = 2 * j < seen ? x.x : -INFINITY;
            x.y = 2 * j + 1 < seen ? x.y : -INFINITY;
        }
        acc[j] = __fadd2_rn(acc[j], make_float2(ex2_approx(x.x), ex2_approx(x.y)));
    }
}

// The weights of columns 64 group .. 64 group + 63 of every item; at its end the
// warps' sums by way of the item's K, which has been used, and the masses.  (TMEM is
// read 32 columns at a time: 16 at a time took a fifth longer in all.)
template <int D>
__device__ void add_up_wide(const MassParams &p, const Ctx<D> &c, uint32_t tmem, int group)
{
    const int lane = threadIdx.x & 31, quad = threadIdx.x / 32 % 4, row = 32 * quad + lane;
    const int tok = row / p.group, tok0 = 32 * quad / p.group;       // query token of the row, and of the warp's first
    const uint32_t s_mine = tmem + ((uint32_t)(32 * quad) << 16) + 64u * (uint32_t)group;
    const int n_mine = row < p.tpt * p.group ? p.n_q : 0;            // the row's query tokens lie before this
    Walk w;
    Turn kt, st;
    bool alive = true;
    if (!walk_first(p, w))
        return;
    do {
        const int tokens = min(kWide, w.L - w.t0), mine = tokens - 64 * group;      // of the warp's 64
        float2 acc[32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
            acc[j] = make_float2(0.f, 0.f);
        // the row's query token in the next block, and the log-sum-exp, read a block
        // ahead; a row behind the last is out
        int i = w.begin * p.tpt + tok;
        const float *src = p.lse + w.b * p.lse_request + i * p.lse_token + w.g * p.group + row - tok * p.group;
        float lse = i < n_mine ? *src : -INFINITY;
        // blocks from which on all of the warp's rows see all of its tokens
        const int rest = w.t0 + 64 * group + 63 - w.past - tok0;
        const int plain = rest > 0 ? (rest + p.tpt - 1) / p.tpt : 0;
#pragma unroll 1
        for (int k = w.begin; k < w.end; ++k) {
            const float l = lse_offset(lse);
            const bool row_in = l != kRowOut;
            i += p.tpt;
            src += p.tpt * p.lse_token;
            lse = i < n_mine ? *src : -INFINITY;
            alive = __all_sync(0xffffffffu, alive && c.wait(c.s_full(st.slot), st.parity));
            if (alive && mine > 0) {
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t s[32];
                    __syncwarp();            // the load is the whole warp's, and lanes without a row skip a half
                    tmem_ld32_nowait(s_mine + 256u * (uint32_t)st.slot + 32u * h, s);
                    tmem_wait_ld();
                    if (h)
                        leave(c.s_empty(st.slot));
                    // (no use of a score moves before its wait: the condition passes through it)
                    int in = row_in;
                    asm volatile("" : "+r"(in)::"memory");
                    // (a zero query of a row that is none and an infinite key make no number)
                    if (in) {
                        if (k >= plain)
                            weigh_row32<false>(s, p.scale_log2, l, 32, acc + 16 * h);
                        else                 // tokens up to past + the row's query token
                            weigh_row32<true>(s, p.scale_log2, l, w.past + i - p.tpt + 1 - w.t0 - 64 * group - 32 * h,
                                              acc + 16 * h);
                    }
                }
            } else {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(c.s_empty(st.slot));
            }
            st.next(2);
        }
        // over the warp's rows: halves of the columns change hands, until a lane has two
        // (columns 2 r, 2 r + 1, the bits of r being the lane's from the top)
        const uint32_t full = 0xffffffffu;
#pragma unroll
        for (int o = 16, n = 16; o; o >>= 1, n >>= 1)
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const bool up = lane & o;
                const float2 send = up ? acc[j] : acc[j + n], keep = up ? acc[j + n] : acc[j];
                acc[j] = make_float2(keep.x + __shfl_xor_sync(full, send.x, o), keep.y + __shfl_xor_sync(full, send.y, o));
            }
        const uint32_t sums = c.k_slot(2 * kt.slot);     // [4 warps][256 tokens]
        if (mine > 0)
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sums + (uint32_t)(quad * kWide + 64 * group + 2 * lane) * 4u),
                         "f"(acc[0].x), "f"(acc[0].y)
                         : "memory");
        named_barrier(1u, 512u);
        if (threadIdx.x < tokens) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[i]) : "r"(sums + (uint32_t)(i * kWide + threadIdx.x) * 4u));
            const int t = w.t0 + threadIdx.x;
            const bool inside = (uint32_t)p.block_table[(int64_t)w.b * p.max_pages + t / p.page_size] <
                                (uint32_t)p.num_pages;
            const float sum = inside ? (v[0] + v[1]) + (v[2] + v[3]) : 0.f;
            if (!w.whole(p))
                p.pieces[(int64_t)piece_of(p, w) * kWide + threadIdx.x] = sum;
            else
                p.mass.out[w.b * p.mass.out_request + w.g * p.mass.out_head + t] =
                    p.mass.in ? fmaf(p.decay, p.mass.in[w.b * p.mass.in_request + w.g * p.mass.in_head + t], sum) : sum;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(c.k_empty(kt.slot));
        kt.next(Ring<D>::kK / 2);
    } while (walk_next(p, w));
}

template <int D, bool kManyRows>
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
            mbar_init(c.k_empty(s), kManyRows ? 16u : 1u);   // the weights' warps, or the MMAs
        }
        for (int s = 0; s < Ring<D>::kQ; ++s) {
            mbar_init(c.q_full(s), 1u);
            mbar_init(c.q_empty(s), kManyRows ? 1u : 18u);   // the issuers' MMAs, and the warps that read the log-sum-exps
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(c.s_full(i), 1u);
            mbar_init(c.s_empty(i), kManyRows ? 16u : 4u);
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
    if (kManyRows) {
        if (warp < kKWarp) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWeightRegs));
            add_up_wide<D>(p, c, tmem, warp / 4);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
            if (warp == kKWarp) {
                copy_k_wide<D>(&tm_k, p, c);
                check_lens(p);
            } else if (warp == kQWarp) {
                copy_q_wide<D>(&tm_q, p, c);
            } else if (warp == kMmaWarp) {
                issue_wide<D>(p, c, tmem);
            }
        }
    } else if (warp == kKWarp) {
        copy_k<D>(&tm_k, p, c);
        check_lens(p);
    } else if (warp == kQWarp) {
        copy_q<D>(&tm_q, p, c);
    } else if (warp >= kMmaWarp) {
        issue<D>(p, c, tmem, warp - kMmaWarp);
    } else {
        add_up<D>(p, c, tmem, warp / 4);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        tmem_dealloc(tmem, kTmemCols);
}

// Items that ranges cut: the sums of the pieces, in the order of the blocks.
// CTA c looks at the cut before range c and does an item's first.
__global__ void __launch_bounds__(kWide) shkv_mass_join_kernel(const __grid_constant__ MassParams p)
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
    const int tokens = p.item_tokens, items = (p.lens[b] + tokens - 1) / tokens;
    const int g = (item - p.item0[b]) / items, t = (item - p.item0[b]) % items * tokens + u;
    if (u >= tokens || t >= p.lens[b])
        return;
    float sum = p.pieces[(int64_t)(2 * (c - 1) + 1) * (kWide) + u];
    for (int i = c; i < p.num_ctas && p.cut_item[i] == item; ++i)
        sum += p.pieces[(int64_t)(2 * i) * (kWide) + u];
    p.mass.out[b * p.mass.out_request + g * p.mass.out_head + t] =
        p.mass.in ? fmaf(p.decay, p.mass.in[b * p.mass.in_request + g * p.mass.in_head + t], sum) : sum;
}

}  // namespace

// tm_k: a column half of one page of one KV head; tm_q: a column half of a block's rows.
cudaError_t launch_mass(const CUtensorMap &tm_k, const CUtensorMap &tm_q, const MassParams &p, bool pieces,
                        cudaStream_t stream)
{
    const bool wide = mass_wide(p.blocks);
    auto kern = p.head_dim == 64 ? (wide ? shkv_mass_kernel<64, true> : shkv_mass_kernel<64, false>)
                                 : (wide ? shkv_mass_kernel<128, true> : shkv_mass_kernel<128, false>);
    const uint32_t smem = p.head_dim == 64 ? Ring<64>::kBytes : Ring<128>::kBytes;
    // a build whose launch has other registers than setmaxnreg hands out could wait
    // for some forever: it is refused
    static std::atomic<int> known[2];
    int regs = (int)kLaunchRegs;
    cudaError_t e = wide ? kernel_registers(kern, known[p.head_dim == 64], &regs) : cudaSuccess;
    if (e == cudaSuccess && regs != (int)kLaunchRegs)
        e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = launch_pdl(kern, p.num_ctas, kThreads, smem, stream, tm_k, tm_q, p);
    if (e == cudaSuccess && pieces)
        e = launch_pdl(shkv_mass_join_kernel, p.num_ctas - 1, kWide, 0u, stream, p);
    return e;
}

}  // namespace shkv
