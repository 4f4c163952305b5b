// q8_chunk.cu -- causal attention of ragged chunks of new tokens over the
// 8-bit KV cache on the 5th-generation tensor cores.
//
// A query tile is TPT = floor(128 / G) new tokens x the G query heads of one
// KV head, 128 MMA rows (row r = i * G + j).  A unit is two consecutive tiles
// X = A, B of one (request, KV head); its 128-key stages of K and V are loaded
// once for both.  Persistent CTAs take contiguous ranges of equal cost over
// all units' stages; a unit that straddles a cut leaves normalised partials
// and log-sum-exps that a second kernel joins (few units, many rows: joined
// by all SMs at once).  Per stage and tile:
//
//   S_X[r, key]  = sum_d (qh + ql)[r, d] k8[key, d]               kind::f8f6f4
//   x_X[r, key]  = S_X 2^eq[r] 2^ek[key] scale log2(e)
//   w_X[r, key]  = 2^(x - m[r] + 7),  m[r] a running maximum of x + ev
//   P_X[r, key]  = w 2^ev[key]                                    fp16, over S in TMEM
//   O_X[r, d]   += sum_key P_X[r, key] v8[key, d]                 kind::f16
//   l[r]        += sum_key w_X[r, key]
//   out = O / l,   lse = ln2 * (m - 7 + log2(l))
//
// The query's two e4m3 terms are as in the stacked kernel (q8_decode.cu); the
// factors of a key are column factors here, read as vectors from shared
// memory.  V's codes are exact in fp16 as they are.  With the key's V exponent
// in m, P is relative to the row's largest weight times value scale: fp16's
// least step, 2^-24, is 2^-31 of that, so 2^20 keys whose P rounds to zero are
// 2^-12 of the sum's largest term.  (P relative to the largest weight alone,
// with V's scales apart by 2^s, loses up to n 2^(s - 32): a first key of much
// weight and little value, as an attention sink is, then lost 10% of a sum over
// 131072 keys at s = 12.)  l is in fp32's range while no V exponent is above 60
// (then the row's largest w is 2^-61 or more) and no w above 2^67.  From the
// first stage on that holds the one (for the whole piece) or the other (for its
// warp), l is summed from a second exponential, relative to a running maximum of
// x of its own; a key whose V is zero stays out of m at all times.  That takes
// values above 2^60, values all below 2^-51, or a key that leads by 2^60 and has
// next to no value; such a stage takes about twice the time.  Sums and O are
// fp32.
//
// As in the bf16 kernel, a stage whose scores are all visible is
// exponentiated against the running maximum without taking its own.  A quarter
// of its sum of w, times the stage's largest value scale, bounds each P in the
// quarter: a row for which that leaves fp16's range sends its warp through the
// exact path.  (Looking at P itself, by a sum with ev in the exponent and l by
// factors 2^-ev or by a packed maximum, costs an instruction a pair and, in the
// first form, a vector load: turns 338 us, the document 1.80 ms, against 317 us
// and 1.59 ms; the exact path it is spared is 2% of the time.)  Three quarters
// of the scores are loaded at first, the last over the third: with all of them
// in registers the kernel spilled more (324 us, 1.77 ms).  Its load and wait stay
// next to each other: nothing may touch the registers between them.
//
// Roles (512 threads): warps 0-3 softmax of tile A, 4-7 of tile B (row = TMEM
// lane), 8 QK issuer, 9 PV issuer, 10 producer of K, 11 producer of V and its
// scale bytes, 12-15 V conversion, one key a thread: also the column factors.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "launch.cuh"
#include "q8.cuh"
#include "q8_chunk.cuh"
#include "q8_wait.cuh"
#include "shkv_device.cuh"

namespace shkv {

namespace {

constexpr int kKT = 128;                 // keys per stage
constexpr int kThreads = 512;
constexpr int kQkWarp = 8, kPvWarp = 9, kKWarp = 10, kVWarp = 11, kConvWarp0 = 12, kConvWarps = 4;
constexpr int kGroupWarps = 4;           // softmax warps per tile
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 2.f;      // in the exact path m moves where it lags the maximum by more
constexpr float kPLog2 = 7.f;            // P at the running maximum
constexpr uint32_t kApart = 1, kMayLead = 2;   // a stage's needs: see the top; a key of it may lead by 2^60
constexpr float kMaxPart = 65504.f;      // fp16's largest: bound of a stage's P taken without its maximum
constexpr int kMaxEv = 60;               // a V exponent above this needs a reference of l's own
constexpr float kMaxLead = 60.f;         // ... as does an x this far above m
constexpr int kKS = 3, kVS = 3;          // ring slots of 16 KB (K) and 32 KB (V)
constexpr uint32_t kKSlotBytes = kKT * 128;
constexpr uint32_t kVSlotBytes = 2 * kKT * 128;
constexpr uint32_t kQTermBytes = 128 * 128;      // one e4m3 term of a tile [128 rows][128 B]
constexpr uint32_t kSoftmaxRegs = 200, kOtherRegs = 56;
static_assert(kSoftmaxRegs * 256 + kOtherRegs * 256 == 128 * kThreads, "register split");

__device__ __forceinline__ uint32_t col_s(int x) { return (uint32_t)(x * 128); }
__device__ __forceinline__ uint32_t col_o(int x) { return (uint32_t)(256 + x * 128); }

struct Smem {
    uint32_t qtile, kring, vring, scales, factor, evs, pfactor, info, bars, misc, tslot, total;
};

// Query tiles [tile][qh | ql][128 rows][128 B], K ring, V ring (slots
// [half][128 keys][128 B], the codes in the upper half until they are
// converted), all 128-byte swizzled; per V slot its scale bytes, the keys'
// score factors, V exponents and factors of P, and four words (valid pages,
// what its V exponents need, the largest sum of w that needs no look at the
// maximum).
__host__ __device__ inline Smem smem_layout()
{
    Smem u;
    u.qtile = 0;
    u.kring = u.qtile + 4 * kQTermBytes;
    u.vring = u.kring + kKS * kKSlotBytes;
    u.scales = u.vring + kVS * kVSlotBytes;
    u.factor = u.scales + kVS * 2 * kKT;
    u.evs = u.factor + kVS * kKT * 4;
    u.pfactor = u.evs + kVS * kKT * 4;
    u.info = u.pfactor + kVS * kKT * 4;
    u.bars = u.info + kVS * 16;
    u.misc = u.bars + (uint32_t)(2 * kKS + 3 * kVS + 9) * 8u;
    u.tslot = u.misc + 8;
    u.total = u.misc + 16 + 1024;
    return u;
}

struct Ctx {
    uint8_t *smem;
    uint32_t base;
    Smem lay;
    volatile uint32_t *abort_flag;
};

__device__ __forceinline__ uint32_t bar_at(const Ctx &c, int i) { return c.base + c.lay.bars + 8u * i; }
__device__ __forceinline__ uint32_t full_k(const Ctx &c, int s) { return bar_at(c, s); }
__device__ __forceinline__ uint32_t empty_k(const Ctx &c, int s) { return bar_at(c, kKS + s); }
__device__ __forceinline__ uint32_t full_v(const Ctx &c, int s) { return bar_at(c, 2 * kKS + s); }
__device__ __forceinline__ uint32_t conv_v(const Ctx &c, int s) { return bar_at(c, 2 * kKS + kVS + s); }
__device__ __forceinline__ uint32_t empty_v(const Ctx &c, int s) { return bar_at(c, 2 * kKS + 2 * kVS + s); }
constexpr int kBar0 = 2 * kKS + 3 * kVS;
__device__ __forceinline__ uint32_t s_full(const Ctx &c, int x) { return bar_at(c, kBar0 + x); }
__device__ __forceinline__ uint32_t p_full(const Ctx &c, int x) { return bar_at(c, kBar0 + 2 + x); }
__device__ __forceinline__ uint32_t pv_done(const Ctx &c, int x) { return bar_at(c, kBar0 + 4 + x); }
__device__ __forceinline__ uint32_t q_ready(const Ctx &c) { return bar_at(c, kBar0 + 6); }
__device__ __forceinline__ uint32_t q_free(const Ctx &c) { return bar_at(c, kBar0 + 7); }
__device__ __forceinline__ uint32_t fin_b(const Ctx &c) { return bar_at(c, kBar0 + 8); }
__device__ __forceinline__ uint32_t k_slot(const Ctx &c, int s) { return c.base + c.lay.kring + (uint32_t)s * kKSlotBytes; }
__device__ __forceinline__ uint32_t v_slot(const Ctx &c, int s) { return c.base + c.lay.vring + (uint32_t)s * kVSlotBytes; }
__device__ __forceinline__ uint32_t ring_par(int k, int n) { return (uint32_t)((k / n) & 1); }

// A piece of a unit: its key stages [s0, s1).
struct Piece {
    int u, b, g;
    int L, prefix;               // request length, cached tokens before the new ones
    int i0[2], ntok[2];          // first new token and new tokens of tiles A and B (B may be empty)
    int nst[2], nst_all;         // key stages each tile attends, and the larger
    int s0, s1;
};

__device__ __forceinline__ void set_unit(const Q8ChunkParams &p, Piece &t)
{
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.units[mid] <= t.u)
            lo = mid;
        else
            hi = mid;
    }
    t.b = lo;
    const int pairs = (p.units[lo + 1] - p.units[lo]) / p.hkv;
    const int rem = t.u - p.units[lo];
    t.g = rem / pairs;
    const int tp = rem - t.g * pairs;
    const int n = p.n_q[lo];
    t.L = p.lens[lo];
    t.prefix = t.L - n;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        t.i0[x] = (2 * tp + x) * p.tpt;
        t.ntok[x] = max(0, min(p.tpt, n - t.i0[x]));
        t.nst[x] = t.ntok[x] > 0 ? (t.prefix + t.i0[x] + t.ntok[x] + kKT - 1) / kKT : 0;
    }
    t.nst_all = max(t.nst[0], t.nst[1]);
}

// The CTA's pieces in order; false when there are no more.
__device__ __forceinline__ bool first_piece(const Q8ChunkParams &p, Piece &t)
{
    const int c = blockIdx.x;
    t.u = p.cut_unit[c];
    t.s0 = p.cut_stage[c];
    if (t.u > p.cut_unit[c + 1] || (t.u == p.cut_unit[c + 1] && t.s0 >= p.cut_stage[c + 1]))
        return false;
    set_unit(p, t);
    t.s1 = t.u == p.cut_unit[c + 1] ? p.cut_stage[c + 1] : t.nst_all;
    return true;
}

__device__ __forceinline__ bool next_piece(const Q8ChunkParams &p, Piece &t)
{
    const int c = blockIdx.x;
    ++t.u;
    t.s0 = 0;
    if (t.u > p.cut_unit[c + 1] || (t.u == p.cut_unit[c + 1] && p.cut_stage[c + 1] == 0))
        return false;
    set_unit(p, t);
    t.s1 = t.u == p.cut_unit[c + 1] ? p.cut_stage[c + 1] : t.nst_all;
    return true;
}

// Partial slot of the piece of unit u that CTA c holds: 0 if it opens the CTA's range.
__device__ __forceinline__ int piece_slot(const Q8ChunkParams &p, int c, int u)
{
    return 2 * c + (u == p.cut_unit[c] ? 0 : 1);
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------
// One lane copies one page: a box of P rows x 128 bytes (at head_dim 64 the
// upper half of the rows is filled with zeros).  The V warp also copies the
// page's 2P scale bytes and publishes the stage's valid pages.
template <bool kIsV>
__device__ void chunk_producer(const CUtensorMap *tm, const Q8ChunkParams &p, const Ctx &c)
{
    constexpr int S = kIsV ? kVS : kKS;
    const int lane = threadIdx.x & 31;
    const int P = p.page_size, RB = kKT / P;
    const uint64_t pol = l2_evict_first_policy();
    if (lane == 0)
        prefetch_tensormap(tm);
    bool alive = true;
    int kbase = 0, last_issued = -1;
    Piece t;
#pragma unroll 1
    for (bool more = first_piece(p, t); more; more = next_piece(p, t)) {
        if (kIsV && lane == 0 && __ldg(p.seq_lens + t.b) != t.L)
            atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
        const int npages = (t.L + P - 1) / P;
        const int32_t *row = p.block_table + (int64_t)t.b * p.max_pages;
        auto entry = [&](int j) {                        // the lane's page of stage j
            const int pg = j * RB + lane;
            return lane < RB && j < t.s1 && pg < npages ? __ldg(row + pg) : -1;
        };
        int nxt = entry(t.s0);
#pragma unroll 1
        for (int j = t.s0; j < t.s1; ++j) {
            const int k = kbase + j - t.s0, slot = k % S;
            const int id = nxt;
            nxt = entry(j + 1);                          // read one stage ahead
            bool ok = true;
            if (alive && lane == 0)
                ok = q8_wait<true>(kIsV ? empty_v(c, slot) : empty_k(c, slot), ring_par(k, S) ^ 1u, c.abort_flag, p.err);
            alive = alive && __all_sync(0xffffffffu, ok);
            const bool inside = lane < RB && j * RB + lane < npages;
            const bool valid = inside && id >= 0 && id < p.num_pages;
            const uint32_t mask = __ballot_sync(0xffffffffu, valid);
            const uint32_t bar = kIsV ? full_v(c, slot) : full_k(c, slot);
            if (kIsV && alive && inside && !valid)
                atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
            if (alive && lane == 0) {
                if (kIsV)
                    reinterpret_cast<volatile uint32_t *>(c.smem + c.lay.info)[slot * 4] = mask;
                mbar_arrive_expect_tx(bar, (uint32_t)__popc(mask) * (uint32_t)P * (kIsV ? 130u : 128u));
            }
            __syncwarp();
            if (alive && valid) {
                const int unit = id * p.hkv + t.g;
                tma_load_2d((kIsV ? v_slot(c, slot) + kKT * 128u : k_slot(c, slot)) + (uint32_t)(lane * P) * 128u, tm, 0,
                            unit * P, bar, pol);
                if (kIsV)
                    bulk_load(c.base + c.lay.scales + (uint32_t)(slot * 2 * kKT + lane * 2 * P),
                              p.scales + (int64_t)unit * 2 * P, 2u * (uint32_t)P, bar);
            }
            if (alive)
                last_issued = k;
            __syncwarp();
        }
        kbase += t.s1 - t.s0;
    }
    if (!alive && lane == 0)
        for (int k = last_issued - S + 1; k <= last_issued; ++k)
            if (k >= 0)
                mbar_drain_bounded(kIsV ? full_v(c, k % S) : full_k(c, k % S), ring_par(k, S));
}

// ---------------------------------------------------------------------------
// V conversion and the keys' factors, one key a thread
// ---------------------------------------------------------------------------
__device__ void chunk_convert(const Q8ChunkParams &p, const Ctx &c)
{
    const int t = threadIdx.x - kConvWarp0 * 32, lane = t & 31;
    const int P = p.page_size, log2P = 31 - __clz(P);
    const int groups = p.head_dim / 64;                  // 64-column halves
    bool alive = true;
    int kbase = 0;
    Piece u;
#pragma unroll 1
    for (bool more = first_piece(p, u); more; more = next_piece(p, u)) {
        bool wide = false;
#pragma unroll 1
        for (int j = u.s0; j < u.s1; ++j) {
            const int k = kbase + j - u.s0, slot = k % kVS;
            bool ok = false;
            if (alive)
                ok = q8_wait<false>(full_v(c, slot), ring_par(k, kVS), c.abort_flag, p.err);
            alive = __all_sync(0xffffffffu, ok);
            if (alive) {
                volatile uint32_t *info = reinterpret_cast<volatile uint32_t *>(c.smem + c.lay.info) + slot * 4;
                const uint32_t mask = info[0];
                const int n = u.L - j * kKT;
                const uint8_t *sc = c.smem + c.lay.scales + slot * 2 * kKT;
                uint32_t top, low;
                // the stage's largest and least V scale byte (NaN rows aside;
                // zero rows have the least), by each warp for itself
                {
                    const int t4 = 4 * lane;
                    const uint32_t w = *reinterpret_cast<const volatile uint32_t *>(
                        sc + ((t4 >> log2P) << (log2P + 1)) + P + (t4 & (P - 1)));
                    const int in = ((mask >> (t4 >> log2P)) & 1u) ? n - t4 : 0;
                    top = 0;
                    low = 255;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t b = (w >> (8 * i)) & 0xffu;
                        top = max(top, i < in && b != 255u ? b : 0u);
                        low = min(low, i < in ? b : 255u);
                    }
                    top = __reduce_max_sync(0xffffffffu, top);
                    low = __reduce_min_sync(0xffffffffu, low);
                    wide = wide || top > 127u + kMaxEv;
                }
                const bool valid = t < n && ((mask >> (t >> log2P)) & 1u);
                const uint8_t *mine = sc + ((t >> log2P) << (log2P + 1)) + (t & (P - 1));
                const int kb = *reinterpret_cast<const volatile uint8_t *>(mine);
                const int vb = *reinterpret_cast<const volatile uint8_t *>(mine + P);
                // a NaN row of V counts as zero and makes its key's scores NaN
                // instead, so that only rows that attend it see it
                const uint8_t *codes = c.smem + c.lay.vring + (uint32_t)slot * kVSlotBytes + (uint32_t)t * 128u + kKT * 128;
                bool zero = false;
                if (valid && vb == 0) {                  // a row of zeros, or one of tiny values
                    uint32_t any = 0;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {        // (at head_dim 64 the upper half is zero)
                        const uint4 w = reinterpret_cast<const uint4 *>(codes)[i];
                        any |= w.x | w.y | w.z | w.w;
                    }
                    zero = (any & 0x7f7f7f7fu) == 0u;
                }
                const bool live = valid && vb != 255 && !zero;
                const float nan = __uint_as_float(0x7fc00000u);
                reinterpret_cast<float *>(c.smem + c.lay.factor)[slot * kKT + t] =
                    !valid ? 0.f : vb == 255 ? nan : q8_scale((uint32_t)kb) * p.scale_log2;
                // (where V is zero P is zero, and its key stays out of P's
                // reference: the weights of the others keep their bits)
                reinterpret_cast<float *>(c.smem + c.lay.evs)[slot * kKT + t] = live ? (float)(vb - 127) : -INFINITY;
                reinterpret_cast<float *>(c.smem + c.lay.pfactor)[slot * kKT + t] = live ? q8_scale((uint32_t)vb) : 0.f;
                if (t == 0) {
                    info[1] = wide ? kApart : low < 127u - (uint32_t)kMaxLead ? kMayLead : 0u;
                    // 65504 / 2^top, 2^67 at most
                    info[2] = __float_as_uint(kMaxPart) + ((127u - max(top, 127u - 51u)) << 23);
                }
                uint8_t *row = c.smem + c.lay.vring + (uint32_t)slot * kVSlotBytes + (uint32_t)t * 128u;
                // (the conversion instruction: the stacked kernel's integer
                // moves are 4% of the kernel slower here)
                // the codes of half h are read before its fp16 values are
                // written; only half 1's land on codes, and those were read
#pragma unroll 1
                for (int h = 0; h < groups; ++h) {
                    uint4 raw[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        raw[i] = live ? *reinterpret_cast<const uint4 *>(row + kKT * 128 + (((4 * h + i) ^ (t & 7)) << 4))
                                      : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                        uint32_t o[8];
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2(
                                (__nv_fp8x2_storage_t)(w[v >> 1] >> (16 * (v & 1))), __NV_E4M3);
                            o[v] = (uint32_t)x.x | (uint32_t)x.y << 16;
                        }
                        uint8_t *dst = row + h * (kKT * 128);
                        *reinterpret_cast<uint4 *>(dst + (((2 * i) ^ (t & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(dst + (((2 * i + 1) ^ (t & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(conv_v(c, slot));
        }
        kbase += u.s1 - u.s0;
    }
}

// ---------------------------------------------------------------------------
// MMA issuers (one lane each)
// ---------------------------------------------------------------------------
constexpr uint32_t idesc_of(int M, int N, bool a_mn, bool b_mn)   // formats 0: e4m3 (f8f6f4), fp16 (f16)
{
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma_f8(uint32_t d_taddr, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_taddr),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// A from TMEM: 128 lanes (rows) x K columns of packed fp16 pairs.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_taddr, uint32_t a_taddr, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_taddr),
                 "r"(a_taddr), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// S_X of each tile that attends the stage, once its previous PV has read the
// P written over S_X.
__device__ void chunk_qk(const Q8ChunkParams &p, const Ctx &c, uint32_t tmem)
{
    constexpr uint32_t idesc = idesc_of(128, kKT, false, false);
    const int steps = p.head_dim / 32;
    const uint64_t qd0 = umma_sdesc_sw128(c.base + c.lay.qtile, 16u, 1024u);
    const uint64_t kd0 = umma_sdesc_sw128(k_slot(c, 0), 16u, 1024u);
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive)
            alive = q8_wait<true>(bar, parity, c.abort_flag, p.err);
    };
    int kbase = 0, seg = 0, done[2] = {0, 0};            // stages each tile has attended
    Piece t;
#pragma unroll 1
    for (bool more = first_piece(p, t); more; more = next_piece(p, t)) {
        wait(q_ready(c), (uint32_t)(seg & 1));
#pragma unroll 1
        for (int j = t.s0; j < t.s1; ++j) {
            const int k = kbase + j - t.s0, slot = k % kKS;
            const uint64_t kd = kd0 + (((uint32_t)slot * kKSlotBytes) >> 4);
            wait(full_k(c, slot), ring_par(k, kKS));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (j >= t.nst[x])
                    continue;
                if (done[x] > 0)
                    wait(pv_done(c, x), (uint32_t)((done[x] - 1) & 1));
                ++done[x];
                if (alive) {
                    tc_fence_after();
                    const uint64_t qd = qd0 + ((2u * (uint32_t)x * kQTermBytes) >> 4);
                    // (rolled, as in q8_decode.cu)
#pragma unroll 1
                    for (int i = 0; i < steps; ++i) {
                        umma_f8(tmem + col_s(x), qd + (uint64_t)(2 * i), kd + (uint64_t)(2 * i), idesc, i ? 1u : 0u);
                        umma_f8(tmem + col_s(x), qd + (kQTermBytes >> 4) + (uint64_t)(2 * i), kd + (uint64_t)(2 * i),
                                idesc, 1u);
                    }
                }
                umma_commit(s_full(c, x));
            }
            umma_commit(empty_k(c, slot));
        }
        umma_commit(q_free(c));
        kbase += t.s1 - t.s0;
        ++seg;
    }
    umma_commit(fin_b(c));
    mbar_drain_bounded(fin_b(c), 0u);
}

__device__ void chunk_pv(const Q8ChunkParams &p, const Ctx &c, uint32_t tmem)
{
    const uint32_t idesc = p.head_dim == 64 ? idesc_of(128, 64, false, true) : idesc_of(128, 128, false, true);
    const uint64_t vd0 = umma_sdesc_sw128(v_slot(c, 0), (uint32_t)(kKT * 128), 1024u);
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive)
            alive = q8_wait<true>(bar, parity, c.abort_flag, p.err);
    };
    int kbase = 0, done[2] = {0, 0};
    Piece t;
#pragma unroll 1
    for (bool more = first_piece(p, t); more; more = next_piece(p, t)) {
#pragma unroll 1
        for (int j = t.s0; j < t.s1; ++j) {
            const int k = kbase + j - t.s0, slot = k % kVS;
            const uint64_t vd = vd0 + (((uint32_t)slot * kVSlotBytes) >> 4);
            wait(conv_v(c, slot), ring_par(k, kVS));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (j >= t.nst[x])
                    continue;
                wait(p_full(c, x), (uint32_t)(done[x] & 1));
                ++done[x];
                if (alive) {
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < kKT / 16; ++ks)
                        umma_f16_ts(tmem + col_o(x), tmem + col_s(x) + (uint32_t)(ks * 8), vd + (uint64_t)(ks * 128), idesc,
                                    (j == t.s0 && ks == 0) ? 0u : 1u);
                }
                umma_commit(pv_done(c, x));
            }
            umma_commit(empty_v(c, slot));
        }
        kbase += t.s1 - t.s0;
    }
    umma_commit(fin_b(c));
    mbar_drain_bounded(fin_b(c), 0u);
}

// ---------------------------------------------------------------------------
// softmax warps of tile x: thread r = MMA row r = (new token i0 + r / G, head r % G)
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max3f(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The warp's 32 rows of the query as two e4m3 terms in their tile; returns the
// scale of this lane's row (a power of two).  src: this lane's row, null for a
// padding row (zeros).  D / 8 neighbouring lanes take a row, 8 columns each,
// and the raw row is copied to where its terms will lie (its 2 D bytes are
// theirs): all 32 rows are in flight at once and no lane reads what another
// copied.  A row a lane through registers, 8 loads in flight, took 10K cycles a
// piece, four rows in flight by neighbouring lanes 15K.
__device__ __forceinline__ float stage_rows(const Ctx &c, const __nv_bfloat16 *src, const __nv_bfloat16 *any, int D, int x,
                                            int r0)
{
    const int lane = threadIdx.x & 31;
    const int shift = D == 64 ? 3 : 4;                   // log2 of a row's lanes
    const int sub = lane & ((1 << shift) - 1), rsub = lane >> shift, rows = 32 >> shift;
    const uint32_t tile = c.lay.qtile + 2u * (uint32_t)x * kQTermBytes;
    // a row's columns 8 sub .. 8 sub + 7 in the first term's tile
    auto place = [&](int row) { return tile + (uint32_t)(row * 128 + (((sub >> 1) ^ (row & 7)) << 4) + (sub & 1) * 8); };
#pragma unroll 1
    for (int i = 0; i < D / 8; ++i) {                    // `rows` rows at a time
        const __nv_bfloat16 *row = reinterpret_cast<const __nv_bfloat16 *>(
            __shfl_sync(0xffffffffu, (unsigned long long)src, i * rows + rsub));
        const uint32_t bytes = row ? 8u : 0u;            // (0: zeros, and nothing is read)
        const uint8_t *from = reinterpret_cast<const uint8_t *>((row ? row : any) + sub * 8);
        const uint32_t to = c.base + place(r0 + i * rows + rsub);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to + kQTermBytes), "l"(from + 8), "r"(bytes)
                     : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    int mine = 0;                                        // scale byte of this lane's row, 255: not finite
#pragma unroll 1
    for (int i0 = 0; i0 < D / 8; i0 += 4) {              // four at a time, their chains of shuffles and conversions side by side
        uint8_t *to[4];
        uint32_t w[4][4], a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            to[i] = c.smem + place(r0 + (i0 + i) * rows + rsub);
            const uint2 v0 = *reinterpret_cast<const uint2 *>(to[i]), v1 = *reinterpret_cast<const uint2 *>(to[i] + kQTermBytes);
            w[i][0] = v0.x;
            w[i][1] = v0.y;
            w[i][2] = v1.x;
            w[i][3] = v1.y;
            const uint32_t m = __vmaxu2(__vmaxu2(v0.x & 0x7fff7fffu, v0.y & 0x7fff7fffu),
                                        __vmaxu2(v1.x & 0x7fff7fffu, v1.y & 0x7fff7fffu));
            a[i] = max(m & 0xffffu, m >> 16);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = max(a[i], __shfl_xor_sync(0xffffffffu, a[i], o));
        }
        if (D != 64) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = max(a[i], __shfl_xor_sync(0xffffffffu, a[i], 8));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool bad = a[i] >= 0x7f80u;            // an infinity or a NaN: the row's scores are NaN
            const int byte = bad ? 255 : max((int)((a[i] + 0x1fu) >> 7) - 8, 0);
            const float inv = __uint_as_float((uint32_t)(254 - min(byte, 253)) << 23);
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // (scaled values are exact in fp16 down to its subnormals, 2^-33 of the row's largest)
                const __half2 f16 = __floats2half2_rn(__uint_as_float(w[i][k] << 16) * inv,
                                                      __uint_as_float(w[i][k] & 0xffff0000u) * inv);
                const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(f16, __NV_SATFINITE, __NV_E4M3);
                const __half2 rest = __hsub2(f16, __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
                const __nv_fp8x2_storage_t l = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E4M3);
                hi[k >> 1] = (k & 1) ? hi[k >> 1] | ((uint32_t)h << 16) : h;
                lo[k >> 1] = (k & 1) ? lo[k >> 1] | ((uint32_t)l << 16) : l;
            }
            const uint32_t n = 0x7f7f7f7fu;
            *reinterpret_cast<uint2 *>(to[i]) = bad ? make_uint2(n, n) : make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(to[i] + kQTermBytes) = bad ? make_uint2(n, n) : make_uint2(lo[0], lo[1]);
            const int got = __shfl_sync(0xffffffffu, byte, (lane & (rows - 1)) << shift);
            if ((lane >> (5 - shift)) == i0 + i)
                mine = got;
        }
    }
    return mine == 255 ? 1.f : q8_scale((uint32_t)mine);
}

__device__ void chunk_softmax(const Q8ChunkParams &p, const Ctx &c, uint32_t tmem, int x)
{
    const int r = threadIdx.x - x * 128;
    const int lane = r & 31, warp = r >> 5;
    const int ti = r / p.group, tj = r - ti * p.group;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const uint32_t orow = tmem + lane_base + col_o(x);
    const uint32_t srow = tmem + lane_base + col_s(x);
    const int P = p.page_size, D = p.head_dim;
    const uint32_t all_pages = (1u << (kKT / P)) - 1u;
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        bool ok = false;
        if (alive)
            ok = q8_wait<false>(bar, parity, c.abort_flag, p.err);
        alive = __all_sync(0xffffffffu, ok) && alive;
        return alive;
    };
    int kbase = 0, seg = 0, done = 0;                    // done: stages this tile has attended
    Piece t;
#pragma unroll 1
    for (bool more = first_piece(p, t); more; more = next_piece(p, t)) {
        const bool row_ok = ti < t.ntok[x];
        const int pos = t.prefix + t.i0[x] + ti;         // keys 0 .. pos
        const int64_t tok = (int64_t)p.q0[t.b] + t.i0[x] + ti;
        const int head = t.g * p.group + tj;
        if (seg > 0)
            wait(q_free(c), (uint32_t)((seg - 1) & 1));
        const __nv_bfloat16 *src = row_ok ? p.q + tok * p.q_stride + (int64_t)head * D : nullptr;
        const float rq = stage_rows(c, src, p.q, D, x, warp * 32);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(q_ready(c));

        float m_use = -INFINITY, lsum = 0.f;
        float m_l = 0.f;                                 // l's reference once they are apart; m_use until then
        bool apart = false;                              // for the warp's stages from here on
        const int s1 = min(t.s1, t.nst[x]);
#pragma unroll 1
        for (int j = t.s0; j < s1; ++j) {
            const int k = kbase + j - t.s0, vs = k % kVS;
            const int key0 = j * kKT;
            wait(conv_v(c, vs), ring_par(k, kVS));
            const volatile uint32_t *info = reinterpret_cast<const volatile uint32_t *>(c.smem + c.lay.info) + vs * 4;
            const uint32_t pmask = alive ? info[0] : 0u;
            const uint32_t needs = info[1];
            const float4 *fac = reinterpret_cast<const float4 *>(c.smem + c.lay.factor + vs * kKT * 4);
            const float4 *evs = reinterpret_cast<const float4 *>(c.smem + c.lay.evs + vs * kKT * 4);
            const float4 *pfac = reinterpret_cast<const float4 *>(c.smem + c.lay.pfactor + vs * kKT * 4);
            // keys this row may see: [key0, key0 + nvis), on pages that were copied
            // (padding rows see all: their scores only reach their own row of O, which is not stored)
            const int nvis = row_ok ? min(kKT, pos - key0 + 1) : kKT;
            const bool dense = pmask == all_pages && nvis == kKT;
            wait(s_full(c, x), (uint32_t)(done & 1));
            if (alive)
                tc_fence_after();
            uint32_t sv[3][32];
#pragma unroll
            for (int q = 0; q < 3; ++q)
                tmem_ld32_nowait(srow + (uint32_t)(q * 32), sv[q]);
            tmem_wait_ld();
            // Common case (see the top): P against the running maximum.
            float part = 0.f;
            bool fast = __all_sync(0xffffffffu, dense && alive && m_use != -INFINITY && !apart && needs != kApart);
            if (fast) {
                const float nmu = kPLog2 - m_use;
                const float2 rq2 = make_float2(rq, rq), nmu2 = make_float2(nmu, nmu);
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                // 32 columns; their P lies over 16 columns further to the left,
                // so that the scores of the first half stay in registers
                auto quarter = [&](int q, const uint32_t (&s)[32]) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 f = fac[q * 8 + i], w = pfac[q * 8 + i];
                        const float2 x0 = __ffma2_rn(__fmul2_rn(make_float2(__uint_as_float(s[4 * i]),
                                                                            __uint_as_float(s[4 * i + 1])),
                                                                make_float2(f.x, f.y)), rq2, nmu2);
                        const float2 x1 = __ffma2_rn(__fmul2_rn(make_float2(__uint_as_float(s[4 * i + 2]),
                                                                            __uint_as_float(s[4 * i + 3])),
                                                                make_float2(f.z, f.w)), rq2, nmu2);
                        float2 p0 = make_float2(ex2_approx(x0.x), ex2_approx(x0.y));
                        float2 p1 = make_float2(ex2_approx(x1.x), ex2_approx(x1.y));
                        acc[0] = __fadd2_rn(acc[0], p0);
                        acc[1] = __fadd2_rn(acc[1], p1);
                        p0 = __fmul2_rn(p0, make_float2(w.x, w.y));
                        p1 = __fmul2_rn(p1, make_float2(w.z, w.w));
                        pk[2 * i] = pack_half2(p0.x, p0.y);
                        pk[2 * i + 1] = pack_half2(p1.x, p1.y);
                    }
                    tmem_st16_nowait(srow + (uint32_t)(q * 16), pk);
                };
                quarter(2, sv[2]);
                quarter(0, sv[0]);
                quarter(1, sv[1]);
                tmem_ld32_nowait(srow + 96u, sv[2]);
                tmem_wait_ld();
                quarter(3, sv[2]);
                part = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                const float most = fmaxf(fmaxf(acc[0].x, acc[0].y), fmaxf(acc[1].x, acc[1].y));
                if (__any_sync(0xffffffffu, row_ok && !(most <= __uint_as_float(info[2])))) {
                    // the scores go back for the exact path
                    tmem_wait_st();
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        tmem_st32(srow + (uint32_t)(q * 32), sv[q]);
                    fast = false;
                }
            }
            if (!fast) {
                // the exact path, 32 columns at a time (short loops: it runs
                // at a piece's first stage, on the diagonal and where a
                // maximum moves, its instructions mostly cold): the stage's
                // masked maximum first, then P
                const int shift = 31 - __clz(P);
                // the scores of columns 32c .. 32c + 31, -inf where not visible
                // (past this row's end, or on a page that was not copied)
                auto columns = [&](int c32, float (&xs)[32]) {
                    uint32_t raw[32];
                    tmem_ld32_nowait(srow + (uint32_t)(c32 * 32), raw);
                    tmem_wait_ld();
                    const uint32_t first = (pmask >> ((c32 * 32) >> shift)) & 1u, second = (pmask >> ((c32 * 32 + 16) >> shift)) & 1u;
                    const int n = alive ? nvis - c32 * 32 : 0;
                    const int n0 = first ? n : 0, n1 = second ? n : 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 f = fac[c32 * 8 + i];
                        const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            xs[4 * i + v] = 4 * i + v < (i < 4 ? n0 : n1) ? __uint_as_float(raw[4 * i + v]) * (fs[v] * rq)
                                                                         : -INFINITY;
                    }
                };
                float cm = -INFINITY, cy = -INFINITY;    // maxima of x and of y
#pragma unroll 1
                for (int c32 = 0; c32 < kKT / 32; ++c32) {
                    float xs[32];
                    columns(c32, xs);
                    if (apart || needs != 0u)
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            cm = max3f(cm, xs[i], xs[i + 1]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 v = evs[c32 * 8 + i];
                        cy = max3f(max3f(cy, xs[4 * i] + v.x, xs[4 * i + 1] + v.y), xs[4 * i + 2] + v.z, xs[4 * i + 3] + v.w);
                    }
                }
                const float m_old = m_use;
                float scale_o = 1.f;
                if (m_use == -INFINITY) {
                    m_use = cy;
                } else if (cy > m_use + kRescaleLog2) {
                    scale_o = ex2_approx(m_use - cy);
                    m_use = cy;
                }
                if (!apart && __any_sync(0xffffffffu, needs == kApart || cm - m_use > kMaxLead)) {
                    apart = true;
                    m_l = m_old;
                }
                if (!apart) {
                    // (in halves: where m rises by V's exponents, up to 2^120, the weights so far can
                    // matter past fp32's least normal number; what they brought to O does not)
                    if (m_use != m_old && m_old != -INFINITY) {
                        const float half = ex2_approx(0.5f * (m_old - m_use));
                        lsum = lsum * half * half;
                    }
                } else if (m_l == -INFINITY) {
                    m_l = cm;
                } else if (cm > m_l + kRescaleLog2) {
                    lsum *= ex2_approx(m_l - cm);
                    m_l = cm;
                }
                if (j > t.s0 && __any_sync(0xffffffffu, scale_o != 1.f)) {
                    // tcgen05.ld/st are warp-wide: lanes that keep their references scale by 1
                    wait(pv_done(c, x), (uint32_t)((done - 1) & 1));
                    if (alive) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c16 = 0; c16 < D / 16; ++c16) {
                            uint32_t ov[16];
                            tmem_ld16_nowait(orow + (uint32_t)(c16 * 16), ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                ov[i] = __float_as_uint(__uint_as_float(ov[i]) * scale_o);
                            tmem_st16_nowait(orow + (uint32_t)(c16 * 16), ov);
                        }
                        tmem_wait_st();
                    }
                }
                const float mu = m_use == -INFINITY ? 0.f : m_use - kPLog2;
                const float mu_l = !apart ? mu : m_l == -INFINITY ? 0.f : m_l - kPLog2;
                float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int c32 = 0; c32 < kKT / 32; ++c32) {       // (P of columns 32c.. lies over columns 16c..)
                    float xs[32];
                    uint32_t pk[16];
                    columns(c32, xs);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 v = (apart ? evs : pfac)[c32 * 8 + i];
                        const float vs4[4] = {v.x, v.y, v.z, v.w};
                        float w[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float wl = ex2_approx(xs[4 * i + u] - mu_l);
                            sums[u] += wl;
                            w[u] = apart ? ex2_approx(xs[4 * i + u] + vs4[u] - mu) : wl * vs4[u];
                        }
                        pk[2 * i] = pack_half2(w[0], w[1]);
                        pk[2 * i + 1] = pack_half2(w[2], w[3]);
                    }
                    tmem_st16_nowait(srow + (uint32_t)(c32 * 16), pk);
                }
                part = (sums[0] + sums[1]) + (sums[2] + sums[3]);
            }
            lsum += part;
            tmem_wait_st();
            tc_fence_before();
            ++done;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(p_full(c, x));
        }

        // --- this row of O_x, normalised, and its log-sum-exp
        const bool whole = t.s0 == 0 && t.s1 == t.nst_all;
        const bool any = s1 > t.s0;                      // this tile attends a stage of the piece
        if (any)
            wait(pv_done(c, x), (uint32_t)((done - 1) & 1));
        if (alive && t.ntok[x] > 0) {
            tc_fence_after();
            // (a NaN sum stays NaN; a tile with no stage here or no visible key gives zeros)
            // (2^(m_use - m_l) in two halves: itself it can leave fp32's range, up to 2^129 or with 1 / l
            // under 2^-126, where its product with O does not)
            const bool none = !any || lsum == 0.f;
            const float half = none || !apart ? 1.f : ex2_approx(0.5f * (m_use - m_l));
            const float f = none ? 0.f : __frcp_rn(lsum) * half;
            const int64_t orr = tok * p.hq + head;
            const int slot = piece_slot(p, blockIdx.x, t.u);
            const int64_t prow = (int64_t)slot * kChunkRows + x * 128 + r;
#pragma unroll 1
            for (int c16 = 0; c16 < D / 16; ++c16) {
                uint32_t ov[16] = {};
                if (any)
                    tmem_ld16_nowait(orow + (uint32_t)(c16 * 16), ov);
                tmem_wait_ld();
                float o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[i] = __uint_as_float(ov[i]) * half * f;
                if (row_ok && whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + orr * D + c16 * 16);
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        dst[v] = make_uint4(pack_bf16x2(o[8 * v], o[8 * v + 1]), pack_bf16x2(o[8 * v + 2], o[8 * v + 3]),
                                            pack_bf16x2(o[8 * v + 4], o[8 * v + 5]), pack_bf16x2(o[8 * v + 6], o[8 * v + 7]));
                } else if (row_ok) {
                    // (four columns of all rows together: neighbouring lanes write neighbouring words)
                    float4 *dst = reinterpret_cast<float4 *>(p.ws_part) +
                                  (((int64_t)slot * 2 + x) * (D / 4) + c16 * 4) * 128 + r;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        dst[v * 128] = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                }
            }
            if (row_ok) {
                const float m = apart ? m_l : m_use;
                const float lse = lsum != 0.f ? ((m == -INFINITY ? 0.f : m - kPLog2) + log2f(lsum)) * 0.6931471805599453f
                                              : -INFINITY;
                if (!whole)
                    p.ws_lse[prow] = lse;
                else if (p.lse_out)
                    p.lse_out[orr] = lse;
            }
        }
        tc_fence_before();
        kbase += t.s1 - t.s0;
        ++seg;
    }
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    shkv_q8_chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ Q8ChunkParams p)
{
    extern __shared__ uint8_t smem_raw[];
    Ctx c;
    {
        const uint32_t raw = smem_u32(smem_raw);
        const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
        c.smem = smem_raw + pad;
        c.base = raw + pad;
    }
    c.lay = smem_layout();
    c.abort_flag = reinterpret_cast<volatile uint32_t *>(c.smem + c.lay.misc);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kKS; ++i) {
            mbar_init(full_k(c, i), 1);
            mbar_init(empty_k(c, i), 1);
        }
        for (int i = 0; i < kVS; ++i) {
            mbar_init(full_v(c, i), 1);
            mbar_init(conv_v(c, i), kConvWarps);
            mbar_init(empty_v(c, i), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full(c, x), 1);
            mbar_init(p_full(c, x), kGroupWarps);
            mbar_init(pv_done(c, x), 1);
        }
        mbar_init(q_ready(c), 2 * kGroupWarps);
        mbar_init(q_free(c), 1);
        mbar_init(fin_b(c), 2);
        *c.abort_flag = 0u;
        fence_barrier_init();
    }
    if (warp == 0)
        tmem_alloc(c.base + c.lay.tslot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(c.smem + c.lay.tslot);
    pdl_wait_prior();
    pdl_launch_dependents();

    if (warp < 2 * kGroupWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        chunk_softmax(p, c, tmem, warp / kGroupWarps);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kKWarp)
            chunk_producer<false>(&tmK, p, c);
        else if (warp == kVWarp)
            chunk_producer<true>(&tmV, p, c);
        else if (warp == kQkWarp) {
            if ((threadIdx.x & 31) == 0)
                chunk_qk(p, c, tmem);
        } else if (warp == kPvWarp) {
            if ((threadIdx.x & 31) == 0)
                chunk_pv(p, c, tmem);
        } else {
            chunk_convert(p, c);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tmem, kTmemCols);
}

// Joins the pieces of split units, 8 rows a block: thread = (row, four
// columns), the rows of a column group neighbours as the pieces hold them.
// Block y takes the unit that cut y (the start of CTA y + 1) falls inside, if
// it is the first cut in it.
__global__ void __launch_bounds__(256) shkv_q8_chunk_join_kernel(const __grid_constant__ Q8ChunkParams p)
{
    __shared__ float maxima[8][8];
    pdl_wait_prior();
    pdl_launch_dependents();
    const int cut = blockIdx.y + 1;
    const int u = p.cut_unit[cut];
    if (p.cut_stage[cut] == 0 || (p.cut_unit[cut - 1] == u && p.cut_stage[cut - 1] > 0))
        return;
    Piece t;
    t.u = u;
    set_unit(p, t);
    const int x = blockIdx.x >> 4, r = (blockIdx.x & 15) * 8 + (threadIdx.x & 7), row = x * 128 + r;
    if (((blockIdx.x & 15) * 8) / p.group >= t.ntok[x])  // the block's first row: none of its rows is in use
        return;
    const int c4 = threadIdx.x >> 3, D = p.head_dim;
    const int ti = r / p.group, tj = r - ti * p.group;
    const bool row_ok = ti < t.ntok[x];
    int last = cut;                              // last CTA that holds a piece
    while (last + 1 < p.num_ctas && p.cut_unit[last + 1] == u && p.cut_stage[last + 1] > 0)
        ++last;
    float M = -INFINITY;                         // NaN as soon as a piece's log-sum-exp is
    if (row_ok) {
        for (int i = cut - 1 + c4; i <= last; i += 32)
            M = max_nan(M, p.ws_lse[(int64_t)piece_slot(p, i, u) * kChunkRows + row]);
    }
    M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, 8));
    M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, 16));
    if ((threadIdx.x & 31) < 8)
        maxima[threadIdx.x >> 5][threadIdx.x & 7] = M;
    __syncthreads();
    M = maxima[0][threadIdx.x & 7];
#pragma unroll
    for (int w = 1; w < 8; ++w)
        M = max_nan(M, maxima[w][threadIdx.x & 7]);
    if (!row_ok || c4 >= D / 4)
        return;
    float wsum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M != M) {
        wsum = acc.x = acc.y = acc.z = acc.w = M;
    } else if (M != -INFINITY) {
#pragma unroll 2
        for (int i = cut - 1; i <= last; ++i) {
            const int64_t slot = piece_slot(p, i, u);
            // (weights of 2^-10 at most: sums of outputs near fp32's largest stay below it)
            const float w = ex2_approx((p.ws_lse[slot * kChunkRows + row] - M) * 1.4426950408889634f) * 0x1p-10f;
            const float4 v = reinterpret_cast<const float4 *>(p.ws_part)[((slot * 2 + x) * (D / 4) + c4) * 128 + r];
            wsum += w;
            acc.x += w * v.x;
            acc.y += w * v.y;
            acc.z += w * v.z;
            acc.w += w * v.w;
        }
    }
    const float winv = wsum != 0.f ? 1.f / wsum : 0.f;
    const int64_t orr = ((int64_t)p.q0[t.b] + t.i0[x] + ti) * p.hq + (int64_t)t.g * p.group + tj;
    *reinterpret_cast<uint2 *>(p.out + orr * D + c4 * 4) =
        make_uint2(pack_bf16x2(acc.x * winv, acc.y * winv), pack_bf16x2(acc.z * winv, acc.w * winv));
    if (c4 == 0 && p.lse_out)
        p.lse_out[orr] = wsum != 0.f ? M + logf(wsum * 0x1p10f) : -INFINITY;
}

// tmK, tmV: 2-D maps of the code pools (box of 128 bytes x P rows, 128-byte swizzle).
cudaError_t launch_q8_chunk(const CUtensorMap &tmK, const CUtensorMap &tmV, const Q8ChunkParams &p, bool splits,
                            cudaStream_t stream)
{
    static std::atomic<int> known;
    int regs;                  // the register split hands out exactly the launch's 128 a thread
    cudaError_t e = kernel_registers(shkv_q8_chunk_kernel, known, &regs);
    if (e != cudaSuccess)
        return e;
    if ((uint32_t)regs * kThreads != kSoftmaxRegs * 256 + kOtherRegs * 256)
        return cudaErrorInvalidConfiguration;
    const uint32_t smem = smem_layout().total;
    e = cudaFuncSetAttribute(shkv_q8_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = launch_pdl(shkv_q8_chunk_kernel, p.num_ctas, kThreads, smem, stream, tmK, tmV, p);
    if (e != cudaSuccess || !splits)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kChunkRows / 8, (unsigned)(p.num_ctas - 1));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, shkv_q8_chunk_join_kernel, p);
}

}  // namespace shkv
