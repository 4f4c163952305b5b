// q8_decode.cu -- attention of up to 64 stacked query rows per (request, KV
// head) over the 8-bit KV cache: a decode step of N decoders, and chunks of a
// few new tokens (causal), on the 5th-generation tensor cores.
//
// Work is split as in the bf16 decode: the (request, KV head, page) chunks are
// cut into contiguous ranges of equal cost, one persistent CTA each; a (b, g)
// unit that straddles a cut leaves partials that its last piece to arrive
// merges by log-sum-exp.  Every page is read once for all rows of its head.
// A stage is 128 tokens of one unit (TMEM lanes = tokens, then head-dim
// columns):
//
//   S^T[t, r]  = sum_d k8[t, d] (qh[r, d] + ql[r, d])             kind::f8f6f4
//   y[t, r]    = S^T[t, r] * 2^ek[t] * 2^eq[r] * scale * log2(e) + ev[t]
//   P^T[t, r]  = 2^(y - m[r] + 7),  m[r] a running maximum of y    fp16
//   O^T[d, r] += sum_t 2^-8 v8[t, d] P^T[t, r]                    kind::f16
//   l[r]      += sum_t P^T[t, r] * 2^-ev[t]                       (P before its rounding)
//   out = 256 O^T / l,   lse = ln2 * (m - 7 + log2(l))
//
// K's codes go to the tensor cores as they lie in the page.  A bf16 query has
// 8 significant bits: its row is scaled by a power of two to at most 448 and
// split into two e4m3 terms, qh nearest and ql = q - qh.  That is exact for
// values of 2^-2 and more after scaling (2^-9.8 of the row's largest at most);
// smaller ones are held to 2^-10, half of e4m3's least step: 2^-17.8 of the
// largest.  (A third term would cost half as many QK products again.)  V's codes
// are moved to fp16 in shared memory (sign and seven bits, exponent bias and all:
// v8 * 2^-8, exactly).  With the token's V exponent inside y, P is relative to the row's
// largest weight times value scale, so that fp16 holds 11 bits of every token
// that matters to the sum, whatever the magnitudes of weights and values apart:
// fp16's least step, 2^-24, is 2^-31 of that largest, and 2^20 tokens below it
// are lost to 2^-12 of it.  V exponents of -40 to 40 (row maxima of 2^-31 to
// 2^48) keep P before its rounding at 2^-81 and more for the largest weight, and
// l's terms under 2^55.  A `low` token, under -40, as a zero row is, takes part in
// l as one of -40 and not in O, while its weight is small enough (see `lead`).
// Where it is not, and in every stage from the first exponent above 40 on, the
// stage is `wide` (each softmax group for itself): its part of l comes from a
// second exponential, relative to a running maximum of y - ev of its own, and a
// token whose V is zero stays out of m.  Such a stage is slow (loops over eight
// rows, four meetings of the group's warps): with all of a segment's wide, 31
// requests of 1k to 8k tokens take 91 us instead of 56 at 8 rows, 266 instead of
// 71 at 32.  Sums and O are fp32.
//
// The softmax is bound by the latency of its chain, not by its instructions:
// up to 48 rows its two groups of four warps take alternate stages, each with
// all rows, a running maximum, sums and O of its own, joined at the segment's
// end.  Above (registers), both groups work on every stage, on half the rows.
//
// Roles (512 threads):
//   warps 0-7    softmax: warp w owns tokens 32*(w%4) .. +31 of its stages;
//                also stages the query rows and reads O^T out
//   warp 8       QK issuer (one lane)
//   warp 9       producer of K pages, scales, query rows and validity words
//   warp 10      PV issuer (one lane)
//   warp 11      producer of V pages
//   warps 12-15  V's conversion, one token a thread: the codes land in the
//                upper 16 KB of a 32 KB slot, where the thread reads its row
//                and writes it back as fp16 over both halves (row t's codes
//                lie inside row t's fp16 bytes, so no thread waits for
//                another).  Above 48 rows also the tokens' factors; below,
//                the softmax's warps find them while they wait for S^T: a
//                stage takes the conversion 1570 cycles with them, 1100
//                without
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "decode_common.cuh"
#include "launch.cuh"
#include "q8_decode.cuh"
#include "q8_wait.cuh"
#include "umma_rows.cuh"

namespace shkv {

namespace {

using namespace detail;

constexpr int kTT = 128;                    // tokens per stage (the MMA's M)
constexpr int kTokenGroups = 4;             // 32-lane TMEM sub-partitions
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kQkWarp = 8;
constexpr int kKWarp = 9;
constexpr int kPvWarp = 10;
constexpr int kVWarp = 11;
constexpr int kConvWarp0 = 12;
constexpr int kConvWarps = 4;
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColS = 0;               // S^T buffers at columns 0 and 64
constexpr uint32_t kColO = 128;             // O^T
constexpr float kRescaleLog2 = 8.f;         // m lags the maximum by at most this
constexpr float kPLog2 = 7.f;               // P is 2^7 at the running maximum: 2^15 at most
constexpr int kVWindow = 40;                // a V exponent above makes a segment wide, one below -kVWindow is low
// A low token leads where its y - m + 7, with -kVWindow for its exponent, is above
// this.  A row of the least scale (zeros, or values under 2^-118) may add
// 2^(8 + kVWindow) to l: what its values would add to O is 2^-86 of the largest
// term at most.  What others would add is under fp16's least step.
constexpr float kLeadLeast = 8.f, kLeadLow = -24.f;
constexpr uint32_t kKSlotBytes = kTT * 128;
constexpr uint32_t kVSlotBytes = 2 * kTT * 128;
constexpr uint32_t kPBytes = kTT * 128;
constexpr int kScaleRing = 8;               // stages of scale bytes, see the note at the producer
// registers: 168 for the softmax warpgroups, 88 for the other two, of the
// launch's 128 a thread
constexpr uint32_t kSoftmaxRegs = 168, kOtherRegs = 88;
static_assert(kSoftmaxRegs * 256 + kOtherRegs * 256 == 128 * kThreads, "register split");

// scratch rows of 64 words: per softmax group the stage maxima and the sums
// [token group], the new 7 - m, the rescaling of O and l, m, and the wide
// stages' part of l and its reference; then the factors of the two groups at the
// segment's end (two halves each), the queries' scales, the rows' output offsets
// and whether the groups had wide stages
constexpr int kScrMax = 0, kScrNew = 4, kScrAlpha = 5, kScrM = 6, kScrL = 7, kScrMl = 8, kScrGroup = 9;
constexpr int kScrEnd = 2 * kScrGroup, kScrQ = kScrEnd + 4, kScrOff = kScrQ + 1, kScrWide = kScrOff + 1,
              kScrRows = kScrWide + 1;

__host__ __device__ constexpr int q_nr(int rows) { return (rows + 15) / 16 * 16; }
// N of the PV MMA: 48 is rounded up to a whole 64-column swizzle span.
__host__ __device__ constexpr int q_npv(int nr) { return nr == 48 ? 64 : nr; }
// The softmax groups take alternate stages.
__host__ __device__ constexpr bool q_pingpong(int nr) { return nr <= 48; }

constexpr int kKS = 4, kVS = 3;             // ring slots
constexpr int kInfo = kVS + 1;              // stages of token factors (see convert_v)
static_assert(kKS <= kScaleRing, "scales of a stage live until its factors are taken");

struct Smem {
    uint32_t vring, pbuf, qtile, qhalf, qbuf, scr, scales, info, bars, meta, misc, tslot, total;
};

// From offset 0: the K ring, the V ring (slots [half][128 tokens][128 B]), P^T
// [128 tokens][128 B] of each group that has its own, and the query tiles
// [qh | ql][NR rows][128 B], all 128-byte swizzled; qbuf holds the next
// segment's bf16 query rows; info a stage's token factors (above 48 rows).
__host__ __device__ constexpr Smem smem_layout(int nr)
{
    Smem u{};
    u.vring = kKS * kKSlotBytes;
    u.pbuf = u.vring + kVS * kVSlotBytes;
    u.qtile = u.pbuf + (q_pingpong(nr) ? 2u : 1u) * kPBytes;
    u.qhalf = (uint32_t)nr * 128u;
    u.qbuf = u.qtile + 2 * u.qhalf;
    u.scr = u.qbuf + (uint32_t)nr * 256u;
    u.scales = u.scr + kScrRows * 64 * 4;
    u.info = u.scales + kScaleRing * 2 * kTT;
    u.bars = u.info + (q_pingpong(nr) ? 0u : kInfo * kTT * 8u);
    u.meta = u.bars + 48 * 8u;
    u.misc = u.meta + kScaleRing * 4u;       // validity words
    u.tslot = u.misc + 8;
    u.total = u.misc + 16 + 1024;           // + slack to align the base to 1024 bytes
    return u;
}
static_assert(smem_layout(64).total <= (uint32_t)kSmemLimit && smem_layout(48).total <= (uint32_t)kSmemLimit, "fits");

struct Ctx4 {
    uint8_t *smem;
    uint32_t base, bars;
    volatile uint32_t *abort_flag;
    uint32_t *bcast;
    int64_t cta_begin, cta_end;
};

// Barriers.
constexpr int kFullK = 0, kEmptyK = kFullK + kKS, kFullV = kEmptyK + kKS, kConvV = kFullV + kVS, kEmptyV = kConvV + kVS,
              kScaleB = kEmptyV + kVS, kInfoB = kScaleB + kScaleRing, kPFull = kInfoB + kInfo, kPvDone = kPFull + 2,
              kQFull = kPvDone + 2, kQEmpty = kQFull + 1, kSFull = kQEmpty + 1, kSFree = kSFull + 2, kQReady = kSFree + 2,
              kQTileFree = kQReady + 1, kFin = kQTileFree + 1, kBars = kFin + 1;
static_assert(kBars <= 48, "room for the barriers");
__device__ __forceinline__ uint32_t bar_at(const Ctx4 &c, int i) { return c.bars + 8u * (uint32_t)i; }

// A ring position that advances with the stages: its slot and the parity of
// the slot's current use.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t par = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == N) {
            slot = 0;
            par ^= 1u;
        }
    }
};

// Stages of a segment.
__device__ __forceinline__ int stages_of(const Segment &s, int P) { return ((s.p1 - s.p0) * P + kTT - 1) / kTT; }

// Offset of token t's K scale byte in a stage's ([page][K, V][P] as in the
// pool); V's is P further on.
__device__ __forceinline__ uint32_t scale_off(int t, int log2P)
{
    return (uint32_t)(((t >> log2P) << (log2P + 1)) + (t & ((1 << log2P) - 1)));
}

// Whether the stage's tokens below `n` on copied pages hold a V exponent above
// the window (NaN rows, 255, aside), by a warp.  w: the V scales of the lane's
// four tokens.
__device__ __forceinline__ bool stage_above(uint32_t w, int n, uint32_t mask, int log2P)
{
    const int t = 4 * (threadIdx.x & 31);
    const int in = ((mask >> (t >> log2P)) & 1u) ? n - t : 0;
    bool out = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int b = (int)((w >> (8 * i)) & 0xffu);
        out = out || (i < in && b != 255 && b > 127 + kVWindow);
    }
    return __any_sync(0xffffffffu, out);
}

// Keys below this are seen by every row of the unit.
__device__ __forceinline__ int keys_all_see(const Q8DecodeParams &q, const Segment &s)
{
    const int L = plan_len(q.d, s);
    return q.causal ? L - q.n_q[s.b] + 1 : L;
}

// D[tmem] (+)= A[smem] . B[smem]^T on e4m3 / on fp16 operands, fp32 accumulate.
__device__ __forceinline__ void umma_f8(uint32_t d_taddr, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_taddr),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}
constexpr uint32_t idesc_of(int M, int N, bool a_mn, bool b_mn)   // formats 0: e4m3 (f8f6f4), fp16 (f16)
{
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Two e4m3 codes of w (the low or the high half) as fp16 pairs, times 2^-8:
// each code's byte with its sign above it, moved so that the sign and the
// exponent and mantissa bits come to lie in fp16's places.  Three full-rate
// integer instructions; the conversion instruction measured slower here.
template <bool kHigh>
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t w)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(kHigh ? 0xB3A2 : 0x9180));
    return (r << 7) & 0xBF80BF80u;
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------
// Stage j of a segment is the 128 tokens from p0*P + j*128.  One lane copies
// one page (a box of P rows x 128 bytes; at head_dim 64 the box's upper half
// is outside the tensor and filled with zeros).  The K warp also copies the
// pages' scale bytes, with one 16-byte asynchronous copy a lane (a bulk copy a
// page took as long to issue as the codes, 600 cycles a stage of 16-token
// pages, and this warp then bounded long contexts), and publishes the stage's
// validity word, on barriers of a ring of their own, so that they wait for no
// V slot.  The K warp writes entry k once QK(k - KS) is complete, and entry
// k - 8 must be through by then.  Above 48 rows QK(i) waits for the factors that
// the V conversion's warps take from the scales of stage i.  Up to 48 it waits for
// the softmax to have read the scores of stage i - 2, whose group took the scales
// of its stage i - 4 before: entries up to k - 8.
__device__ __forceinline__ void cp_async16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// One arrival on the barrier once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int NR, bool kIsK>
__device__ void producer_q8(const CUtensorMap *tm, const Q8DecodeParams &q, const Ctx4 &c)
{
    constexpr Smem L = smem_layout(NR);
    constexpr int kSlots = kIsK ? kKS : kVS;
    const DecodeParams &p = q.d;
    const int lane = threadIdx.x & 31;
    const int P = p.page_size, RB = kTT / P, log2P = 31 - __clz(P);
    const uint64_t pol = l2_evict_first_policy();
    if (lane == 0)
        prefetch_tensormap(tm);
    bool alive = true;
    int k = 0, seg = 0, q_issued = -1;
    Ring<kSlots> ring;
    Segment s = locate(p, c.cta_begin, c.cta_end);
    int pre = unit_entry(p.block_table, p, s.b, s.p0 + lane, s.p1);
#pragma unroll 1
    for (;;) {
        const bool has_next = s.seg_end < c.cta_end;
        Segment sn;
        int pre_next = -1;
        if (has_next) {
            sn = next_segment(p, s, c.cta_end);
            pre_next = unit_entry(p.block_table, p, sn.b, lane, sn.p1);
        }
        const int dev_len = kIsK && lane == 0 ? __ldg(p.seq_lens + s.b) : 0;
        if (kIsK) {
            if (alive) {
                const bool ok = q8_wait<true>(bar_at(c, kQEmpty), (uint32_t)((seg & 1) ^ 1), c.abort_flag, p.err);
                alive = __all_sync(0xffffffffu, ok);
            }
            if (alive) {
                const int n = q.n_q[s.b];
                const uint32_t bytes = (uint32_t)(p.group * q.head_dim * 2);
                if (lane == 0)
                    mbar_arrive_expect_tx(bar_at(c, kQFull), bytes * (uint32_t)n);
                __syncwarp();
                const __nv_bfloat16 *src = p.q + (int64_t)q.q0[s.b] * q.q_stride + (int64_t)s.g * p.group * q.head_dim;
#pragma unroll 1
                for (int i = lane; i < n; i += 32)
                    bulk_load(c.base + L.qbuf + (uint32_t)i * bytes, src + (int64_t)i * q.q_stride, bytes,
                              bar_at(c, kQFull));
                q_issued = seg;
            }
        }
        int left = s.p1 - s.p0;                          // pages still to copy
        int w = 0;                                       // position in the window of 32 table entries
        int cur = pre;
        int next_j = s.p0 + 32 + lane;
        int nxt = unit_entry(p.block_table, p, s.b, next_j, s.p1);
#pragma unroll 1
        for (; left > 0; left -= RB) {
            if (w == 32) {                               // a stage's pages never straddle a window
                w = 0;
                cur = nxt;
                next_j += 32;
                nxt = unit_entry(p.block_table, p, s.b, next_j, s.p1);
            }
            const int id = __shfl_sync(0xffffffffu, cur, (w + lane) & 31);
            w += RB;
            bool ok = true;
            if (alive)
                ok = q8_wait<true>(bar_at(c, (kIsK ? kEmptyK : kEmptyV) + ring.slot), ring.par ^ 1u, c.abort_flag, p.err);
            alive = alive && __all_sync(0xffffffffu, ok);
            const bool inside = lane < RB && lane < left;
            const bool valid = inside && (uint32_t)id < (uint32_t)p.num_pages;
            const uint32_t mask = __ballot_sync(0xffffffffu, valid);
            if (kIsK && alive && inside && !valid)
                atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
            const uint32_t bar = bar_at(c, (kIsK ? kFullK : kFullV) + ring.slot);
            const uint32_t sbar = bar_at(c, kScaleB + k % kScaleRing);
            if (alive && lane == 0) {
                const uint32_t rows = (uint32_t)(__popc(mask) * P);
                if (kIsK) {
                    reinterpret_cast<volatile uint32_t *>(c.smem + L.meta)[k % kScaleRing] =
                        mask | ((uint32_t)k << 8);       // valid pages + stage tag
                    mbar_arrive(sbar);
                }
                mbar_arrive_expect_tx(bar, 128u * rows);
            }
            __syncwarp();
            if (alive && valid) {
                const int unit = id * p.hkv + s.g;
                const uint32_t dst = c.base + (kIsK ? (uint32_t)ring.slot * kKSlotBytes
                                                    : L.vring + (uint32_t)ring.slot * kVSlotBytes + kTT * 128u);
                tma_load_2d(dst + (uint32_t)(lane * P) * 128u, tm, 0, unit * P, bar, pol);
            }
            if (kIsK) {
                // 16 bytes a lane, P / 8 lanes a page
                const int page = (lane << 3) >> log2P, in = lane & (P / 8 - 1);
                const int pid = __shfl_sync(0xffffffffu, id, page & 31);
                if (alive) {
                    if (page < RB && ((mask >> page) & 1u))
                        cp_async16(c.base + L.scales + (uint32_t)((k % kScaleRing) * 2 * kTT + lane * 16),
                                   q.scales + ((int64_t)pid * p.hkv + s.g) * 2 * P + in * 16);
                    cp_async_arrive(sbar);
                }
            }
            __syncwarp();
            if (alive) {
                ++k;
                ring.next();
            }
        }
        if (kIsK && lane == 0 && dev_len != plan_len(p, s))
            atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
        ++seg;
        if (!has_next)
            break;
        s = sn;
        pre = pre_next;
    }
    // After an abort, wait (bounded) for the copies still in flight (stages up
    // to k - 1) so no copy lands after the CTA exits.
    if (!alive && lane == 0) {
        for (int i = max(0, k - kSlots); i < k; ++i)
            mbar_drain_bounded(bar_at(c, (kIsK ? kFullK : kFullV) + i % kSlots), (uint32_t)((i / kSlots) & 1));
        if (kIsK && q_issued >= 0)
            mbar_drain_bounded(bar_at(c, kQFull), (uint32_t)(q_issued & 1));
    }
    if (kIsK)
        asm volatile("cp.async.wait_all;" ::: "memory");
}

// Before the previous grid is waited for: L2 prefetch of the CTA's first
// stages.  The table entries may be stale; they are used for nothing else.
__device__ void warm_l2_q8(const CUtensorMap *tm, const DecodeParams &p, const Ctx4 &c, int slots)
{
    const int lane = threadIdx.x & 31;
    const Segment s = locate(p, c.cta_begin, c.cta_end);
    const int pages = min(s.p1 - s.p0, min(32, slots * kTT / p.page_size));
    if (lane < pages) {
        const int id = __ldcg(p.block_table + (int64_t)s.b * p.max_pages + s.p0 + lane);
        if (id >= 0 && id < p.num_pages)
            tma_prefetch_2d(tm, 0, (id * p.hkv + s.g) * p.page_size);
    }
}

// What a token brings to the softmax: (score factor, first row that sees it
// | kMasked if some token of the warp is not seen by all | kWide if the stage
// holds a V exponent above the window | V's scale byte << 16).  kb, vb: the
// token's scale bytes; at: its distance from the first key some row does not
// see.  A NaN row of V makes its key's scores NaN, so that only rows that attend
// it see it.
constexpr int kMasked = 0x100, kWide = 0x200;
__device__ __forceinline__ float2 token_factors(const DecodeParams &p, int kb, int vb, bool valid, int at, bool above)
{
    const int ve = !valid || vb == 255 ? 127 : vb;
    // rows from row_min on see the token (new token i from position L - n + i on)
    const int row_min = valid ? min(64, max(0, (at + 1) * p.group)) : 64;
    const int flags = (__any_sync(0xffffffffu, row_min > 0) ? kMasked : 0) | (above ? kWide : 0);
    return make_float2(!valid ? 0.f : vb == 255 ? __uint_as_float(0x7fc00000u) : q8_scale((uint32_t)kb) * p.scale_log2,
                       __int_as_float(row_min | flags | ve << 16));
}

// ---------------------------------------------------------------------------
// V conversion
// ---------------------------------------------------------------------------
// Every code becomes fp16, whatever its token: the bits give finite values, and
// where a token is not seen P is 0.
template <int NR>
__device__ void convert_v(const Q8DecodeParams &q, const Ctx4 &c)
{
    constexpr Smem L = smem_layout(NR);
    constexpr bool kPing = q_pingpong(NR);
    const DecodeParams &p = q.d;
    const int t = threadIdx.x - kConvWarp0 * 32, lane = t & 31;
    const int P = p.page_size, log2P = 31 - __clz(P);
    volatile uint32_t *meta = reinterpret_cast<volatile uint32_t *>(c.smem + L.meta);
    const uint8_t *sc_mine = c.smem + L.scales + scale_off(t, log2P);
    const uint8_t *sc_four = c.smem + L.scales + scale_off(4 * lane, log2P) + P;
    const int page = t >> log2P;
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        bool ok = false;
        if (alive)
            ok = q8_wait<false>(bar, parity, c.abort_flag, p.err);
        alive = __all_sync(0xffffffffu, ok);
    };
    uint32_t k = 0;
    Ring<kScaleRing> sring;
    Ring<kVS> vring;
    Segment s = locate(p, c.cta_begin, c.cta_end);
#pragma unroll 1
    for (;;) {
        const int tok_end = s.p1 * P;
        const int lim = min(plan_len(p, s), tok_end);
        const int all_see = keys_all_see(q, s);
#pragma unroll 1
        for (int tok0 = s.p0 * P; tok0 < tok_end; tok0 += kTT, ++k) {
            if (!kPing) {
                // --- the token's factors (up to 48 rows the softmax's warps
                // have the time to find them).  (Entry k % kInfo was last used by
                // stage k - kVS - 1, whose PV was done before V(k - 1) was loaded.)
                const uint32_t entry = k % kInfo;
                wait(bar_at(c, kScaleB + sring.slot), sring.par);
                const uint32_t tagged = alive ? meta[sring.slot] : 0u;
                if (alive && (tagged >> 8) != (k & 0xffffffu)) {
                    if (lane == 0) {
                        atomicOr(p.err, SHKV_ERRF_PIPELINE);
                        *c.abort_flag = 1u;
                    }
                    alive = false;
                }
                const uint32_t mask = tagged & 0xffu;
                const int so = sring.slot * 2 * kTT;
                const uint32_t four = *reinterpret_cast<const volatile uint32_t *>(sc_four + so);
                const int kb = *(const volatile uint8_t *)(sc_mine + so), vb = *(const volatile uint8_t *)(sc_mine + so + P);
                const bool valid = alive && tok0 + t < lim && ((mask >> page) & 1u);
                const float2 f = token_factors(p, kb, vb, valid, tok0 + t - all_see,
                                               stage_above(four, lim - tok0, mask, log2P));
                if (alive)
                    reinterpret_cast<float2 *>(c.smem + L.info)[entry * kTT + t] = f;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar_at(c, kInfoB + (int)entry));
                sring.next();
            }
            // --- V
            wait(bar_at(c, kFullV + vring.slot), vring.par);
            if (alive) {
                uint8_t *row = c.smem + L.vring + (uint32_t)vring.slot * kVSlotBytes + (uint32_t)t * 128u;
                uint4 raw[8];
#pragma unroll
                for (int ch = 0; ch < 8; ++ch)
                    raw[ch] = *reinterpret_cast<const uint4 *>(row + kTT * 128 + ((ch ^ (t & 7)) << 4));
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) {
                    uint8_t *dst = row + (ch >> 2) * (kTT * 128);
                    const int c0 = (2 * ch) & 7;
                    *reinterpret_cast<uint4 *>(dst + ((c0 ^ (t & 7)) << 4)) =
                        make_uint4(widen_e4m3x2<false>(raw[ch].x), widen_e4m3x2<true>(raw[ch].x),
                                   widen_e4m3x2<false>(raw[ch].y), widen_e4m3x2<true>(raw[ch].y));
                    *reinterpret_cast<uint4 *>(dst + (((c0 + 1) ^ (t & 7)) << 4)) =
                        make_uint4(widen_e4m3x2<false>(raw[ch].z), widen_e4m3x2<true>(raw[ch].z),
                                   widen_e4m3x2<false>(raw[ch].w), widen_e4m3x2<true>(raw[ch].w));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_at(c, kConvV + vring.slot));
            vring.next();
        }
        if (s.seg_end >= c.cta_end)
            break;
        s = next_segment(p, s, c.cta_end);
    }
}

// ---------------------------------------------------------------------------
// MMA issuers (one lane each)
// ---------------------------------------------------------------------------
template <int NR>
__device__ void qk_issuer(const Q8DecodeParams &q, const Ctx4 &c, uint32_t tmem)
{
    constexpr Smem L = smem_layout(NR);
    constexpr bool kPing = q_pingpong(NR);
    constexpr uint32_t idesc = idesc_of(128, NR, false, false);
    const DecodeParams &p = q.d;
    const int steps = q.head_dim / 32;                   // 32 codes an MMA
    const uint64_t kd0 = umma_sdesc_sw128(c.base, 16u, 1024u);
    const uint64_t qh0 = umma_sdesc_sw128(c.base + L.qtile, 16u, 1024u);
    const uint64_t ql0 = umma_sdesc_sw128(c.base + L.qtile + L.qhalf, 16u, 1024u);
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive)
            alive = q8_wait<true>(bar, parity, c.abort_flag, p.err);
    };
    int seg = 0;
    uint32_t k = 0;
    Ring<kKS> ring;
    Segment s = locate(p, c.cta_begin, c.cta_end);
#pragma unroll 1
    for (;;) {
        wait(bar_at(c, kQReady), (uint32_t)(seg & 1));
#pragma unroll 1
        for (int left = stages_of(s, p.page_size); left > 0; --left, ++k) {
            const uint32_t buf = k & 1u;
            const uint64_t kd = kd0 + (uint64_t)(((uint32_t)ring.slot * kKSlotBytes) >> 4);
            wait(bar_at(c, kFullK + ring.slot), ring.par);
            if (!kPing)
                wait(bar_at(c, kInfoB + (int)(k % kInfo)), (k / kInfo) & 1u);
            wait(bar_at(c, kSFree + (int)buf), ((k >> 1) & 1u) ^ 1u);
            if (!kPing)
                mbar_arrive(bar_at(c, kSFull + (int)buf));   // passes the factors on to the softmax
            if (alive) {
                tc_fence_after();
                const uint32_t d = tmem + kColS + buf * 64u;
                // (rolled: unrolled, with the accumulate flag a constant, the first
                // product of a stage was added to what TMEM held before)
#pragma unroll 1
                for (int i = 0; i < steps; ++i) {
                    umma_f8(d, kd + (uint64_t)(2 * i), qh0 + (uint64_t)(2 * i), idesc, i ? 1u : 0u);
                    umma_f8(d, kd + (uint64_t)(2 * i), ql0 + (uint64_t)(2 * i), idesc, 1u);
                }
            }
            umma_commit(bar_at(c, kSFull + (int)buf));
            umma_commit(bar_at(c, kEmptyK + ring.slot));
            ring.next();
        }
        umma_commit(bar_at(c, kQTileFree));
        ++seg;
        if (s.seg_end >= c.cta_end)
            break;
        s = next_segment(p, s, c.cta_end);
    }
    umma_commit(bar_at(c, kFin));
    mbar_drain_bounded(bar_at(c, kFin), 0u);
}

template <int NR>
__device__ void pv_issuer(const Q8DecodeParams &q, const Ctx4 &c, uint32_t tmem)
{
    constexpr Smem L = smem_layout(NR);
    constexpr uint32_t idesc = idesc_of(128, q_npv(NR), true, true);
    constexpr bool kPing = q_pingpong(NR);
    const DecodeParams &p = q.d;
    const uint64_t vd0 = umma_sdesc_sw128(c.base + L.vring, (uint32_t)(kTT * 128), 1024u);
    const uint64_t pd0 = umma_sdesc_sw128(c.base + L.pbuf, (uint32_t)(kTT * 128), 1024u);
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive)
            alive = q8_wait<true>(bar, parity, c.abort_flag, p.err);
    };
    uint32_t k = 0;
    Ring<kVS> ring;
    Segment s = locate(p, c.cta_begin, c.cta_end);
#pragma unroll 1
    for (;;) {
        const int nst = stages_of(s, p.page_size);
#pragma unroll 1
        for (int j = 0; j < nst; ++j, ++k) {
            const uint64_t vd = vd0 + (uint64_t)(((uint32_t)ring.slot * kVSlotBytes) >> 4);
            const uint32_t g = kPing ? k & 1u : 0u;      // softmax group, its P and O
            const uint64_t pd = pd0 + (uint64_t)(g * (kPBytes >> 4));
            wait(bar_at(c, kConvV + ring.slot), ring.par);
            wait(bar_at(c, kPFull + (int)g), (kPing ? k >> 1 : k) & 1u);
            if (alive) {
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kTT / 16; ++ks)
                    umma_bf16(tmem + kColO + g * 64u, vd + (uint64_t)(ks * 128), pd + (uint64_t)(ks * 128), idesc,
                              (j < (kPing ? 2 : 1) && ks == 0) ? 0u : 1u);
            }
            umma_commit(bar_at(c, kPvDone + (int)g));
            umma_commit(bar_at(c, kEmptyV + ring.slot));
            ring.next();
        }
        if (s.seg_end >= c.cta_end)
            break;
        s = next_segment(p, s, c.cta_end);
    }
    umma_commit(bar_at(c, kFin));
    mbar_drain_bounded(bar_at(c, kFin), 0u);
}

// ---------------------------------------------------------------------------
// softmax warps
// ---------------------------------------------------------------------------
template <int NR>
__device__ void softmax_q8(const Q8DecodeParams &q, const Ctx4 &c, uint32_t tmem)
{
    constexpr bool kPing = q_pingpong(NR);
    constexpr int NH = kPing ? NR : NR / 2;    // rows per thread of a stage
    constexpr int NE = NR / 2;                 // rows per thread at the segment's end
    // 7 - m of the rows: in registers up to 32 a thread, above read where it is used
    constexpr bool kNmRegs = NH <= 32;
    constexpr int kLoad = NH <= 32 ? NH / 8 : 3;   // 8-column chunks of S^T in flight
    constexpr int kMerge = NR == 16 ? 1 : 4;   // rows a warp merges at a time
    constexpr Smem L = smem_layout(NR);
    const DecodeParams &p = q.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tg = warp & (kTokenGroups - 1), hh = warp / kTokenGroups;
    const int grp = kPing ? hh : 0;            // whose maxima, sums, P and O
    const int t = tg * 32 + lane;
    const int P = p.page_size, log2P = 31 - __clz(P);
    const int D = q.head_dim;
    const volatile uint32_t *meta = reinterpret_cast<const volatile uint32_t *>(c.smem + L.meta);
    const uint8_t *sc_four = c.smem + L.scales + scale_off(4 * lane, log2P) + P;
    const uint32_t lane_base = (uint32_t)(tg * 32) << 16;
    const uint32_t bar_id = 1u + (uint32_t)grp, bar_threads = kPing ? 128u : 256u;
    constexpr uint32_t kAllBar = 3;            // both groups
    float *scr = reinterpret_cast<float *>(c.smem + L.scr);
    const int *scr_i = reinterpret_cast<const int *>(scr);
    float *mine = scr + grp * kScrGroup * 64;
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        bool ok = false;
        if (alive)
            ok = q8_wait<false>(bar, parity, c.abort_flag, p.err);
        alive = __all_sync(0xffffffffu, ok) && alive;
        return alive;
    };
    // element i of a thread's rows of a stage is stacked row row_of(i): all of
    // them, or its half's 8-row chunks; every TMEM access is 8 columns
    auto row_of = [&](int i) { return kPing ? i : half_row(hh, i); };
    auto chunk_col = [&](int ch) { return kPing ? 8 * ch : 16 * ch + 8 * hh; };

    // Query rows of segment `sg`: bf16 staging buffer -> the two swizzled
    // e4m3 tiles and the rows' scales; D/8 lanes a row.  Rows past the unit's
    // are zero.
    auto stage_q = [&](int sg, const Segment &u) {
        wait(bar_at(c, kQFull), (uint32_t)(sg & 1));
        const int LR = D / 8, log2LR = 31 - __clz(LR);
        const int rows = q.n_q[u.b] * p.group;
        const int l = threadIdx.x & (LR - 1);
#pragma unroll 1
        for (int r = threadIdx.x >> log2LR; r < NR; r += kSoftmaxThreads >> log2LR) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (alive && r < rows)
                v = *reinterpret_cast<const uint4 *>(c.smem + L.qbuf + r * D * 2 + l * 16);
            const uint32_t xs[4] = {v.x, v.y, v.z, v.w};
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a = __vmaxu2(a, xs[i] & 0x7fff7fffu);
            a = max(a & 0xffffu, a >> 16);
            for (int o = LR / 2; o > 0; o >>= 1)
                a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
            int byte = (int)(a >> 7) - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0);
            byte = byte < 0 ? 0 : byte;
            const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = make_float2(__uint_as_float(xs[i] << 16) * inv,
                                             __uint_as_float(xs[i] & 0xffff0000u) * inv);
                const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
                const float2 hf = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
                const __nv_fp8x2_storage_t d = __nv_cvt_float2_to_fp8x2(make_float2(f.x - hf.x, f.y - hf.y),
                                                                        __NV_SATFINITE, __NV_E4M3);
                hi[i >> 1] = (i & 1) ? hi[i >> 1] | ((uint32_t)h << 16) : h;
                lo[i >> 1] = (i & 1) ? lo[i >> 1] | ((uint32_t)d << 16) : d;
            }
            const bool bad = a >= 0x7f80u;                // an infinity or a NaN: the row's scores are NaN
            if (bad)
                hi[0] = hi[1] = lo[0] = lo[1] = 0x7f7f7f7fu;
            if (alive) {
                uint8_t *dst = c.smem + L.qtile + (uint32_t)r * 128u + (((l >> 1) ^ (r & 7)) << 4) + (l & 1) * 8;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2 *>(dst + L.qhalf) = make_uint2(lo[0], lo[1]);
                if (l == 0)
                    scr[kScrQ * 64 + r] = bad ? 1.f : q8_scale((uint32_t)byte);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar_at(c, kQEmpty));
            mbar_arrive(bar_at(c, kQReady));
        }
    };

    // A wide stage (see the top), eight rows at a time: short loops with their
    // state in shared memory, as the common stage has the registers.  first: the
    // segment's first of the group; has_o: O holds earlier stages; pv_par: parity
    // of the group's previous product.  Leaves the new 7 - m, and in kScrAlpha
    // half of what the common stages' l takes (twice: where m rises by V's
    // exponents, up to 2^167, the weights so far can matter past fp32's least
    // normal number; what they brought to O does not).
    auto wide_stage = [&](float k_factor, int w4, bool first, bool has_o, int k, uint32_t pv_par, uint8_t *prow) {
        const int r = kPing ? t : (int)threadIdx.x;      // the row this thread keeps, below NR
        const int row_min = w4 & 0xff, vb = w4 >> 16;
        // V's codes, where the scale alone does not tell a zero row from one of tiny values
        wait(bar_at(c, kConvV + k % kVS), (uint32_t)(k / kVS) & 1u);
        bool zero = false;
        if (alive && vb == 0) {
            const uint8_t *row = c.smem + L.vring + (uint32_t)(k % kVS) * kVSlotBytes + (uint32_t)t * 128u;
            uint32_t any = 0;
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                const uint4 w = *reinterpret_cast<const uint4 *>(row + (i >> 3) * (kTT * 128) + (i & 7) * 16);
                any |= w.x | w.y | w.z | w.w;
            }
            zero = (any & 0x7fff7fffu) == 0u;
        }
        const float ev = zero ? -INFINITY : (float)(vb - 127);
        // y - ev of rows chunk_col(ch) .. + 7, -inf where not seen
        auto scores8 = [&](int ch, float (&x)[8]) {
            uint32_t sv[8];
            tmem_ld8_nowait(tmem + lane_base + kColS + (uint32_t)((k & 1) * 64 + chunk_col(ch)), sv);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = chunk_col(ch) + i;
                x[i] = row < row_min ? -INFINITY : __uint_as_float(sv[i]) * (k_factor * scr[kScrQ * 64 + row]);
            }
        };
        // the warp's maxima of x + add over its tokens -> kScrMax
        auto maxima = [&](float add) {
#pragma unroll 1
            for (int ch = 0; ch < NH / 8; ++ch) {
                float x[8];
                scores8(ch, x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] += add;
                ReduceScatter<8, 16, true>::run(x, lane);
                if (rs_owner<8>(lane))
                    mine[(kScrMax + tg) * 64 + chunk_col(ch) + rs_base<8>(lane)] = x[0];
            }
        };
        // the row's reference from the one before and kScrMax
        auto moved = [&](float old) {
            float top = -INFINITY;
#pragma unroll
            for (int g = 0; g < kTokenGroups; ++g)
                top = fmaxf(top, mine[(kScrMax + g) * 64 + r]);
            return old == -INFINITY || top > old + kRescaleLog2 ? top : old;
        };
        maxima(ev);
        named_barrier(bar_id, bar_threads);
        bool moves = false;
        float half = 1.f;
        if (r < NR) {
            const float mo = mine[kScrM * 64 + r], mn = moved(mo);
            if (first) {
                mine[kScrMl * 64 + r] = -INFINITY;
                mine[kScrL * 64 + r] = 0.f;
            }
            moves = mn != mo;
            mine[kScrNew * 64 + r] = mn == -INFINITY ? 1e30f : kPLog2 - mn;
            mine[kScrAlpha * 64 + r] = moves ? ex2_approx(mo - mn) : 1.f;
            half = moves ? ex2_approx(0.5f * (mo - mn)) : 1.f;
            mine[kScrM * 64 + r] = mn;
        }
        if (bar_red_or(bar_id, bar_threads, moves) && has_o) {
            wait(bar_at(c, kPvDone + grp), pv_par);
            if (alive) {
                tc_fence_after();
#pragma unroll 1
                for (int ch = 0; ch < NH / 8; ++ch) {
                    const uint32_t col = tmem + lane_base + kColO + (uint32_t)(grp * 64 + chunk_col(ch));
                    uint32_t ov[8];
                    tmem_ld8_nowait(col, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        ov[i] = __float_as_uint(__uint_as_float(ov[i]) * mine[kScrAlpha * 64 + chunk_col(ch) + i]);
                    tmem_st8_nowait(col, ov);
                }
                tmem_wait_st();
            }
        }
        maxima(0.f);
        named_barrier(bar_id, bar_threads);
        if (r < NR) {
            const float ml = mine[kScrMl * 64 + r], mn = moved(ml);
            if (mn != ml)
                mine[kScrL * 64 + r] *= ex2_approx(ml - mn);
            mine[kScrMl * 64 + r] = mn;
            mine[kScrAlpha * 64 + r] = half;
        }
        named_barrier(bar_id, bar_threads);
        if (k >= (kPing ? 2 : 1))
            wait(bar_at(c, kPvDone + grp), pv_par);
#pragma unroll 1
        for (int ch = 0; ch < NH / 8; ++ch) {
            float x[8], w[8];
            scores8(ch, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float m = mine[kScrM * 64 + chunk_col(ch) + i], ml = mine[kScrMl * 64 + chunk_col(ch) + i];
                w[i] = ex2_approx(x[i] + ev - (m == -INFINITY ? 0.f : m - kPLog2));
                x[i] = ex2_approx(x[i] - (ml == -INFINITY ? 0.f : ml - kPLog2));
            }
            if (alive)
                *reinterpret_cast<uint4 *>(prow + (((chunk_col(ch) / 8) ^ (t & 7)) << 4)) =
                    make_uint4(pack_half2(w[0], w[1]), pack_half2(w[2], w[3]), pack_half2(w[4], w[5]),
                               pack_half2(w[6], w[7]));
            ReduceScatter<8, 16, false>::run(x, lane);
            if (rs_owner<8>(lane))
                mine[(kScrMax + tg) * 64 + chunk_col(ch) + rs_base<8>(lane)] = x[0];
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar_at(c, kSFree + (k & 1)));
            mbar_arrive(bar_at(c, kPFull + grp));
        }
        named_barrier(bar_id, bar_threads);
        if (r < NR) {
            float sum = mine[kScrL * 64 + r];
#pragma unroll
            for (int g = 0; g < kTokenGroups; ++g)
                sum += mine[(kScrMax + g) * 64 + r];
            mine[kScrL * 64 + r] = sum;
        }
        named_barrier(bar_id, bar_threads);
    };

    int kbase = 0, seg = 0;
    Segment s = locate(p, c.cta_begin, c.cta_end);
    stage_q(0, s);
#pragma unroll 1
    for (;;) {
        const int nst = stages_of(s, P);
        const int R = q.n_q[s.b] * p.group;
        bool wide = false, had_wide = false;    // the group's stages from here on are; some were
        float2 nmu[kNmRegs ? NH / 2 : 1], l[NH / 2];   // 7 - m (1e30: no key yet), and this token's share of l
#pragma unroll
        for (int i = 0; i < NH / 2; ++i) {
            if (kNmRegs)
                nmu[kNmRegs ? i : 0] = make_float2(1e30f, 1e30f);
            l[i] = make_float2(0.f, 0.f);
        }
        if (threadIdx.x < NR)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                scr[(g * kScrGroup + kScrM) * 64 + threadIdx.x] = -INFINITY;
                scr[(g * kScrGroup + kScrNew) * 64 + threadIdx.x] = 1e30f;
            }
        named_barrier(kAllBar, kSoftmaxThreads);   // the rows' scales and initial maxima are in place

        // this group's first stage of the segment
        const int j0 = kPing ? (kbase ^ grp) & 1 : 0;
        const int tok_first = s.p0 * P, lim = min(plan_len(p, s), s.p1 * P), all_see = keys_all_see(q, s);
#pragma unroll 1
        for (int j = j0; j < nst; j += kPing ? 2 : 1) {
            const int k = kbase + j, buf = k & 1;
            // the token's factors and S^T
            float2 f;
            if (kPing) {
                const int slot = k % kScaleRing;
                wait(bar_at(c, kScaleB + slot), (uint32_t)(k / kScaleRing) & 1u);
                const uint8_t *sc = c.smem + L.scales + slot * 2 * kTT + scale_off(t, log2P);
                const uint32_t mask = meta[slot];
                const uint32_t four = *reinterpret_cast<const volatile uint32_t *>(sc_four + slot * 2 * kTT);
                const int kb = *(const volatile uint8_t *)sc, vb = *(const volatile uint8_t *)(sc + P);
                if (alive && (mask >> 8) != ((uint32_t)k & 0xffffffu)) {
                    if (lane == 0) {
                        atomicOr(p.err, SHKV_ERRF_PIPELINE);
                        *c.abort_flag = 1u;
                    }
                    alive = false;
                }
                const int tok0 = tok_first + j * kTT;
                f = token_factors(p, kb, vb, tok0 + t < lim && ((mask >> (t >> log2P)) & 1u), tok0 + t - all_see,
                                  stage_above(four, lim - tok0, mask & 0xffu, log2P));
            }
            if (wait(bar_at(c, kSFull + buf), (uint32_t)((k >> 1) & 1)))
                tc_fence_after();
            if (!kPing)
                f = reinterpret_cast<const float2 *>(c.smem + L.info)[(k % kInfo) * kTT + t];
            const int w4 = alive ? __float_as_int(f.y) : 64 | kMasked | 127 << 16;
            // the token's V exponent (a low token's: the window's least), and 2^-ev
            const int vc = max(w4 >> 16, 127 - kVWindow);
            const bool low = vc > w4 >> 16;
            const float ev = (float)(vc - 127), inv_ev = __uint_as_float((uint32_t)(254 - vc) << 23);
            const int row_min = w4 & 0xff;
            const bool masked = (w4 & kMasked) != 0;     // for some token of the warp
            uint8_t *prow = c.smem + L.pbuf + (uint32_t)grp * kPBytes + (uint32_t)t * 128u;
            const uint32_t pv_par = (uint32_t)(((kPing ? k >> 1 : k) - 1) & 1);   // of the group's previous product
            // y - m + 7 of this thread's rows (nm = 7 - m), -inf where not seen
            float2 d[NH / 2];
            auto scores = [&](bool relative) {       // (or y itself)
                const float2 ts2 = make_float2(f.x, f.x), ev2 = make_float2(ev, ev);
#pragma unroll
                for (int c0 = 0; c0 < NH / 8; c0 += kLoad) {
                    uint32_t sv[8 * kLoad];
#pragma unroll
                    for (int ch = 0; ch < kLoad; ++ch)
                        tmem_ld8_nowait(tmem + lane_base + kColS + (uint32_t)(buf * 64 + chunk_col(c0 + ch)), sv + 8 * ch);
                    tmem_wait_ld();
#pragma unroll
                    for (int ch = 0; ch < kLoad; ++ch) {
                        const float4 *rq = reinterpret_cast<const float4 *>(scr + kScrQ * 64 + chunk_col(c0 + ch));
                        const float4 qa = rq[0], qb = rq[1];
                        const float2 q2[4] = {make_float2(qa.x, qa.y), make_float2(qa.z, qa.w), make_float2(qb.x, qb.y),
                                              make_float2(qb.z, qb.w)};
                        float2 nm[4];
                        if (kNmRegs) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                nm[i] = nmu[kNmRegs ? 4 * (c0 + ch) + i : 0];
                        } else {
                            const float4 *sm = reinterpret_cast<const float4 *>(mine + kScrNew * 64 + chunk_col(c0 + ch));
                            const float4 na = sm[0], nb = sm[1];
                            nm[0] = make_float2(na.x, na.y);
                            nm[1] = make_float2(na.z, na.w);
                            nm[2] = make_float2(nb.x, nb.y);
                            nm[3] = make_float2(nb.z, nb.w);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int o = 4 * ch + i;
                            const float2 s2 = make_float2(__uint_as_float(sv[2 * o]), __uint_as_float(sv[2 * o + 1]));
                            d[4 * c0 + o] = __ffma2_rn(s2, __fmul2_rn(ts2, q2[i]), relative ? __fadd2_rn(ev2, nm[i]) : ev2);
                        }
                    }
                }
                if (masked)
#pragma unroll
                    for (int o = 0; o < NH / 2; ++o) {
                        d[o].x = row_of(2 * o) < row_min ? -INFINITY : d[o].x;
                        d[o].y = row_of(2 * o + 1) < row_min ? -INFINITY : d[o].y;
                    }
            };
            bool go_wide = wide, refresh = false;
            if (!wide) {
                scores(true);
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < NH / 2; ++i)
                    top = fmaxf(top, fmaxf(d[i].x, d[i].y));
                // all warps of the stage agree, also where one of them gave up waiting
                const bool lead = low && top > (w4 >> 16 ? kLeadLow : kLeadLeast);
                const bool need = lead || (w4 & kWide) != 0;
                refresh = bar_red_or(bar_id, bar_threads, need || (!low && top > kPLog2 + kRescaleLog2));
                if (refresh)
                    go_wide = bar_red_or(bar_id, bar_threads, need);
            }
            if (go_wide) {
                wide_stage(f.x, w4, !had_wide, j > j0, k, pv_par, prow);
                had_wide = true;
                wide = bar_red_or(bar_id, bar_threads, wide || (w4 & kWide) != 0);
#pragma unroll
                for (int i = 0; i < NH / 2; ++i) {
                    const int rr = row_of(2 * i);
                    if (kNmRegs)
                        nmu[kNmRegs ? i : 0] = make_float2(mine[kScrNew * 64 + rr], mine[kScrNew * 64 + rr + 1]);
                    const float2 half = make_float2(mine[kScrAlpha * 64 + rr], mine[kScrAlpha * 64 + rr + 1]);
                    l[i] = __fmul2_rn(__fmul2_rn(l[i], half), half);
                }
                continue;
            }
            // --- lazy refresh of the maxima
            if (refresh) {
                scores(false);
                {
                    constexpr int M = pow2_at_least(NH);
                    float v[M];
#pragma unroll
                    for (int i = 0; i < M; ++i)
                        v[i] = i < NH ? ((i & 1) ? d[(i < NH ? i : 0) / 2].y : d[(i < NH ? i : 0) / 2].x) : -INFINITY;
                    ReduceScatter<M, 16, true>::run(v, lane);
                    const int base = rs_base<M>(lane);
                    if (rs_owner<M>(lane))
#pragma unroll
                        for (int jj = 0; jj < (M >= 32 ? M / 32 : 1); ++jj)
                            if (base + jj < NH)
                                mine[(kScrMax + tg) * 64 + row_of(base + jj)] = v[jj];
                }
                named_barrier(bar_id, bar_threads);
                const int r = kPing ? t : (int)threadIdx.x;
                if (r < NR) {
                    const float mo = mine[kScrM * 64 + r];
                    float mn = mo;
#pragma unroll
                    for (int g = 0; g < kTokenGroups; ++g)
                        mn = fmaxf(mn, mine[(kScrMax + g) * 64 + r]);
                    mine[kScrNew * 64 + r] = mn == -INFINITY ? 1e30f : kPLog2 - mn;
                    mine[kScrAlpha * 64 + r] = mn == -INFINITY ? 1.f : ex2_approx(mo - mn);
                    mine[kScrM * 64 + r] = mn;
                }
                named_barrier(bar_id, bar_threads);
                if (j > j0) {
                    // O^T holds the group's stages before: rescale this thread's part once their PV is done
                    wait(bar_at(c, kPvDone + grp), pv_par);
                    if (alive) {
                        tc_fence_after();
#pragma unroll
                        for (int ch = 0; ch < NH / 8; ++ch) {
                            const uint32_t col = tmem + lane_base + kColO + (uint32_t)(grp * 64 + chunk_col(ch));
                            uint32_t ov[8];
                            tmem_ld8_nowait(col, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                ov[i] = __float_as_uint(__uint_as_float(ov[i]) * mine[kScrAlpha * 64 + chunk_col(ch) + i]);
                            tmem_st8_nowait(col, ov);
                        }
                        tmem_wait_st();
                    }
                }
#pragma unroll
                for (int i = 0; i < NH / 2; ++i) {
                    const int rr = row_of(2 * i);
                    const float2 nm = make_float2(mine[kScrNew * 64 + rr], mine[kScrNew * 64 + rr + 1]);
                    if (kNmRegs)
                        nmu[kNmRegs ? i : 0] = nm;
                    d[i] = __fadd2_rn(d[i], nm);
                    l[i] = __fmul2_rn(l[i], make_float2(mine[kScrAlpha * 64 + rr], mine[kScrAlpha * 64 + rr + 1]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_at(c, kSFree + buf));
            uint32_t pk[NH / 2];
#pragma unroll
            for (int i = 0; i < NH / 2; ++i) {
                const float2 pe = make_float2(ex2_approx(d[i].x), ex2_approx(d[i].y));
                l[i] = __ffma2_rn(pe, make_float2(inv_ev, inv_ev), l[i]);
                pk[i] = pack_half2(pe.x, pe.y);
            }
            if (low)
#pragma unroll
                for (int i = 0; i < NH / 2; ++i)
                    pk[i] = 0u;
            // --- P^T, once the group's previous product has read the buffer
            if (k >= (kPing ? 2 : 1))
                wait(bar_at(c, kPvDone + grp), pv_par);
            if (alive) {
#pragma unroll
                for (int ch = 0; ch < NH / 8; ++ch)
                    *reinterpret_cast<uint4 *>(prow + (((chunk_col(ch) / 8) ^ (t & 7)) << 4)) =
                        make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar_at(c, kPFull + grp));
        }

        // --- next segment's query rows, as soon as the last QK of this one is done
        const bool has_next = s.seg_end < c.cta_end;
        Segment sn;
        if (has_next) {
            sn = next_segment(p, s, c.cta_end);
            wait(bar_at(c, kQTileFree), (uint32_t)(seg & 1));
            named_barrier(kAllBar, kSoftmaxThreads);  // every warp is past its last use of the rows' scales
            stage_q(seg + 1, sn);
        }

        // --- segment end: row sums across the 128 tokens
        {
            constexpr int M = pow2_at_least(NH);
            float v[M];
#pragma unroll
            for (int i = 0; i < M; ++i)
                v[i] = i < NH ? ((i & 1) ? l[(i < NH ? i : 0) / 2].y : l[(i < NH ? i : 0) / 2].x) : 0.f;
            ReduceScatter<M, 16, false>::run(v, lane);
            const int base = rs_base<M>(lane);
            if (rs_owner<M>(lane))
#pragma unroll
                for (int jj = 0; jj < (M >= 32 ? M / 32 : 1); ++jj)
                    if (base + jj < NH)
                        mine[(kScrMax + tg) * 64 + row_of(base + jj)] = v[jj];
        }
        if (t == 0 && (kPing || warp == 0))
            *reinterpret_cast<int *>(scr + kScrWide * 64 + grp) = had_wide;
        named_barrier(kAllBar, kSoftmaxThreads);
        const bool whole = (s.seg_begin == s.unit_begin) && (s.seg_end == s.unit_end);
        const int slot_id = whole ? 0 : 2 * (int)blockIdx.x + (s.seg_begin == c.cta_begin ? 0 : 1);
        const int64_t row0 = (int64_t)q.q0[s.b] * p.hq + (int64_t)s.g * p.group;
        const int *rowoff = scr_i + kScrOff * 64;
        if (threadIdx.x < NR) {
            const int r = threadIdx.x;
            // the groups' parts, relative to the larger reference of their sums
            float m[2], a[2], ref[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float *o = scr + g * kScrGroup * 64;
                m[g] = ref[g] = -INFINITY;
                a[g] = 0.f;
                if (kPing || g == 0) {
                    m[g] = ref[g] = o[kScrM * 64 + r];
#pragma unroll
                    for (int i = 0; i < kTokenGroups; ++i)
                        a[g] += o[(kScrMax + i) * 64 + r];
                    if (scr_i[kScrWide * 64 + g]) {
                        // the larger of the common and the wide stages' parts decides, by its exponent (a sum may
                        // be 2^-120 beside its reference, see the wide stage)
                        const float ml = o[kScrMl * 64 + r];
                        const float b = o[kScrL * 64 + r];
                        const float ta = a[g] > 0.f ? m[g] + (float)ilogbf(a[g]) : -INFINITY;
                        const float tb = b > 0.f ? ml + (float)ilogbf(b) : -INFINITY;
                        ref[g] = fmaxf(ta, tb);
                        const float ha = ta == -INFINITY ? 1.f : ex2_approx(0.5f * (m[g] - ref[g]));
                        const float hb = tb == -INFINITY ? 1.f : ex2_approx(0.5f * (ml - ref[g]));
                        a[g] = a[g] * ha * ha + b * hb * hb;     // (NaN where one is)
                    }
                }
            }
            const float mm = fmaxf(ref[0], ref[1]);
            float sum = 0.f;
#pragma unroll
            for (int g = 0; g < 2; ++g)
                sum += ref[g] == -INFINITY ? a[g] : a[g] * ex2_approx(ref[g] - mm);
            const float inv = sum != 0.f ? __frcp_rn(sum) : 0.f;     // (a NaN sum stays NaN)
            // 2^(m - mm), in two halves: itself it can leave fp32's range, up to 2^135 or under
            // 2^-126, where its product with O does not
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float half = m[g] == -INFINITY ? 0.f : ex2_approx(0.5f * (m[g] - mm));
                scr[(kScrEnd + 2 * g) * 64 + r] = half * inv;
                scr[(kScrEnd + 2 * g + 1) * 64 + r] = half;
            }
            if (alive && r < R) {
                const float lse = sum != 0.f ? ((mm == -INFINITY ? 0.f : mm - kPLog2) + log2f(sum)) * kLn2
                                             : -INFINITY;
                if (whole) {
                    if (p.lse_out)
                        p.lse_out[row0 + rowoff[r]] = lse;
                } else {
                    p.ws_lse[(int64_t)slot_id * p.rows + r] = lse;
                }
            }
        }
        named_barrier(kAllBar, kSoftmaxThreads);

        // --- column d = t of O^T for half the rows, normalised
        float o[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i)
            o[i] = 0.f;
#pragma unroll
        for (int g = 0; g < (kPing ? 2 : 1); ++g) {
            // the group's last stage of the segment, if it had one
            const int last = kPing ? nst - 1 - ((kbase + nst - 1 + g) & 1) : nst - 1;
            if (last < 0)
                continue;
            wait(bar_at(c, kPvDone + g), (uint32_t)((kPing ? (kbase + last) >> 1 : kbase + last) & 1));
            if (alive) {
                tc_fence_after();
                uint32_t ov[NE];
                tmem_ld_half<NE>(tmem + lane_base + kColO + (uint32_t)(g * 64), hh, ov);
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    o[i] = fmaf(__uint_as_float(ov[i]) * 256.f * scr[(kScrEnd + 2 * g + 1) * 64 + half_row(hh, i)],
                                scr[(kScrEnd + 2 * g) * 64 + half_row(hh, i)], o[i]);
            }
        }
        if (alive && t < D) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int r = half_row(hh, i);
                if (r < R) {
                    if (!whole)
                        p.ws_part[((int64_t)slot_id * p.rows + r) * D + t] = o[i];
                    else
                        p.out[(row0 + rowoff[r]) * D + t] = __float2bfloat16_rn(o[i]);
                }
            }
        }
        tc_fence_before();
        named_barrier(kAllBar, kSoftmaxThreads);

        kbase += nst;
        ++seg;
        if (!has_next)
            break;
        s = sn;
    }

    // --- split units: the last piece to arrive merges all pieces.  A CTA's
    // first and last segments can be pieces; both arrive here, after the last,
    // under one fence (3.5K cycles, which the first would pay alone before the
    // next segment's stages).
    const Segment first = locate(p, c.cta_begin, c.cta_end);
    const bool split[2] = {seg > 1 && first.seg_begin != first.unit_begin,
                           s.seg_begin != s.unit_begin || s.seg_end != s.unit_end};
    if (!split[0] && !split[1])
        return;
    if (threadIdx.x == 0) {
        uint32_t before[2] = {0u, 0u}, last = 0u;
        __threadfence();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (split[i])
                before[i] = atomicAdd(p.ws_count + (int64_t)(i ? s.b : first.b) * p.hkv + (i ? s.g : first.g), 1u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Segment &u = i ? s : first;
            if (split[i] && before[i] == (uint32_t)(cta_of(p, u.unit_end - 1) - cta_of(p, u.unit_begin)))
                last |= 1u << i;
        }
        *c.bcast = last;
    }
    named_barrier(kAllBar, kSoftmaxThreads);
    const uint32_t mine_last = *c.bcast;
    if (mine_last)
        __threadfence();
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        if (!((mine_last >> i) & 1u))
            continue;
        const int b = i ? s.b : first.b, g = i ? s.g : first.g;
        const int64_t unit_begin = i ? s.unit_begin : first.unit_begin;
        const int cb = cta_of(p, unit_begin), ce = cta_of(p, (i ? s.unit_end : first.unit_end) - 1);
        const int R = q.n_q[b] * p.group, dq = D / 4;
        const int64_t row0 = (int64_t)q.q0[b] * p.hq + (int64_t)g * p.group;
        const int *rowoff = scr_i + kScrOff * 64;
        // kMerge rows of a warp at a time: their loads in flight together (one
        // row at a time, 32 rows took 6 us)
#pragma unroll 1
        for (int r0 = warp; r0 < R; r0 += kMerge * kSoftmaxWarps) {
            float M[kMerge];                             // NaN as soon as a piece's log-sum-exp is
#pragma unroll
            for (int m = 0; m < kMerge; ++m)
                M[m] = -INFINITY;
#pragma unroll 1
            for (int cc = cb + lane; cc <= ce; cc += 32) {
                const float *lse = p.ws_lse + (int64_t)piece_slot(p, cc, unit_begin) * p.rows;
#pragma unroll
                for (int m = 0; m < kMerge; ++m)
                    if (r0 + m * kSoftmaxWarps < R)
                        M[m] = max_nan(M[m], __ldcg(lse + r0 + m * kSoftmaxWarps));
            }
#pragma unroll
            for (int o_ = 16; o_ > 0; o_ >>= 1)
#pragma unroll
                for (int m = 0; m < kMerge; ++m)
                    M[m] = max_nan(M[m], __shfl_xor_sync(0xffffffffu, M[m], o_));
            float wsum[kMerge];
            float4 acc[kMerge];
#pragma unroll
            for (int m = 0; m < kMerge; ++m) {
                wsum[m] = 0.f;
                acc[m] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll 1
            for (int cc = cb; cc <= ce; ++cc) {
                const int64_t pr = (int64_t)piece_slot(p, cc, unit_begin) * p.rows + r0;
                float x[kMerge];
                float4 v[kMerge];
#pragma unroll
                for (int m = 0; m < kMerge; ++m) {
                    const bool in = r0 + m * kSoftmaxWarps < R;
                    x[m] = in ? __ldcg(p.ws_lse + pr + m * kSoftmaxWarps) : -INFINITY;
                    v[m] = in && lane < dq
                                ? __ldcg(reinterpret_cast<const float4 *>(p.ws_part + (pr + m * kSoftmaxWarps) * D) + lane)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int m = 0; m < kMerge; ++m) {
                    // (no piece has a key the row sees: weights of 0; else of 2^-10
                    // at most: sums of outputs near fp32's largest stay below it)
                    const float w = M[m] == -INFINITY ? 0.f : ex2_approx((x[m] - M[m]) * 1.4426950408889634f) * 0x1p-10f;
                    wsum[m] += w;
                    acc[m].x += w * v[m].x;
                    acc[m].y += w * v[m].y;
                    acc[m].z += w * v[m].z;
                    acc[m].w += w * v[m].w;
                }
            }
#pragma unroll
            for (int m = 0; m < kMerge; ++m) {
                const int rr = r0 + m * kSoftmaxWarps;
                if (rr >= R)
                    continue;
                const float winv = wsum[m] != 0.f ? 1.f / wsum[m] : 0.f;
                const int64_t orr = row0 + rowoff[rr];
                if (lane < dq)
                    *reinterpret_cast<uint2 *>(p.out + orr * D + lane * 4) =
                        make_uint2(pack_bf16x2(acc[m].x * winv, acc[m].y * winv),
                                   pack_bf16x2(acc[m].z * winv, acc[m].w * winv));
                if (lane == 0 && p.lse_out)
                    p.lse_out[orr] = wsum[m] != 0.f ? M[m] + logf(wsum[m] * 0x1p10f) : -INFINITY;
            }
        }
        if (threadIdx.x == 0)
            p.ws_count[(int64_t)b * p.hkv + g] = 0u;
    }
}

// Rows of requests that hold no key: zeros and -inf.
__device__ void write_empty(const Q8DecodeParams &q)
{
    const DecodeParams &p = q.d;
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        if (p.page_prefix[b + 1] != p.page_prefix[b])
            continue;
        const int64_t r0 = (int64_t)q.q0[b] * p.hq, rows = (int64_t)q.n_q[b] * p.hq;
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + r0 * q.head_dim);
        for (int64_t i = threadIdx.x; i < rows * q.head_dim / 8; i += kSoftmaxThreads)
            dst[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse_out)
            for (int64_t i = threadIdx.x; i < rows; i += kSoftmaxThreads)
                p.lse_out[r0 + i] = -INFINITY;
    }
}

}  // namespace

template <int NR>
__global__ void __launch_bounds__(kThreads, 1)
    shkv_q8_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ Q8DecodeParams q)
{
    extern __shared__ uint8_t smem_raw[];
    const DecodeParams &p = q.d;
    Ctx4 c;
    {
        const uint32_t raw = smem_u32(smem_raw);
        const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
        c.smem = smem_raw + pad;
        c.base = raw + pad;
    }
    constexpr Smem L = smem_layout(NR);
    c.bars = c.base + L.bars;
    c.abort_flag = reinterpret_cast<volatile uint32_t *>(c.smem + L.misc);
    c.bcast = reinterpret_cast<uint32_t *>(c.smem + L.misc + 4);
    c.cta_begin = p.cta_cut[blockIdx.x];
    c.cta_end = p.cta_cut[blockIdx.x + 1];
    const bool work = c.cta_begin < c.cta_end;
    const int warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        constexpr uint32_t kStageWarps = q_pingpong(NR) ? kSoftmaxWarps / 2 : kSoftmaxWarps;   // that take a stage
#pragma unroll 1
        for (int i = 0; i < kBars; ++i) {
            uint32_t n = 1;
            if (i >= kConvV && i < kEmptyV || i >= kInfoB && i < kPFull)
                n = kConvWarps;
            else if (i >= kPFull && i < kPvDone || i >= kSFree && i < kQReady)
                n = kStageWarps;
            else if (i >= kScaleB && i < kInfoB)
                n = 33;                      // the K warp's lanes' copies and the validity word
            else if (i == kQEmpty || i == kQReady)
                n = kSoftmaxWarps;
            else if (i >= kSFull && i < kSFree)
                n = q_pingpong(NR) ? 1 : 2;  // the QK's commit, and its issuer where it passes factors on
            else if (i == kFin)
                n = 2;                       // one commit per issuer
            mbar_init(bar_at(c, i), n);
        }
        *c.abort_flag = 0u;
        *c.bcast = 0u;
        fence_barrier_init();
    }
    if (threadIdx.x < 64) {
        const int r = threadIdx.x;
        reinterpret_cast<int *>(c.smem + L.scr)[kScrOff * 64 + r] = r / p.group * p.hq + r % p.group;
    }
    if (warp == 0)
        tmem_alloc(c.base + L.tslot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(c.smem + L.tslot);
    if (work && warp == kKWarp)
        warm_l2_q8(&tmK, p, c, kKS);
    else if (work && warp == kVWarp)
        warm_l2_q8(&tmV, p, c, kVS);
    pdl_wait_prior();                       // global memory only from here on
    pdl_launch_dependents();                // (after the wait: see launch.cuh)

    if (warp < kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        if (q.has_empty)
            write_empty(q);
        if (work)
            softmax_q8<NR>(q, c, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (work) {
            if (warp == kKWarp)
                producer_q8<NR, true>(&tmK, q, c);
            else if (warp == kVWarp)
                producer_q8<NR, false>(&tmV, q, c);
            else if (warp == kQkWarp) {
                if ((threadIdx.x & 31) == 0)
                    qk_issuer<NR>(q, c, tmem);
            } else if (warp == kPvWarp) {
                if ((threadIdx.x & 31) == 0)
                    pv_issuer<NR>(q, c, tmem);
            } else {
                convert_v<NR>(q, c);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {

template <int NR>
cudaError_t launch_nr(const CUtensorMap &tmK, const CUtensorMap &tmV, const Q8DecodeParams &q, cudaStream_t stream)
{
    static std::atomic<int> known;
    int regs;                  // the register split hands out exactly the launch's 128 a thread
    cudaError_t e = kernel_registers(shkv_q8_decode_kernel<NR>, known, &regs);
    if (e != cudaSuccess)
        return e;
    if ((uint32_t)regs * kThreads != kSoftmaxRegs * 256 + kOtherRegs * 256)
        return cudaErrorInvalidConfiguration;
    constexpr uint32_t smem = smem_layout(NR).total;
    e = cudaFuncSetAttribute(shkv_q8_decode_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(shkv_q8_decode_kernel<NR>, q.d.num_ctas, kThreads, smem, stream, tmK, tmV, q);
}

}  // namespace

// tmK, tmV: 2-D maps of the code pools (box of 128 bytes x P rows, 128-byte swizzle).
cudaError_t launch_q8_decode(const CUtensorMap &tmK, const CUtensorMap &tmV, const Q8DecodeParams &q, cudaStream_t stream)
{
    switch (q_nr(q.d.rows)) {
    case 16:
        return launch_nr<16>(tmK, tmV, q, stream);
    case 32:
        return launch_nr<32>(tmK, tmV, q, stream);
    case 48:
        return launch_nr<48>(tmK, tmV, q, stream);
    case 64:
        return launch_nr<64>(tmK, tmV, q, stream);
    default:
        return cudaErrorInvalidValue;
    }
}

}  // namespace shkv
