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
//   O^T[d, r] += sum_t v8[t, d] P^T[t, r]                         kind::f16
//   l[r]      += sum_t P^T[t, r] * 2^(E - ev[t])                  (P before its rounding)
//   out = O^T * 2^E / l,   lse = ln2 * (m - 7 - E + log2(l))
//
// K's codes go to the tensor cores as they lie in the page.  A bf16 query has
// 8 significant bits: its row is scaled by a power of two to at most 448 and
// split into two e4m3 terms, qh nearest and ql = q - qh, which is exact but
// for values under 2^-15 of the row's largest.  V's codes are widened to fp16
// in shared memory, exactly.  With the token's V exponent inside y, P is
// relative to the row's largest weight times value scale, so that fp16 holds
// 11 bits of every token that matters to the sum, whatever the magnitudes of
// weights and values apart: fp16's least step, 2^-24, is 2^-31 of that
// largest, and 2^20 tokens below it are lost to 2^-12 of it.  E, a running
// upper bound (at least 2^-67) of the V exponents of the segment's keys that
// every row sees, keeps the fp32 sums l at 2^7 or more; a draft's key, which
// some rows only see, may exceed it by 2^100.  A token whose V exponent is
// under E - 60 takes part with V = 0 and that exponent, which bounds l's terms
// by 2^75; where E rises over tokens already summed, m is kept high enough for
// 2^97 (b[r] is that bound).  Sums and O are fp32.
//
// Roles (512 threads):
//   warps 0-7    softmax: warp w owns tokens 32*(w%4) .. +31 and half w/4 of
//                the rows; also stages the query rows and reads O^T out
//   warp 8       QK issuer (one lane)
//   warp 9       producer of K pages, scales, query rows and validity words
//   warp 10      PV issuer (one lane)
//   warp 11      producer of V pages
//   warps 12-15  V conversion, one token a thread: the codes land in the upper
//                16 KB of a 32 KB slot, where the thread reads its row and
//                writes it back as fp16 over both halves (row t's codes lie
//                inside row t's fp16 bytes, so no thread waits for another)
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "decode_common.cuh"
#include "launch.cuh"
#include "q8_decode.cuh"
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
constexpr int kMinE = 60;                   // scale byte of the least E
constexpr int kEHeadroom = 4;               // E moves to this much above a stage's largest V exponent
constexpr int kVWindow = 60;                // V exponents under E - 60 count as zero values
constexpr float kTermLog2 = kVWindow + kRescaleLog2;   // a new term of l is at most 2^(this + 7)
constexpr float kMaxTermLog2 = 90.f;        // ... and stays at most 2^(this + 7): 2^20 of them fit fp32
constexpr uint32_t kKSlotBytes = kTT * 128;
constexpr uint32_t kVSlotBytes = 2 * kTT * 128;
constexpr int kScaleRing = 8;               // see the note at the producer
constexpr int kMaxKSlots = 4;
static_assert(kMaxKSlots + 4 <= kScaleRing, "scales of a stage live until its V is converted");
// registers: 168 for the softmax warpgroups, 88 for the other two, of the
// launch's 128 a thread
constexpr uint32_t kSoftmaxRegs = 168, kOtherRegs = 88;
static_assert(kSoftmaxRegs * 256 + kOtherRegs * 256 == 128 * kThreads, "register split");

// scratch rows of 64 words
constexpr int kScrMax = 0, kScrNew = 4, kScrAlpha = 5, kScrL = 6, kScrM = 10, kScrInv = 11, kScrQ = 12, kScrOff = 13,
              kScrAlphaL = 14, kScrB = 15, kScrRows = 16;

__host__ __device__ constexpr int q_nr(int rows) { return (rows + 15) / 16 * 16; }
// N of the PV MMA: 48 is rounded up to a whole 64-column swizzle span.
__host__ __device__ constexpr int q_npv(int nr) { return nr == 48 ? 64 : nr; }

struct Smem {
    uint32_t kring, vring, pbuf, qtile, qhalf, qbuf, scr, scales, bars, meta, misc, tslot, total;
};

// K ring, V ring (slots [half][128 tokens][128 B]), P^T [128 tokens][128 B]
// and the query tiles [qh | ql][NR rows][128 B] are 128-byte swizzled; qbuf
// holds the next segment's bf16 query rows.
__host__ __device__ inline Smem smem_layout(int rows, int head_dim, int ks, int vs)
{
    Smem u;
    u.kring = 0;
    u.vring = u.kring + (uint32_t)ks * kKSlotBytes;
    u.pbuf = u.vring + (uint32_t)vs * kVSlotBytes;
    u.qtile = u.pbuf + kTT * 128;
    u.qhalf = (uint32_t)q_nr(rows) * 128u;
    u.qbuf = u.qtile + 2 * u.qhalf;
    u.scr = align_up(u.qbuf + (uint32_t)(rows * head_dim * 2), 128);
    u.scales = u.scr + kScrRows * 64 * 4;
    u.bars = u.scales + kScaleRing * 2 * kTT;
    // full_k[ks], empty_k[ks], full_v[vs], conv[vs], empty_v[vs], scale[ring],
    // p_full, pv_done, qfull, qempty, s_full[2], s_free[2], q_ready, q_tile_free, fin
    u.meta = u.bars + (uint32_t)(2 * ks + 3 * vs + kScaleRing + 11) * 8u;
    u.misc = u.meta + kScaleRing * 4;
    u.tslot = u.misc + 8;
    u.total = u.misc + 16 + 1024;           // + slack to align the base to 1024 bytes
    return u;
}

struct Ctx4 {
    uint8_t *smem;
    uint32_t base;
    Smem lay;
    int ks, vs;
    volatile uint32_t *abort_flag;
    uint32_t *bcast;
    int64_t cta_begin, cta_end;
};

__device__ __forceinline__ uint32_t bar_at(const Ctx4 &c, int i) { return c.base + c.lay.bars + 8u * i; }
__device__ __forceinline__ uint32_t full_k(const Ctx4 &c, int s) { return bar_at(c, s); }
__device__ __forceinline__ uint32_t empty_k(const Ctx4 &c, int s) { return bar_at(c, c.ks + s); }
__device__ __forceinline__ uint32_t full_v(const Ctx4 &c, int s) { return bar_at(c, 2 * c.ks + s); }
__device__ __forceinline__ uint32_t conv_v(const Ctx4 &c, int s) { return bar_at(c, 2 * c.ks + c.vs + s); }
__device__ __forceinline__ uint32_t empty_v(const Ctx4 &c, int s) { return bar_at(c, 2 * c.ks + 2 * c.vs + s); }
__device__ __forceinline__ uint32_t scale_b(const Ctx4 &c, int i) { return bar_at(c, 2 * c.ks + 3 * c.vs + i); }
__device__ __forceinline__ uint32_t tail_b(const Ctx4 &c, int i) { return scale_b(c, kScaleRing + i); }
__device__ __forceinline__ uint32_t p_full(const Ctx4 &c) { return tail_b(c, 0); }
__device__ __forceinline__ uint32_t pv_done(const Ctx4 &c) { return tail_b(c, 1); }
__device__ __forceinline__ uint32_t qfull(const Ctx4 &c) { return tail_b(c, 2); }
__device__ __forceinline__ uint32_t qempty(const Ctx4 &c) { return tail_b(c, 3); }
__device__ __forceinline__ uint32_t s_full(const Ctx4 &c, int b) { return tail_b(c, 4 + b); }
__device__ __forceinline__ uint32_t s_free(const Ctx4 &c, int b) { return tail_b(c, 6 + b); }
__device__ __forceinline__ uint32_t q_ready(const Ctx4 &c) { return tail_b(c, 8); }
__device__ __forceinline__ uint32_t q_tile_free(const Ctx4 &c) { return tail_b(c, 9); }
__device__ __forceinline__ uint32_t fin_b(const Ctx4 &c) { return tail_b(c, 10); }
__device__ __forceinline__ uint32_t k_slot(const Ctx4 &c, int s) { return c.base + c.lay.kring + (uint32_t)s * kKSlotBytes; }
__device__ __forceinline__ uint32_t v_slot(const Ctx4 &c, int s) { return c.base + c.lay.vring + (uint32_t)s * kVSlotBytes; }
__device__ __forceinline__ uint32_t ring_par(int k, int n) { return (uint32_t)((k / n) & 1); }

__device__ __forceinline__ int stages_of(const Segment &s, int P) { return ((s.p1 - s.p0) * P + kTT - 1) / kTT; }

// The stage's scale bytes of token t: K's and V's ([page][K, V][P] as in the pool).
__device__ __forceinline__ uint32_t scale_at(const Ctx4 &c, int k, int t, int log2P, int kv)
{
    const uint32_t off = (uint32_t)(((t >> log2P) << (log2P + 1)) + (kv << log2P) + (t & ((1 << log2P) - 1)));
    return reinterpret_cast<const volatile uint8_t *>(c.smem + c.lay.scales)[(k % kScaleRing) * 2 * kTT + off];
}

// Largest V scale byte of the stage's tokens below `n` on copied pages (NaN
// rows, 255, aside), by a warp; 0 if there are none.
__device__ __forceinline__ int stage_top_scale(const Ctx4 &c, int k, int n, uint32_t mask, int log2P)
{
    const int t = 4 * (threadIdx.x & 31);
    const uint32_t off = (uint32_t)(((t >> log2P) << (log2P + 1)) + (1 << log2P) + (t & ((1 << log2P) - 1)));
    const uint32_t w = *reinterpret_cast<const volatile uint32_t *>(c.smem + c.lay.scales + (k % kScaleRing) * 2 * kTT + off);
    const int in = ((mask >> (t >> log2P)) & 1u) ? n - t : 0;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = i < in ? (w >> (8 * i)) & 0xffu : 0u;
        top = max(top, b == 255u ? 0u : b);
    }
    return (int)__reduce_max_sync(0xffffffffu, top);
}

// Keys below this are seen by every row of the unit.
__device__ __forceinline__ int keys_all_see(const Q8DecodeParams &q, const Segment &s)
{
    const int L = plan_len(q.d, s);
    return q.causal ? L - q.n_q[s.b] + 1 : L;
}

// E (as a scale byte) from the one before and a stage's largest scale byte.
__device__ __forceinline__ int next_e(int e, int top) { return top > e ? min(top + kEHeadroom, 254) : e; }

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

// Two e4m3 codes (low 16 bits) as fp16.
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t codes)
{
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// ---------------------------------------------------------------------------
// producers
// ---------------------------------------------------------------------------
// Stage j of a segment is the 128 tokens from p0*P + j*128.  One lane copies
// one page (a box of P rows x 128 bytes; at head_dim 64 the box's upper half
// is outside the tensor and filled with zeros).  The K warp also copies each
// page's 2P scale bytes and publishes the stage's validity word, on barriers
// of a ring of their own: a stage's scales are read by the softmax and by the
// V conversion, after its K slot may have been refilled.  The K warp writes
// entry k once QK(k - KS) is complete; QK(i) is issued after the softmax has
// read S and the scales of stage i - 2, and its P of stage i - 3 waits for
// PV(i - 4), whose V was converted: entries up to k - KS - 4 are free.
template <bool kIsK>
__device__ void producer_q8(const CUtensorMap *tm, const Q8DecodeParams &q, const Ctx4 &c)
{
    const DecodeParams &p = q.d;
    const int lane = threadIdx.x & 31;
    const int P = p.page_size, RB = kTT / P, log2P = 31 - __clz(P);
    const int slots = kIsK ? c.ks : c.vs;
    const uint64_t pol = l2_evict_first_policy();
    if (lane == 0)
        prefetch_tensormap(tm);
    bool alive = true;
    int kbase = 0, seg = 0, last_issued = -1, q_issued = -1;
    Segment s = locate(p, c.cta_begin, c.cta_end);
    int pre = unit_entry(p.block_table, p, s.b, s.p0 + lane, s.p1);
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
                const bool ok = mbar_wait_bounded(qempty(c), (uint32_t)((seg & 1) ^ 1), c.abort_flag, p.err);
                alive = __all_sync(0xffffffffu, ok);
            }
            if (alive) {
                const int n = q.n_q[s.b];
                const uint32_t bytes = (uint32_t)(p.group * q.head_dim * 2);
                if (lane == 0)
                    mbar_arrive_expect_tx(qfull(c), bytes * (uint32_t)n);
                __syncwarp();
                const __nv_bfloat16 *src = p.q + (int64_t)q.q0[s.b] * q.q_stride + (int64_t)s.g * p.group * q.head_dim;
                for (int i = lane; i < n; i += 32)
                    bulk_load(c.base + c.lay.qbuf + (uint32_t)i * bytes, src + (int64_t)i * q.q_stride, bytes, qfull(c));
                q_issued = seg;
            }
        }
        const int nst = stages_of(s, P);
        int w0 = s.p0;                                   // block-table window [w0, w0+32)
        int cur = pre;
        int nxt = unit_entry(p.block_table, p, s.b, w0 + 32 + lane, s.p1);
        for (int j = 0; j < nst; ++j) {
            const int k = kbase + j, slot = k % slots;
            const int page0 = s.p0 + j * RB;
            if (page0 >= w0 + 32) {                      // a stage's pages never straddle a window
                w0 += 32;
                cur = nxt;
                nxt = unit_entry(p.block_table, p, s.b, w0 + 32 + lane, s.p1);
            }
            const int id = __shfl_sync(0xffffffffu, cur, (page0 + lane - w0) & 31);
            bool ok = true;
            if (alive)
                ok = mbar_wait_bounded(kIsK ? empty_k(c, slot) : empty_v(c, slot), ring_par(k, slots) ^ 1u,
                                       c.abort_flag, p.err);
            alive = alive && __all_sync(0xffffffffu, ok);
            const bool inside = lane < RB && page0 + lane < s.p1;
            const bool valid = inside && id >= 0 && id < p.num_pages;
            const uint32_t mask = __ballot_sync(0xffffffffu, valid);
            if (kIsK && alive && inside && !valid)
                atomicOr(p.err, SHKV_ERRF_PAGE_OOB);
            const uint32_t bar = kIsK ? full_k(c, slot) : full_v(c, slot);
            const uint32_t sbar = scale_b(c, k % kScaleRing);
            if (alive && lane == 0) {
                const uint32_t pages = (uint32_t)__popc(mask);
                if (kIsK) {
                    reinterpret_cast<volatile uint32_t *>(c.smem + c.lay.meta)[k % kScaleRing] =
                        mask | ((uint32_t)k << 8);       // valid pages + stage tag
                    mbar_arrive_expect_tx(sbar, pages * 2u * (uint32_t)P);
                }
                mbar_arrive_expect_tx(bar, pages * (uint32_t)P * 128u);
            }
            __syncwarp();
            if (alive && valid) {
                const int unit = id * p.hkv + s.g;
                const uint32_t dst = (kIsK ? k_slot(c, slot) : v_slot(c, slot) + kTT * 128u) + (uint32_t)(lane * P) * 128u;
                tma_load_2d(dst, tm, 0, unit * P, bar, pol);
                if (kIsK)
                    bulk_load(c.base + c.lay.scales + (uint32_t)((k % kScaleRing) * 2 * kTT + lane * 2 * P),
                              q.scales + (int64_t)unit * 2 * P, 2u * (uint32_t)P, sbar);
            }
            if (alive)
                last_issued = k;
            __syncwarp();
        }
        if (kIsK && lane == 0 && dev_len != plan_len(p, s))
            atomicOr(p.err, SHKV_ERRF_SEQ_LEN);
        kbase += nst;
        ++seg;
        if (!has_next)
            break;
        s = sn;
        pre = pre_next;
    }
    // After an abort, wait (bounded) for the copies still in flight so no
    // copy lands after the CTA exits.
    if (!alive && lane == 0) {
        for (int k = last_issued - slots + 1; k <= last_issued; ++k)
            if (k >= 0)
                mbar_drain_bounded(kIsK ? full_k(c, k % slots) : full_v(c, k % slots), ring_par(k, slots));
        if (kIsK) {
            for (int k = last_issued - kScaleRing + 1; k <= last_issued; ++k)
                if (k >= 0)
                    mbar_drain_bounded(scale_b(c, k % kScaleRing), ring_par(k, kScaleRing));
            if (q_issued >= 0)
                mbar_drain_bounded(qfull(c), (uint32_t)(q_issued & 1));
        }
    }
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

// ---------------------------------------------------------------------------
// V conversion
// ---------------------------------------------------------------------------
__device__ void convert_v(const Q8DecodeParams &q, const Ctx4 &c)
{
    const DecodeParams &p = q.d;
    const int t = threadIdx.x - kConvWarp0 * 32, lane = t & 31;
    const int P = p.page_size, log2P = 31 - __clz(P);
    bool alive = true;
    int kbase = 0;
    Segment s = locate(p, c.cta_begin, c.cta_end);
    for (;;) {
        const int nst = stages_of(s, P);
        const int lim = min(plan_len(p, s), s.p1 * P);
        const int all_see = keys_all_see(q, s);
        int e = kMinE;
        for (int j = 0; j < nst; ++j) {
            const int k = kbase + j, slot = k % c.vs;
            bool ok = false;
            if (alive)
                ok = mbar_wait_bounded(full_v(c, slot), ring_par(k, c.vs), c.abort_flag, p.err) &&
                     mbar_wait_bounded(scale_b(c, k % kScaleRing), ring_par(k, kScaleRing), c.abort_flag, p.err);
            alive = __all_sync(0xffffffffu, ok);
            if (alive) {
                const uint32_t mask = reinterpret_cast<volatile uint32_t *>(c.smem + c.lay.meta)[k % kScaleRing] & 0xffu;
                const int tok0 = s.p0 * P + j * kTT, n = lim - tok0;   // tokens of the stage that count
                e = next_e(e, stage_top_scale(c, k, min(n, all_see - tok0), mask, log2P));
                const int vb = (int)scale_at(c, k, t, log2P, 1);
                // a row that does not count, and a NaN row (its key's score is
                // made NaN instead, so that only rows that attend it see it), is zero
                const bool live = t < n && ((mask >> (t >> log2P)) & 1u) && vb != 255 && vb >= e - kVWindow;
                uint8_t *row = c.smem + c.lay.vring + (uint32_t)slot * kVSlotBytes + (uint32_t)t * 128u;
                uint4 raw[8];
#pragma unroll
                for (int ch = 0; ch < 8; ++ch)
                    raw[ch] = live ? *reinterpret_cast<const uint4 *>(row + kTT * 128 + ((ch ^ (t & 7)) << 4))
                                   : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) {
                    const uint32_t w[4] = {raw[ch].x, raw[ch].y, raw[ch].z, raw[ch].w};
                    uint32_t o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o[i] = widen_e4m3x2(w[i >> 1] >> (16 * (i & 1)));
                    uint8_t *dst = row + (ch >> 2) * (kTT * 128);
                    const int c0 = (2 * ch) & 7;
                    *reinterpret_cast<uint4 *>(dst + ((c0 ^ (t & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(dst + (((c0 + 1) ^ (t & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(conv_v(c, slot));
        }
        kbase += nst;
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
    const DecodeParams &p = q.d;
    constexpr uint32_t idesc = idesc_of(128, NR, false, false);
    const int steps = q.head_dim / 32;                   // 32 codes an MMA
    const uint64_t kd0 = umma_sdesc_sw128(k_slot(c, 0), 16u, 1024u);
    const uint64_t qh0 = umma_sdesc_sw128(c.base + c.lay.qtile, 16u, 1024u);
    const uint64_t ql0 = umma_sdesc_sw128(c.base + c.lay.qtile + c.lay.qhalf, 16u, 1024u);
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive)
            alive = mbar_wait_bounded(bar, parity, c.abort_flag, p.err);
    };
    int kbase = 0, seg = 0;
    Segment s = locate(p, c.cta_begin, c.cta_end);
    for (;;) {
        const int nst = stages_of(s, p.page_size);
        wait(q_ready(c), (uint32_t)(seg & 1));
        for (int j = 0; j < nst; ++j) {
            const int k = kbase + j, buf = k & 1, slot = k % c.ks;
            const uint64_t kd = kd0 + (((uint32_t)slot * kKSlotBytes) >> 4);
            wait(full_k(c, slot), ring_par(k, c.ks));
            wait(s_free(c, buf), (uint32_t)(((k >> 1) & 1) ^ 1));
            if (alive) {
                tc_fence_after();
                const uint32_t d = tmem + kColS + (uint32_t)(buf * 64);
                for (int i = 0; i < steps; ++i) {
                    umma_f8(d, kd + (uint64_t)(2 * i), qh0 + (uint64_t)(2 * i), idesc, i ? 1u : 0u);
                    umma_f8(d, kd + (uint64_t)(2 * i), ql0 + (uint64_t)(2 * i), idesc, 1u);
                }
            }
            umma_commit(s_full(c, buf));
            umma_commit(empty_k(c, slot));
            if (j == nst - 1)
                umma_commit(q_tile_free(c));
        }
        kbase += nst;
        ++seg;
        if (s.seg_end >= c.cta_end)
            break;
        s = next_segment(p, s, c.cta_end);
    }
    umma_commit(fin_b(c));
    mbar_drain_bounded(fin_b(c), 0u);
}

template <int NR>
__device__ void pv_issuer(const Q8DecodeParams &q, const Ctx4 &c, uint32_t tmem)
{
    const DecodeParams &p = q.d;
    constexpr uint32_t idesc = idesc_of(128, q_npv(NR), true, true);
    const uint64_t vd0 = umma_sdesc_sw128(v_slot(c, 0), (uint32_t)(kTT * 128), 1024u);
    const uint64_t pd0 = umma_sdesc_sw128(c.base + c.lay.pbuf, (uint32_t)(kTT * 128), 1024u);
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive)
            alive = mbar_wait_bounded(bar, parity, c.abort_flag, p.err);
    };
    int kbase = 0;
    Segment s = locate(p, c.cta_begin, c.cta_end);
    for (;;) {
        const int nst = stages_of(s, p.page_size);
        for (int j = 0; j < nst; ++j) {
            const int k = kbase + j, slot = k % c.vs;
            const uint64_t vd = vd0 + (((uint32_t)slot * kVSlotBytes) >> 4);
            wait(conv_v(c, slot), ring_par(k, c.vs));
            wait(p_full(c), (uint32_t)(k & 1));
            if (alive) {
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kTT / 16; ++ks)
                    umma_bf16(tmem + kColO, vd + (uint64_t)(ks * 128), pd0 + (uint64_t)(ks * 128), idesc,
                              (j == 0 && ks == 0) ? 0u : 1u);
            }
            umma_commit(pv_done(c));
            umma_commit(empty_v(c, slot));
        }
        kbase += nst;
        if (s.seg_end >= c.cta_end)
            break;
        s = next_segment(p, s, c.cta_end);
    }
    umma_commit(fin_b(c));
    mbar_drain_bounded(fin_b(c), 0u);
}

// ---------------------------------------------------------------------------
// softmax warps
// ---------------------------------------------------------------------------
template <int NR>
__device__ void softmax_q8(const Q8DecodeParams &q, const Ctx4 &c, uint32_t tmem)
{
    constexpr int NH = NR / 2;                 // rows per thread
    const DecodeParams &p = q.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tg = warp & (kTokenGroups - 1), hh = warp / kTokenGroups;
    const int t = tg * 32 + lane;
    const int P = p.page_size, log2P = 31 - __clz(P);
    const int D = q.head_dim;
    const uint32_t lane_base = (uint32_t)(tg * 32) << 16;
    const volatile uint32_t *meta = reinterpret_cast<const volatile uint32_t *>(c.smem + c.lay.meta);
    float *scr = reinterpret_cast<float *>(c.smem + c.lay.scr);
    int *scr_i = reinterpret_cast<int *>(scr);
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        bool ok = false;
        if (alive)
            ok = mbar_wait_bounded(bar, parity, c.abort_flag, p.err);
        alive = __all_sync(0xffffffffu, ok) && alive;
        return alive;
    };

    // Query rows of segment `sg`: bf16 staging buffer -> the two swizzled
    // e4m3 tiles and the rows' scales; D/8 lanes a row.  Rows past the unit's
    // are zero.
    auto stage_q = [&](int sg, const Segment &u) {
        wait(qfull(c), (uint32_t)(sg & 1));
        const int LR = D / 8, log2LR = 31 - __clz(LR);
        const int rows = q.n_q[u.b] * p.group;
        const int l = threadIdx.x & (LR - 1);
        for (int r = threadIdx.x >> log2LR; r < NR; r += kSoftmaxThreads >> log2LR) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (alive && r < rows)
                v = *reinterpret_cast<const uint4 *>(c.smem + c.lay.qbuf + r * D * 2 + l * 16);
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
                uint8_t *dst = c.smem + c.lay.qtile + (uint32_t)r * 128u + (((l >> 1) ^ (r & 7)) << 4) + (l & 1) * 8;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2 *>(dst + c.lay.qhalf) = make_uint2(lo[0], lo[1]);
                if (l == 0)
                    scr[kScrQ * 64 + r] = bad ? 1.f : q8_scale((uint32_t)byte);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(qempty(c));
            mbar_arrive(q_ready(c));
        }
    };

    int kbase = 0, seg = 0;
    Segment s = locate(p, c.cta_begin, c.cta_end);
    stage_q(0, s);
    for (;;) {
        const int nst = stages_of(s, P);
        const int R = q.n_q[s.b] * p.group;
        const int lim = min(plan_len(p, s), s.p1 * P);
        const int all_see = keys_all_see(q, s);
        int e = kMinE;                          // scale byte of E
        float2 nmu[NH / 2], l[NH / 2];          // 7 - m (1e30: no key yet), and this token's share of l
#pragma unroll
        for (int i = 0; i < NH / 2; ++i) {
            nmu[i] = make_float2(1e30f, 1e30f);
            l[i] = make_float2(0.f, 0.f);
        }
        named_barrier(1, kSoftmaxThreads);      // the rows' scales are in place

        for (int j = 0; j < nst; ++j) {
            const int k = kbase + j, buf = k & 1;
            // --- the token's scales, which come with K
            wait(scale_b(c, k % kScaleRing), ring_par(k, kScaleRing));
            const uint32_t tagged = alive ? meta[k % kScaleRing] : 0u;
            if (alive && (tagged >> 8) != ((uint32_t)k & 0xffffffu)) {
                if (lane == 0) {
                    atomicOr(p.err, SHKV_ERRF_PIPELINE);
                    *c.abort_flag = 1u;
                }
                alive = false;
            }
            const int tok0 = s.p0 * P + j * kTT;
            const int de = next_e(e, stage_top_scale(c, k, min(lim, all_see) - tok0, tagged & 0xffu, log2P)) - e;
            e += de;
            const bool valid = alive && (((tagged & 0xffu) >> (t >> log2P)) & 1u) && tok0 + t < lim;
            // the token's factor of the scores (NaN where its K or V row is),
            // its V exponent, and the factor that takes it out of l again
            const int vb = (int)scale_at(c, k, t, log2P, 1);
            const float ts = vb == 255 ? __uint_as_float(0x7fc00000u)
                                       : q8_scale(scale_at(c, k, t, log2P, 0)) * p.scale_log2;
            const int ve = !valid || vb == 255 ? e : max(vb, e - kVWindow);
            const float ev = (float)(ve - 127);
            const float undo = __uint_as_float((uint32_t)max(127 + e - ve, 1) << 23);
            // rows from this one on see the token (new token i from position L - n + i on)
            const int row_min = valid ? max(0, (tok0 + t - all_see + 1) * p.group) : 64;
            const bool masked = __any_sync(0xffffffffu, row_min > 0);
            // y - m + 7 of this thread's rows (nm = 7 - m), -inf where not seen
            float2 d[NH / 2];
            auto scores = [&](const float2 (&nm)[NH / 2]) {
                uint32_t sv[NH];
                tmem_ld_half<NH>(tmem + lane_base + kColS + (uint32_t)(buf * 64), hh, sv);
                const float2 ts2 = make_float2(ts, ts), ev2 = make_float2(ev, ev);
#pragma unroll
                for (int ch = 0; ch < NH / 8; ++ch) {
                    const float4 *rq = reinterpret_cast<const float4 *>(scr + kScrQ * 64 + 16 * ch + 8 * hh);
                    const float4 qa = rq[0], qb = rq[1];
                    const float2 q2[4] = {make_float2(qa.x, qa.y), make_float2(qa.z, qa.w), make_float2(qb.x, qb.y),
                                          make_float2(qb.z, qb.w)};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int o = 4 * ch + i;
                        const float2 s2 = make_float2(__uint_as_float(sv[2 * o]), __uint_as_float(sv[2 * o + 1]));
                        d[o] = __ffma2_rn(s2, __fmul2_rn(ts2, q2[i]), __fadd2_rn(ev2, nm[o]));
                        if (masked) {
                            if (half_row(hh, 2 * o) < row_min)
                                d[o].x = -INFINITY;
                            if (half_row(hh, 2 * o + 1) < row_min)
                                d[o].y = -INFINITY;
                        }
                    }
                }
            };
            if (wait(s_full(c, buf), (uint32_t)((k >> 1) & 1)))
                tc_fence_after();
            scores(nmu);
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < NH / 2; ++i)
                top = fmaxf(top, fmaxf(d[i].x, d[i].y));
            // --- lazy refresh of the maxima: all warps agree
            if (bar_red_or(1, kSoftmaxThreads, top > kPLog2 + kRescaleLog2 || de > 0)) {
                const float2 none[NH / 2] = {};
                scores(none);                   // y
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
                                scr[(kScrMax + tg) * 64 + half_row(hh, base + jj)] = v[jj];
                }
                named_barrier(1, kSoftmaxThreads);
                if (threadIdx.x < NR) {
                    const int r = threadIdx.x;
                    const float mo = scr[kScrM * 64 + r];
                    float mn = mo;
#pragma unroll
                    for (int g = 0; g < kTokenGroups; ++g)
                        mn = fmaxf(mn, scr[(kScrMax + g) * 64 + r]);
                    if (mo != -INFINITY) {
                        const float b = scr[kScrB * 64 + r] + (float)de;
                        mn = fmaxf(mn, mo + (b - kMaxTermLog2));
                        scr[kScrB * 64 + r] = fmaxf(b - (mn - mo), kTermLog2);
                    }
                    scr[kScrNew * 64 + r] = mn == -INFINITY ? 1e30f : kPLog2 - mn;
                    scr[kScrAlpha * 64 + r] = mn == -INFINITY ? 1.f : ex2_approx(mo - mn);
                    scr[kScrAlphaL * 64 + r] = mn == -INFINITY ? 1.f : ex2_approx(mo - mn + (float)de);
                    scr[kScrM * 64 + r] = mn;
                }
                named_barrier(1, kSoftmaxThreads);
                const float *alpha = scr + kScrAlpha * 64;
                if (j >= 1) {
                    // O^T holds stages up to k-1: rescale this thread's part once PV(k-1) is done
                    wait(pv_done(c), (uint32_t)((k - 1) & 1));
                    if (alive) {
                        tc_fence_after();
                        uint32_t ov[NH];
                        tmem_ld_half<NH>(tmem + lane_base + kColO, hh, ov);
#pragma unroll
                        for (int i = 0; i < NH; ++i)
                            ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha[half_row(hh, i)]);
                        tmem_st_half<NH>(tmem + lane_base + kColO, hh, ov);
                    }
                }
#pragma unroll
                for (int i = 0; i < NH / 2; ++i) {
                    const int r = half_row(hh, 2 * i);
                    nmu[i] = make_float2(scr[kScrNew * 64 + r], scr[kScrNew * 64 + r + 1]);
                    d[i] = __fadd2_rn(d[i], nmu[i]);
                    l[i] = __fmul2_rn(l[i], make_float2(scr[kScrAlphaL * 64 + r], scr[kScrAlphaL * 64 + r + 1]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(s_free(c, buf));
            uint32_t pk[NH / 2];
#pragma unroll
            for (int i = 0; i < NH / 2; ++i) {
                const float2 pe = make_float2(ex2_approx(d[i].x), ex2_approx(d[i].y));
                l[i] = __ffma2_rn(pe, make_float2(undo, undo), l[i]);
                pk[i] = pack_half2(pe.x, pe.y);
            }
            // --- P^T, once the previous stage's product has read the buffer
            if (k > 0)
                wait(pv_done(c), (uint32_t)((k - 1) & 1));
            if (alive) {
                uint8_t *prow = c.smem + c.lay.pbuf + (uint32_t)t * 128u;
#pragma unroll
                for (int ch = 0; ch < NH / 8; ++ch)
                    *reinterpret_cast<uint4 *>(prow + (((2 * ch + hh) ^ (t & 7)) << 4)) =
                        make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(p_full(c));
        }

        // --- next segment's query rows, as soon as the last QK of this one is done
        const bool has_next = s.seg_end < c.cta_end;
        Segment sn;
        if (has_next) {
            sn = next_segment(p, s, c.cta_end);
            wait(q_tile_free(c), (uint32_t)(seg & 1));
            named_barrier(1, kSoftmaxThreads);  // every warp is past its last use of the rows' scales
            stage_q(seg + 1, sn);
        }

        // --- segment end: row sums across the 128 tokens, log-sum-exp
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
                        scr[(kScrL + tg) * 64 + half_row(hh, base + jj)] = v[jj];
        }
        named_barrier(1, kSoftmaxThreads);
        const bool whole = (s.seg_begin == s.unit_begin) && (s.seg_end == s.unit_end);
        const int slot_id = whole ? 0 : 2 * (int)blockIdx.x + (s.seg_begin == c.cta_begin ? 0 : 1);
        const int64_t row0 = (int64_t)q.q0[s.b] * p.hq + (int64_t)s.g * p.group;
        const int *rowoff = scr_i + kScrOff * 64;
        if (threadIdx.x < NR) {
            const int r = threadIdx.x;
            float a = 0.f;
#pragma unroll
            for (int g = 0; g < kTokenGroups; ++g)
                a += scr[(kScrL + g) * 64 + r];
            scr[kScrInv * 64 + r] = a != 0.f ? __frcp_rn(a) : 0.f;    // (a NaN sum stays NaN)
            const float m = scr[kScrM * 64 + r];
            scr[kScrM * 64 + r] = -INFINITY;        // the next segment starts afresh
            scr[kScrB * 64 + r] = kTermLog2;
            if (alive && r < R) {
                const float lse = a != 0.f ? ((m == -INFINITY ? 0.f : m - kPLog2) - (float)(e - 127) + log2f(a)) * kLn2 : -INFINITY;
                if (whole) {
                    if (p.lse_out)
                        p.lse_out[row0 + rowoff[r]] = lse;
                } else {
                    p.ws_lse[(int64_t)slot_id * p.rows + r] = lse;
                }
            }
        }
        named_barrier(1, kSoftmaxThreads);

        // --- column d = t of O^T for this thread's rows, normalised
        wait(pv_done(c), (uint32_t)((kbase + nst - 1) & 1));
        if (alive) {
            tc_fence_after();
            const float ef = q8_scale((uint32_t)e);
            uint32_t ov[NH];
            tmem_ld_half<NH>(tmem + lane_base + kColO, hh, ov);
            if (t < D) {
#pragma unroll
                for (int i = 0; i < NH; ++i) {
                    const int r = half_row(hh, i);
                    if (r < R) {
                        const float o = __uint_as_float(ov[i]) * scr[kScrInv * 64 + r] * ef;
                        if (!whole)
                            p.ws_part[((int64_t)slot_id * p.rows + r) * D + t] = o;
                        else
                            p.out[(row0 + rowoff[r]) * D + t] = __float2bfloat16_rn(o);
                    }
                }
            }
        }
        tc_fence_before();
        named_barrier(1, kSoftmaxThreads);

        // --- split unit: the last piece to arrive merges all pieces
        if (!whole) {
            const int cb = cta_of(p, s.unit_begin);
            const int ce = cta_of(p, s.unit_end - 1);
            uint32_t *counter = p.ws_count + (int64_t)s.b * p.hkv + s.g;
            if (threadIdx.x == 0) {
                __threadfence();
                const uint32_t prev = atomicAdd(counter, 1u);
                *c.bcast = (prev == (uint32_t)(ce - cb)) ? 1u : 0u;
            }
            named_barrier(1, kSoftmaxThreads);
            if (*c.bcast) {
                __threadfence();
                const int dq = D / 4;
                for (int rr = warp; rr < R; rr += kSoftmaxWarps) {
                    float M = -INFINITY;
                    for (int cc = cb + lane; cc <= ce; cc += 32) {
                        const float x = __ldcg(p.ws_lse + (int64_t)piece_slot(p, cc, s.unit_begin) * p.rows + rr);
                        M = x != x ? x : fmaxf(M, x);
                    }
                    const bool nan = __any_sync(0xffffffffu, M != M);
#pragma unroll
                    for (int o_ = 16; o_ > 0; o_ >>= 1)
                        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o_));
                    float wsum = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (nan) {
                        wsum = acc.x = acc.y = acc.z = acc.w = __uint_as_float(0x7fc00000u);
                    } else if (M != -INFINITY) {
                        for (int cc = cb; cc <= ce; ++cc) {
                            const int sl = piece_slot(p, cc, s.unit_begin);
                            const float w = ex2_approx((__ldcg(p.ws_lse + (int64_t)sl * p.rows + rr) - M) *
                                                       1.4426950408889634f);
                            wsum += w;
                            if (lane < dq) {
                                const float4 v = __ldcg(
                                    reinterpret_cast<const float4 *>(p.ws_part + ((int64_t)sl * p.rows + rr) * D) + lane);
                                acc.x += w * v.x;
                                acc.y += w * v.y;
                                acc.z += w * v.z;
                                acc.w += w * v.w;
                            }
                        }
                    }
                    const float winv = wsum != 0.f ? 1.f / wsum : 0.f;
                    const int64_t orr = row0 + rowoff[rr];
                    if (lane < dq) {
                        uint2 packed;
                        packed.x = pack_bf16x2(acc.x * winv, acc.y * winv);
                        packed.y = pack_bf16x2(acc.z * winv, acc.w * winv);
                        *reinterpret_cast<uint2 *>(p.out + orr * D + lane * 4) = packed;
                    }
                    if (lane == 0 && p.lse_out)
                        p.lse_out[orr] = wsum != 0.f ? M + logf(wsum) : -INFINITY;
                }
                if (threadIdx.x == 0)
                    *counter = 0u;
            }
            named_barrier(1, kSoftmaxThreads);
        }

        kbase += nst;
        ++seg;
        if (!has_next)
            break;
        s = sn;
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
    c.ks = q.k_slots;
    c.vs = q.v_slots;
    c.lay = smem_layout(p.rows, q.head_dim, c.ks, c.vs);
    c.abort_flag = reinterpret_cast<volatile uint32_t *>(c.smem + c.lay.misc);
    c.bcast = reinterpret_cast<uint32_t *>(c.smem + c.lay.misc + 4);
    c.cta_begin = p.cta_cut[blockIdx.x];
    c.cta_end = p.cta_cut[blockIdx.x + 1];
    const bool work = c.cta_begin < c.cta_end;
    const int warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < c.ks; ++i) {
            mbar_init(full_k(c, i), 1);
            mbar_init(empty_k(c, i), 1);
        }
        for (int i = 0; i < c.vs; ++i) {
            mbar_init(full_v(c, i), 1);
            mbar_init(conv_v(c, i), kConvWarps);
            mbar_init(empty_v(c, i), 1);
        }
        for (int i = 0; i < kScaleRing; ++i)
            mbar_init(scale_b(c, i), 1);
        mbar_init(p_full(c), kSoftmaxWarps);
        mbar_init(pv_done(c), 1);
        mbar_init(qfull(c), 1);
        mbar_init(qempty(c), kSoftmaxWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(c, i), 1);
            mbar_init(s_free(c, i), kSoftmaxWarps);
        }
        mbar_init(q_ready(c), kSoftmaxWarps);
        mbar_init(q_tile_free(c), 1);
        mbar_init(fin_b(c), 2);                              // one commit per MMA issuer
        *c.abort_flag = 0u;
        *c.bcast = 0u;
        fence_barrier_init();
    }
    if (threadIdx.x < 64) {
        const int r = threadIdx.x;
        reinterpret_cast<float *>(c.smem + c.lay.scr)[kScrM * 64 + r] = -INFINITY;
        reinterpret_cast<float *>(c.smem + c.lay.scr)[kScrB * 64 + r] = kTermLog2;
        reinterpret_cast<int *>(c.smem + c.lay.scr)[kScrOff * 64 + r] = r / p.group * p.hq + r % p.group;
    }
    if (warp == 0)
        tmem_alloc(c.base + c.lay.tslot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(c.smem + c.lay.tslot);
    if (work && warp == kKWarp)
        warm_l2_q8(&tmK, p, c, c.ks);
    else if (work && warp == kVWarp)
        warm_l2_q8(&tmV, p, c, c.vs);
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
                producer_q8<true>(&tmK, q, c);
            else if (warp == kVWarp)
                producer_q8<false>(&tmV, q, c);
            else if (warp == kQkWarp) {
                if ((threadIdx.x & 31) == 0)
                    qk_issuer<NR>(q, c, tmem);
            } else if (warp == kPvWarp) {
                if ((threadIdx.x & 31) == 0)
                    pv_issuer<NR>(q, c, tmem);
            } else {
                convert_v(q, c);
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
cudaError_t launch_nr(const CUtensorMap &tmK, const CUtensorMap &tmV, Q8DecodeParams &q, cudaStream_t stream)
{
    static int regs = -1;      // the register split hands out exactly the launch's 128 a thread
    if (regs < 0) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, shkv_q8_decode_kernel<NR>);
        if (e != cudaSuccess)
            return e;
        regs = fa.numRegs;
    }
    if ((uint32_t)regs * kThreads != kSoftmaxRegs * 256 + kOtherRegs * 256)
        return cudaErrorInvalidConfiguration;
    q.k_slots = kMaxKSlots;
    q.v_slots = 4;
    while (smem_layout(q.d.rows, q.head_dim, q.k_slots, q.v_slots).total > (uint32_t)kSmemLimit)
        --q.v_slots;
    const uint32_t smem = smem_layout(q.d.rows, q.head_dim, q.k_slots, q.v_slots).total;
    const cudaError_t e =
        cudaFuncSetAttribute(shkv_q8_decode_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(shkv_q8_decode_kernel<NR>, q.d.num_ctas, kThreads, smem, stream, tmK, tmV, q);
}

}  // namespace

// tmK, tmV: 2-D maps of the code pools (box of 128 bytes x P rows, 128-byte swizzle).
cudaError_t launch_q8_decode(const CUtensorMap &tmK, const CUtensorMap &tmV, Q8DecodeParams &q, cudaStream_t stream)
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
