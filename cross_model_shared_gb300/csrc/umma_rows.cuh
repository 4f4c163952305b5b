// umma_rows.cuh -- how the tcgen05 decode kernels share the stacked rows of a
// TMEM lane between two warps, and the reductions over a stage's tokens.
#pragma once

#include <stdint.h>

#include "shkv_device.cuh"

namespace shkv {

namespace {

// A softmax thread's rows: 8-row chunks alternate between the two row
// halves, so element i of half hh is stacked row 16*(i/8) + 8*hh + i%8, and
// every TMEM access is 8 columns at a multiple of 8.
__device__ __forceinline__ int half_row(int hh, int i) { return ((i >> 3) << 4) + (hh << 3) + (i & 7); }

// This thread's N columns (N a multiple of 8) of a TMEM region starting at
// column `taddr`, as N/8 chunks of 8 at a stride of 16 from `taddr + 8*hh`.
template <int N>
__device__ __forceinline__ void tmem_ld_half(uint32_t taddr, int hh, uint32_t (&r)[N])
{
#pragma unroll
    for (int c = 0; c < N / 8; ++c)
        tmem_ld8_nowait(taddr + (uint32_t)(16 * c + 8 * hh), r + 8 * c);
    tmem_wait_ld();
}

template <int N>
__device__ __forceinline__ void tmem_st_half(uint32_t taddr, int hh, const uint32_t (&r)[N])
{
#pragma unroll
    for (int c = 0; c < N / 8; ++c)
        tmem_st8_nowait(taddr + (uint32_t)(16 * c + 8 * hh), r + 8 * c);
    tmem_wait_st();
}

// Warp reduce-scatter by recursive halving: at the butterfly step with lane
// offset O a lane keeps half of its M values and combines it with the
// partner's copy of that half.  Afterwards lane l holds in v[0 .. M/32 - 1]
// (v[0] if M < 32) the warp totals of columns rs_base<M>(l) + j; for M < 32,
// lanes that differ only in their low log2(32/M) bits hold the same column.
// M/2 + M/4 + ... shuffles instead of 5*M for a butterfly per column.
template <int M, int O, bool kMax>
struct ReduceScatter {
    static __device__ __forceinline__ void run(float *v, int lane)
    {
        if constexpr (O > 0) {
            if constexpr (M > 1) {
                const bool up = (lane & O) != 0;
#pragma unroll
                for (int i = 0; i < M / 2; ++i) {
                    const float send = up ? v[i] : v[i + M / 2];
                    const float keep = up ? v[i + M / 2] : v[i];
                    const float recv = __shfl_xor_sync(0xffffffffu, send, O);
                    v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
                }
                ReduceScatter<M / 2, O / 2, kMax>::run(v, lane);
            } else {
                const float recv = __shfl_xor_sync(0xffffffffu, v[0], O);
                v[0] = kMax ? fmaxf(v[0], recv) : v[0] + recv;
                ReduceScatter<1, O / 2, kMax>::run(v, lane);
            }
        }
    }
};

template <int M>
__device__ __forceinline__ int rs_base(int lane)
{
    int base = 0, m = M;
    for (int o = 16; o >= 1 && m > 1; o >>= 1) {
        if (lane & o)
            base += m / 2;
        m /= 2;
    }
    return base;
}

// lanes that hold a distinct column after a reduce-scatter of M values
template <int M>
__device__ __forceinline__ bool rs_owner(int lane)
{
    return M >= 32 || (lane & (32 / M - 1)) == 0;
}

__host__ __device__ constexpr int pow2_at_least(int n) { return n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64; }

}  // namespace

}  // namespace shkv
