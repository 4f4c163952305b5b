// q8_wait.cuh -- bounded mbarrier waits of the 8-bit cache's kernels
// (internal to the library).  They are kept to a few instructions: the roles
// of these kernels share an SM sub-partition's instruction cache, and waits
// are at every step of their loops.
#pragma once

#include <stdint.h>

#include "shkv_device.cuh"

namespace shkv {

// SM cycles that a wait may take: 2 s at 2 GHz.
constexpr long long kQ8WaitCycles = 4000000000ll;

// Waits for the phase with the given parity; kSleep suspends the thread on the
// barrier between tries (issuers, producers: it leaves the issue slots to the
// others).  False if the CTA's abort flag is raised or the wait runs over
// kQ8WaitCycles (then the flag is raised and SHKV_ERRF_TIMEOUT recorded).
template <bool kSleep>
__device__ __forceinline__ bool q8_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag, uint32_t *err)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const long long t0 = clock64();
#pragma unroll 1
    for (;;) {
        uint32_t ok;
        if (kSleep)
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(bar), "r"(parity), "r"(20000u)
                : "memory");
        else
            ok = mbar_try_wait(bar, parity);
        if (ok)
            return true;
        if (*abort_flag)
            return false;
        if (clock64() - t0 > kQ8WaitCycles)
            break;
    }
    *abort_flag = 1u;
    atomicOr(err, SHKV_ERRF_TIMEOUT);
    return false;
}

}  // namespace shkv
