// The waits of prompt_attention's bf16 kernel.
#pragma once

#include <stdint.h>

#include "rx_device.cuh"

namespace rx {

// Whether an mbarrier phase has completed, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// A whole warp's bounded wait (2 s, unless the self-test gives less) on an mbarrier phase; on
// time-out it sets *abort, which ends every role's waits and is reported once, at the end.  As short
// as can be: there are some thirty waits in the kernel, and an item of a short sequence runs every
// role's code once, so that fetching instructions is much of its time.
__device__ __forceinline__ bool pt_wait_on(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t limit_ns = 2000000000u) {
    auto now = [] {
        uint32_t t;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
        return t;
    };
    const uint32_t t0 = now();
    bool ok;
    do ok = mbar_try_wait(bar, parity);
    while (!ok && !*abort && now() - t0 < limit_ns);
    if (!ok) *abort = 1;
    return ok;
}

__device__ __forceinline__ bool pt_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t limit_ns = 2000000000u) {
    bool ok = mbar_try_wait(bar, parity);     // up to 100 us by itself
    if (!ok) ok = pt_wait_on(bar, parity, abort, limit_ns);
    return __all_sync(0xffffffffu, ok);
}

}  // namespace rx
