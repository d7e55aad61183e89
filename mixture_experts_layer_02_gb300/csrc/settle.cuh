// settle.cuh -- the end of bulk copies that no barrier is waited on for any more.
#pragma once

#include "device.cuh"

namespace moe {

// After a wait that ran out (kWaitLimitNs): copies that this thread started and whose
// barrier nobody waits for any more land long before this ends, or never.  Shared
// memory that they write is not used again or given back before.
__device__ __forceinline__ void settle_copies() {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kWaitLimitNs / 100) __nanosleep(1000);
}

}  // namespace moe
