// A bounded mbarrier wait for pipelines whose stages turn over in about a microsecond.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace veda {

// As ptx::mbar_wait (false when `*abort` is raised or after `timeout_ns`, raising it then), but the clock is first
// read after a number of tries, each of which sleeps until the phase completes or its hint runs out: reading the global
// timer on every wait that does not pass at once costs more than the wait itself, and tries without a hint come back
// at once and take issue slots from the warps that work.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
        if (ptx::mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    return ptx::mbar_wait(bar, parity, abort, timeout_ns);
}

// the same for a converged warp, with one answer for all its lanes
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort, timeout_ns));
}

}  // namespace veda
