// A bounded mbarrier wait for pipelines whose stages turn over in about a microsecond.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace veda {

// As ptx::mbar_wait (false when `*abort` is raised or after `timeout_ns`, raising it then), but the clock is first
// read after a number of try_waits, each of which the hardware suspends for a while: reading the global timer on
// every wait that does not pass at once costs more than the wait itself.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (ptx::mbar_try_wait(bar, parity)) return true;
    return ptx::mbar_wait(bar, parity, abort, timeout_ns);
}

// the same for a converged warp, with one answer for all its lanes
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t timeout_ns) {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort, timeout_ns));
}

}  // namespace veda
