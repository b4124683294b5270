// Warp-wide reductions.
#pragma once

#include <cuda_runtime.h>

namespace veda {

// the largest value of a converged warp, NaN passed over (one instruction of this architecture)
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

}  // namespace veda
