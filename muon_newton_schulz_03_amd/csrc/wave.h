// Lanes of one wave that exchange data through LDS without a barrier.
#pragma once

#include <hip/hip_runtime.h>

namespace muon {

// Orders a wave's LDS accesses, which its lanes make in turn.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace muon
