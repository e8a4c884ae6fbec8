// Ordering within one wave.
#pragma once

#include <hip/hip_runtime.h>

namespace prism {

// Orders this wave's LDS accesses, which the hardware keeps in order: what its
// lanes wrote before is read after.
__device__ inline void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace prism
