// arrive.hpp -- joining parts of a result by the workgroup that finishes last.
#pragma once

#include "device.hpp"

namespace w4a16 {

// A workgroup's part of a result is stored (device scope) and complete for this wave; counts
// the workgroup's arrival at `counter`.  Returns true in all threads of the workgroup that
// arrives last of `parts`, which then sees every part (through device-scope loads) and has
// put the counter back to 0.  No workgroup waits for another.  All threads must call it;
// `flag` is a word of LDS that nothing else uses meanwhile.
__device__ inline bool arrive_last(uint32_t* counter, uint32_t parts, uint32_t* flag) {
  __builtin_amdgcn_s_waitcnt(0);                 // this wave's stores have reached the device's memory
  __syncthreads();                               // ... and every other wave's
  if (threadIdx.x == 0) {
    const uint32_t before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before == parts - 1u) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *flag = before == parts - 1u;
  }
  __syncthreads();
  const bool last = *flag != 0u;
  __syncthreads();                               // (the word may be written again after this)
  return last;
}

}  // namespace w4a16
