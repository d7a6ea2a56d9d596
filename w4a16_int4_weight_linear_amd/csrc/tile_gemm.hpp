// tile_gemm.hpp -- what the tiled kernels share: the LDS barrier, and the tile order and work
// split of split_plan.hpp.
#pragma once

#include <type_traits>

#include "device.hpp"
#include "kernels.hpp"
#include "split_plan.hpp"

namespace w4a16 {

#define W4A16_LDS(p) ((__attribute__((address_space(3))) void*)(p))

// Barrier that publishes LDS: this thread's LDS reads and global-to-LDS
// loads are complete before it, and no LDS access moves across it.
__device__ inline void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace w4a16
