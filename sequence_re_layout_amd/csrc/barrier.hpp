// barrier.hpp -- a work-group barrier that waits for LDS alone: a full one also
// waits until every store has arrived in memory.
#pragma once

#include <hip/hip_runtime.h>

namespace basp {

__device__ inline void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace basp
