// Device-side helpers of the operators beside the stream mixing.
#pragma once

#include "hc_device.h"

namespace hc {

// 8 consecutive elements at any element-aligned address, as whole accesses: global
// memory needs no more alignment than that, and the compiler keeps the copy one access.
__device__ __forceinline__ void load8_any(const float* p, float v[8]) { __builtin_memcpy(v, p, 32); }

__device__ __forceinline__ void store8_any(float* p, const float v[8]) { __builtin_memcpy(p, v, 32); }

// A barrier that orders LDS alone: global loads that are on their way stay on their way.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace hc
