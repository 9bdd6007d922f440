// Values that one workgroup stores and another reads within a launch (gfx950: every XCD has
// an L2 of its own).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8k {

// What other CUs read in the same launch goes past the caches that are not shared, and is
// counted once it is there (vmcnt 0 in every wave, then a barrier): no cache is written
// back or invalidated.  (With release and acquire fences instead, which write back and
// invalidate an XCD's whole L2, a call measured 10 us longer.)
__device__ __forceinline__ void store_shared(float* p, float v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t load_shared(const uint32_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_shared(const float* p) {  // 8-byte aligned
    const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__builtin_bit_cast(float, (uint32_t)v), __builtin_bit_cast(float, (uint32_t)(v >> 32)));
}

}  // namespace q8k
