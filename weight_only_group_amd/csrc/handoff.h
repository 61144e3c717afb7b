// Handing partial results to the block that arrives last, across the XCDs' L2s.
//
// An agent-scope release fence writes back the XCD's whole L2, and a launch's
// fences queue up behind each other: at 768 blocks they took 200 of 250 us. So no
// fence is used: what is handed over is written and read by agent-scope atomics,
// which go past the L2s one by one; a block counts itself in once all its waves'
// writes have been acknowledged (the wait and the barrier below).
#pragma once

#include "common.h"

namespace qmm {
namespace {

__device__ __forceinline__ void handoff_store(float* p, float a, float b) {  // p 8-byte aligned
  const uint64_t v = (uint64_t)__builtin_bit_cast(uint32_t, b) << 32 | __builtin_bit_cast(uint32_t, a);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void handoff_store(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void handoff_store(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t handoff_load(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float handoff_load(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
struct FloatPair {
  float a, b;
};
__device__ __forceinline__ FloatPair handoff_load_pair(const float* p) {  // p 8-byte aligned
  const uint64_t v = handoff_load(reinterpret_cast<const uint64_t*>(p));
  const uint32_t lo = (uint32_t)v, hi = (uint32_t)(v >> 32);
  return {__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}

// Whether this block is the last of n to come here; every thread calls it, after
// its handoff_stores. The counter is left at zero.
__device__ __forceinline__ bool handoff_last(uint32_t* counter, uint32_t n, int* shared_flag) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t ticket = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *shared_flag = ticket == n - 1;
    if (ticket == n - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *shared_flag != 0;
}

}  // namespace
}  // namespace qmm
