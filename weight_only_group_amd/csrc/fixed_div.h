// Division by a divisor that the host knows.
#pragma once

#include "common.h"

namespace qmm {
namespace {

// Division of 0 <= n < 2^31 by a fixed divisor: n mul >> shift, with mul = ceil(2^shift / d)
// and shift = 31 + ceil(log2 d) (the excess of mul stays below one part in n).
struct FixedDiv {
  uint32_t mul;
  int shift;
  __device__ __forceinline__ int operator()(int n) const { return (int)((uint64_t)(uint32_t)n * mul >> shift); }
};
inline FixedDiv fixed_div(int d) {
  int l = 0;
  while ((1ll << l) < d) ++l;
  return {(uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), 31 + l};
}

}  // namespace
}  // namespace qmm
