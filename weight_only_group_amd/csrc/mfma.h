// Matrix-core and 16-bit pair helpers of the layer operators' kernels.
#pragma once

#include "common.h"

namespace qmm {
namespace {

// N 32-bit words as one vector.
template <int N> struct Words;
template <> struct Words<2> { typedef u32x2 T; };
template <> struct Words<4> { typedef u32x4 T; };

// V_MFMA_F32_16X16X32: lane l holds row (column, for b) l & 15 and the eight k
// from 8 (l >> 4) on; of the result column l & 15 and rows 4 (l >> 4) + r.
template <bool BF>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// V_MFMA_F32_32X32X16: lane l holds row (column, for b) l & 31 and the eight k from
// 8 (l >> 5) on; of the result column l & 31 and, as register i, row 8 (i / 4) +
// 4 (l >> 5) + i % 4.
template <bool BF>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// c + the pair's two values.
template <bool BF>
__device__ __forceinline__ float add_pair(uint32_t pair, float c) {
  if constexpr (BF) return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, 0x3F803F80u), c, false);
  else return __builtin_amdgcn_fdot2(as_f16x2(pair), as_f16x2(0x3C003C00u), c, false);
}

// Two floats as a pair (the first in the low half), each rounded to nearest even.
template <bool BF>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  if constexpr (BF) return pack_bf16(lo, hi);
  else return as_u32(f16x2{(f16)lo, (f16)hi});
}

}  // namespace
}  // namespace qmm
