// What the attention kernels over the 4-bit cache have in common.
//
// The formulas of the attention to a cache of 16-bit values, with k_j = m + s (c - 8) per
// group of channels, taken apart so that what the matrix cores see is exact in fp16:
//   q.k_j = sum_d q_d [s_j (c_jd - 8)] + sum_g m_jg Q_g,     Q_g = sum of the group's q_d
//   sum_j p_j v_j = sum_j p_j [s_j (c_jd - 8)] + sum_j p_j m_jg
// s has 8 significant bits and c - 8 three and a sign, so the brackets are fp16 numbers.
// A code becomes one by an AND, an OR and half a packed multiply-add: the half 16 + c
// has it in the top of its mantissa, and s (16 + c) - 24 s is rounded once, so not at all.
// The second sums are one matrix operation more for all channels together, with
// the middles as further channels; Q, an fp32 sum, goes in fp16 parts: three (all of it) where a block has few rows, two (to 2^-22
// of it) in blocks of many, whose lane groups are two. A row of ones among the value's middles gives the weights' sum.
//
// Queries are scaled by a power of two, so that a row's largest is in [1, 2): the matrix operations take fp16 operands, which
// hold codes times scales exactly (bf16 would not). Values below 2^-14 of it (bf16: 2^-17), subnormal then, are rounded to steps of
// 2^-24: a score is off by 2^-25 of the largest times the key's values there at most, about what one rounding of the largest
// one's product costs in fp32. The weights p are fp16, times 2^7.
// (Of a product with a subnormal half, a scale, middle or weight below 2^-14, the matrix cores keep fewer bits: a sum of
// 4096 of them at 2^-24 came out 4.6e-5 too small, less than the weights' rounding, 2^-12, may move it.)
#pragma once

#include "attention_rows.h"
#include "cache.h"

namespace qmm {
namespace {

// A row's maximum is left where it is while no weight passes 2^kSlack of it; weights are
// kept times 2^kLift, so that they pass neither end of fp16.
constexpr float kLift = 7.f, kSlack = 8.f;

// The AND's and the OR's constant, in registers: as literals they would take an instruction each.
struct DecodeMasks {
  uint32_t code, sixteen;
  __device__ __forceinline__ DecodeMasks() {
    asm("s_mov_b32 %0, 0x03C003C0" : "=s"(code));
    asm("v_mov_b32 %0, 0x4C004C00" : "=v"(sixteen));
  }
};

// Two of a word's codes, nibbles R and R + 4, as s (c - 8); c24 = -24 s.
template <int R>
__device__ __forceinline__ uint32_t decode(uint32_t w, f16x2 s, f16x2 c24, const DecodeMasks& k) {
  const uint32_t at = R == 0 ? w << 6 : R == 1 ? w << 2 : R == 2 ? w >> 2 : w >> 6;
  return as_u32(__builtin_elementwise_fma(as_f16x2((at & k.code) | k.sixteen), s, c24));
}
// Exact (10 bits) up to kKv4LargestScale, and beyond it infinite, as every code of the group then is.
__device__ __forceinline__ f16x2 times_24(f16x2 s) { return s * f16x2{(f16)-24.f, (f16)-24.f}; }

// Two groups' middles, NaN where the group stands for NaN (the middle is not finite or the scale s too large): an infinity
// alone would give infinite sums, and a weight of 0 to the key whose score is minus infinity.
__device__ __forceinline__ uint32_t middles_or_nan(uint32_t m, uint32_t s) {
  const f16x2 v = as_f16x2(m), none = times_24(as_f16x2(s)) * f16x2{(f16)0.f, (f16)0.f};  // 0 or NaN
  return as_u32(__builtin_elementwise_fma(v, none, v));
}

// Whether the low half is no middle, no scale of a group that stands for numbers.
__device__ __forceinline__ bool bad_middle(uint32_t m) { return not_finite<false>(m); }
__device__ __forceinline__ bool bad_scale(uint32_t s) {
  constexpr uint32_t most = __builtin_bit_cast(uint16_t, (f16)kKv4LargestScale);
  return (s & 0x7FFFu) > most;
}
// The same of both halves of a pair, as a mask of the bad ones.
__device__ __forceinline__ uint32_t bad_middles(uint32_t m) {
  return (bad_middle(m) ? 0xFFFFu : 0u) | (bad_middle(m >> 16) ? 0xFFFF0000u : 0u);
}
__device__ __forceinline__ uint32_t bad_scales(uint32_t s) {
  return (bad_scale(s) ? 0xFFFFu : 0u) | (bad_scale(s >> 16) ? 0xFFFF0000u : 0u);
}

// BYTES (a multiple of 4, up to 32) from p as 32-bit words.
template <int BYTES>
__device__ __forceinline__ void load_words(uint32_t* to, const uint8_t* p) {
  if constexpr (BYTES % 16 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(p + 16 * i);
#pragma unroll
      for (int x = 0; x < 4; ++x) to[4 * i + x] = v[x];
    }
  } else if constexpr (BYTES == 8) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    to[0] = v[0];
    to[1] = v[1];
  } else {
    to[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

constexpr uint32_t kOnes = 0x3C003C00u;  // two halves of 1

// A row's query (N * 8 values in each of LANES lanes, 64 / LANES apart) as fp16, scaled by a
// power of two; returns what undoes that. All NaN where a value is not finite.
template <int LANES, int N>
__device__ __forceinline__ float scale_query(u32x4 (&q)[N], bool bf16_data) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 pairs = {0, 0};  // of the values' bits without a sign, in the order of their sizes
#pragma unroll
  for (int s = 0; s < N; ++s)
#pragma unroll
    for (int x = 0; x < 4; ++x) pairs = __builtin_elementwise_max(pairs, __builtin_bit_cast(u16x2, q[s][x] & 0x7FFF7FFFu));
  int most = max(pairs[0], pairs[1]);
  if (LANES == 4) most = max(most, __shfl_xor(most, 16));
  most = max(most, __shfl_xor(most, 32));
  if (bf16_data) {
    const int up = min(max(254 - (most >> 7), 1), 253);  // the factor's exponent
    const float factor = most < 0x7F80 ? __builtin_bit_cast(float, (uint32_t)up << 23) : NAN;
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        q[s][x] = pack_pair<false>(__builtin_bit_cast(float, q[s][x] << 16) * factor, __builtin_bit_cast(float, q[s][x] & 0xFFFF0000u) * factor);
    return __builtin_bit_cast(float, (uint32_t)(254 - up) << 23);
  }
  const int up = min(max(30 - (most >> 10), 1), 30);  // (within fp16's: tiny queries stay below 1)
  const f16 factor = most < 0x7C00 ? __builtin_bit_cast(f16, (uint16_t)(up << 10)) : (f16)NAN;
#pragma unroll
  for (int s = 0; s < N; ++s)
#pragma unroll
    for (int x = 0; x < 4; ++x) q[s][x] = as_u32(as_f16x2(q[s][x]) * f16x2{factor, factor});
  return __builtin_bit_cast(float, (uint32_t)(127 + 15 - up) << 23);
}

}  // namespace
}  // namespace qmm
