// The append to the 4-bit cache, and tokens of it as 16-bit values.
//
// A pair (a, b) of a head turns into (a c - b s, b c + a s); keys in fp64, rounded to fp32, so
// that a code does not hang on the order of an fp32 sum. Of a group's values x: s =
// fp16(bf16((hi - lo) / 15)), m = fp16(lo + 8 s), code 8 + rint((x - m) / s). The 8 bits
// of s make s (c - 8) exact in fp16, which the attention builds on; m is the value of code 8,
// so that what the codes add is of the size of the values' spread.
#include "cache.h"
#include "fixed_div.h"

namespace qmm {
namespace {

constexpr float kLargest = kKv4Largest;

// Eight values' scale, middle and codes (nibble e: code of x[e]); the group is
// `lanes` neighbouring lanes, all of which come here.
struct Quantised {
  f16 s, m;
  uint32_t codes;
};
__device__ __forceinline__ Quantised quantise(float (&x)[8], int lanes) {
  float lo = INFINITY, hi = -INFINITY;
  int nan = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    nan |= x[e] != x[e];
    x[e] = fminf(fmaxf(x[e], -kLargest), kLargest);
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
  }
  for (int o = 1; o < lanes; o <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, o));
    hi = fmaxf(hi, __shfl_xor(hi, o));
    nan |= __shfl_xor(nan, o);
  }
  Quantised r;
  r.s = (f16)(float)(bf16)((hi - lo) / 15.f);
  const float s = (float)r.s;
  r.m = (f16)(lo + 8 * s);
  const float m = (float)r.m;
  // rint(d / s) without the division's own steps: `near` is within two units of the quotient's last place, so
  // that (s has 8 bits) d - near s is exact, and `quotient` is d / s to 2^-21 of a unit, rounded. Where d / s is no half-integer itself
  // it differs from one by d's unit over s, more than half a unit of its own by a part in 2^8 (s < 2 - 2^-7 times its
  // power of two): both are rounded to the same integer.
  const float inverse = __builtin_amdgcn_rcpf(s);
  r.codes = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float d = x[e] - m, near = d * inverse, quotient = fmaf(fmaf(-near, s, d), inverse, near);
    const float c = s > 0 ? fminf(fmaxf(rintf(quotient), -8.f), 7.f) : 0.f;
    r.codes |= (uint32_t)((int)c + 8) << (4 * e);
  }
  if (nan) {
    r.s = r.m = (f16)NAN;
    r.codes = 0x88888888u;
  }
  return r;
}

struct AppendKernelArgs {
  AppendArgs a;
  FixedDiv by_page;
  int groups;
  FixedDiv by_heads;
  int chunk_shift;               // log2 of a head's threads
  int group_lanes, group_shift;  // lanes per group; log2 of it
  unsigned xcds;
};

// Eight values of one head per thread. A thread of a rotated half loads its partner's
// eight values too: a group's values then lie in neighbouring lanes. 16381 tokens (24 heads of 64 over 4,
// 118 MB in all) take 26.7 us, 4.4 TB/s. The queries alone reach 5.1 TB/s; keys and values wait for the vector ALUs too
// (rotation in fp64, codes), with plain divisions 28.2 us, with indices in 64 bits 31.2 us. (Neighbouring tokens on different XCDs: 30.8
// us for 29.6. Threads of two and four heads, which load a token's angles and slot once: 31.0 and 34.8 us for 30.8, and 7
// tokens 5.4 and 7.8 us for 4.1.)
template <bool BF, bool ADJ>
__global__ void __launch_bounds__(256) kv4_append_kernel(AppendKernelArgs p) {
  const AppendArgs& a = p.a;
  const int chunks = 1 << p.chunk_shift;
  // Neighbouring tokens on one XCD (blocks go round them), whose L2 then holds a block of the cache whole.
  const unsigned block_i = blockIdx.x % p.xcds * (gridDim.x / p.xcds) + blockIdx.x / p.xcds;
  const int i = (int)(block_i * 256 + threadIdx.x);  // (below 2^31: three times T Hq D / 8 at most)
  const int c = i & (chunks - 1), th = i >> p.chunk_shift, token = p.by_heads(th), h = th - token * (a.Hq + 2 * a.Hkv);
  if (token >= a.T) return;
  const long long t = token;

  const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
  const uint16_t* src;
  uint8_t* block = nullptr;
  int at = 0;
  if (is_q) {
    src = a.q + t * a.q_stride + (long long)h * a.D;
  } else {
    const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= (long long)a.pages * a.page_size) return;
    const int page = p.by_page((int)slot);
    at = (int)slot - page * a.page_size;
    src = (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + (long long)hk * a.D;
    const long long row = ((long long)page * a.Hkv + hk) * a.page_size + at;
    block = reinterpret_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + row / kBlockTokens * kv4_block_bytes(a.D, p.groups);
    at %= kBlockTokens;
  }

  const u32x4 raw = *reinterpret_cast<const u32x4*>(src + 8 * c);
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = bits_to_float<BF>((uint16_t)(raw[e / 2] >> (16 * (e & 1))));
  if (!is_v && 8 * c < a.R) {
    const int pos = min(max(a.positions[t], 0), a.P - 1);
    const float* cs = a.cos + (long long)pos * (a.R / 2);
    const float* sn = a.sin + (long long)pos * (a.R / 2);
    float y[8], co[8], si[8];  // partners (the second of a pair: with its sign), cosines and sines
    if constexpr (ADJ) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = e & 1 ? x[e - 1] : -x[e + 1];
        co[e] = cs[4 * c + e / 2];
        si[e] = sn[4 * c + e / 2];
      }
    } else {
      const int half = a.R / 2;
      const bool second = 8 * c >= half;
      const u32x4 other = *reinterpret_cast<const u32x4*>(src + 8 * c + (second ? -half : half));
      const int from = 8 * c - (second ? half : 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = bits_to_float<BF>((uint16_t)(other[e / 2] >> (16 * (e & 1))));
        y[e] = second ? o : -o;
        co[e] = cs[from + e];
        si[e] = sn[from + e];
      }
    }
    if (is_q) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * co[e] + y[e] * si[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (float)((double)x[e] * (double)co[e] + (double)y[e] * (double)si[e]);
    }
  }
  if (is_q) {
    u32x4 out = raw;
    if (8 * c < a.R)
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = float_to_bits<BF>(x[2 * e]) | (uint32_t)float_to_bits<BF>(x[2 * e + 1]) << 16;
    *reinterpret_cast<u32x4*>(a.q_out + (t * a.Hq + h) * a.D + 8 * c) = out;
    return;
  }
  const Quantised z = quantise(x, p.group_lanes);
  const int g = c >> p.group_shift;
  const bool first = (c & (p.group_lanes - 1)) == 0;
  f16* rest = reinterpret_cast<f16*>(block + 4 * a.D);
  if (!is_v) {
    // Nibbles of a word: the even channels, then the odd ones.
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= (z.codes >> (4 * e) & 15) << (4 * (e / 2 + 4 * (e & 1)));
    reinterpret_cast<uint32_t*>(block)[at * chunks + (a.D / 32) * (c & 3) + c / 4] = w;
    if (first) {
      rest[at * 2 * p.groups + g] = z.s;
      rest[at * 2 * p.groups + p.groups + g] = z.m;
    }
  } else {
    uint16_t* codes = reinterpret_cast<uint16_t*>(block);
    codes[(2 * c) * kBlockTokens + at] = (uint16_t)z.codes;
    codes[(2 * c + 1) * kBlockTokens + at] = (uint16_t)(z.codes >> 16);
    if (first) {
      rest[g * 2 * kBlockTokens + at] = z.s;
      rest[(g * 2 + 1) * kBlockTokens + at] = z.m;
    }
  }
}

struct GatherKernelArgs {
  Kv4GatherArgs a;
  FixedDiv by_page;
  int chunk_shift, group_shift;  // log2 of a head's threads and of a group's
};

// Eight values of a token per thread, of HEADS heads: blockIdx.y tells which, of the keys, then the values. Bound by memory,
// the results' writes above all: 50021 tokens (8 heads of 128, 259 MB in all) take 50 us, 5.2 TB/s, as fast as a large
// copy, and 58 us pass after pass; with one head per thread 80 us, with the results kept in the L2s 66. Where one head per thread does not fill the
// CUs' waves it is faster (7 tokens 3.4 against 3.9 us).
template <bool BF, int HEADS>
__global__ void __launch_bounds__(256) kv4_gather_kernel(GatherKernelArgs p) {
  const Kv4GatherArgs& a = p.a;
  const int chunks = 1 << p.chunk_shift;
  const unsigned i = blockIdx.x * 256 + threadIdx.x;
  const int c = i & (chunks - 1);
  const long long t = i >> p.chunk_shift;
  if (t >= a.T) return;
  const int parts = (a.Hkv + HEADS - 1) / HEADS;
  const bool is_v = (int)blockIdx.y >= parts;
  const int h0 = ((int)blockIdx.y - (is_v ? parts : 0)) * HEADS, here = min(HEADS, a.Hkv - h0);
  uint16_t* dst = (is_v ? a.v : a.k) + (t * a.Hkv + h0) * a.D + 8 * c;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= (long long)a.pages * a.page_size) {
    for (int h = 0; h < here; ++h) *reinterpret_cast<u32x4*>(dst + h * a.D) = u32x4{0, 0, 0, 0};
    return;
  }
  const int page = p.by_page((int)slot);
  int at = (int)slot - page * a.page_size;
  const int groups = a.D / a.group_size, block_bytes = kv4_block_bytes(a.D, groups);
  const long long row = ((long long)page * a.Hkv + h0) * a.page_size + at;
  const uint8_t* block = (is_v ? a.v_cache : a.k_cache) + row / kBlockTokens * block_bytes;
  const size_t to_next = (size_t)a.page_size / kBlockTokens * block_bytes;  // the next head's
  at %= kBlockTokens;
  const int g = c >> p.group_shift;
  uint32_t w[HEADS];
  f16 s[HEADS], m[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    const uint8_t* from = block + (h < here ? h : 0) * to_next;
    const f16* rest = reinterpret_cast<const f16*>(from + 4 * a.D);
    if (!is_v) {
      w[h] = reinterpret_cast<const uint32_t*>(from)[at * chunks + (a.D / 32) * (c & 3) + c / 4];
      s[h] = rest[at * 2 * groups + g];
      m[h] = rest[at * 2 * groups + groups + g];
    } else {
      const uint16_t* codes = reinterpret_cast<const uint16_t*>(from);
      w[h] = codes[(2 * c) * kBlockTokens + at] | (uint32_t)codes[(2 * c + 1) * kBlockTokens + at] << 16;
      s[h] = rest[g * 2 * kBlockTokens + at];
      m[h] = rest[(g * 2 + 1) * kBlockTokens + at];
    }
  }
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    float sh = (float)s[h], mh = (float)m[h];
    if (!(fabsf(sh) <= kKv4LargestScale) || !(fabsf(mh) < INFINITY)) sh = mh = NAN;
    u32x4 out;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int lo = is_v ? 8 * x : 4 * x, hi = is_v ? 8 * x + 4 : 16 + 4 * x;
      const float u = mh + sh * (float)((int)(w[h] >> lo & 15) - 8), v = mh + sh * (float)((int)(w[h] >> hi & 15) - 8);
      out[x] = float_to_bits<BF>(u) | (uint32_t)float_to_bits<BF>(v) << 16;
    }
    if (h >= here) continue;
    u32x4* to = reinterpret_cast<u32x4*>(dst + h * a.D);
    // (more than fits in the L2s, which then keep the cache's lines for the threads that come back to them)
    if (HEADS > 1) __builtin_nontemporal_store(out, to);
    else *to = out;
  }
}

int log2_of(int n) { return __builtin_ctz((unsigned)n); }

template <bool BF, int HEADS>
void launch_gather_heads(const GatherKernelArgs& p, hipStream_t stream) {
  const long long n = (long long)p.a.T * (p.a.D / 8);
  kv4_gather_kernel<BF, HEADS><<<dim3((unsigned)((n + 255) / 256), 2 * ((p.a.Hkv + HEADS - 1) / HEADS)), 256, 0, stream>>>(p);
}

}  // namespace

hipError_t launch_kv4_append(const AppendArgs& a, int group_size, bool bf16, bool adjacent, hipStream_t stream) {
  const long long n = (long long)a.T * (a.Hq + 2 * a.Hkv) * (a.D / 8);
  const int xcds = device_topology().xcds;
  const dim3 grid((unsigned)((n + 256 * xcds - 1) / (256 * xcds) * xcds));
  const AppendKernelArgs p = {a, fixed_div(a.page_size), a.D / group_size, fixed_div(a.Hq + 2 * a.Hkv), log2_of(a.D / 8), group_size / 8, log2_of(group_size / 8), (unsigned)xcds};
  if (bf16 && adjacent) kv4_append_kernel<true, true><<<grid, 256, 0, stream>>>(p);
  else if (bf16) kv4_append_kernel<true, false><<<grid, 256, 0, stream>>>(p);
  else if (adjacent) kv4_append_kernel<false, true><<<grid, 256, 0, stream>>>(p);
  else kv4_append_kernel<false, false><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_kv4_gather(const Kv4GatherArgs& a, bool bf16, hipStream_t stream) {
  const GatherKernelArgs p = {a, fixed_div(a.page_size), log2_of(a.D / 8), log2_of(a.group_size / 8)};
  const bool many = (long long)a.T * 2 * a.Hkv * (a.D / 8) > 32ll * 64 * device_topology().cus;
  if (many) bf16 ? launch_gather_heads<true, 2>(p, stream) : launch_gather_heads<false, 2>(p, stream);
  else bf16 ? launch_gather_heads<true, 1>(p, stream) : launch_gather_heads<false, 1>(p, stream);
  return hipGetLastError();
}

}  // namespace qmm
