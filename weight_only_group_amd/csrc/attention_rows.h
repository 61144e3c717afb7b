// What the attention kernels over a paged cache have in common: the rows of a tile,
// the keys that they see, the score of a product.
//
// The rows of one key head are the (token, head of the group) pairs of a
// sequence, i * G + g; sixteen rows make a tile, and a wave takes 32 keys of a
// tile at a time (a chunk). Scores are kept times log2(e), so that the exponentials
// are powers of two.
#pragma once

#include "fixed_div.h"
#include "handoff.h"
#include "layer.h"
#include "mfma.h"

namespace qmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 16;   // rows per tile
constexpr int kChunk = 32;  // keys per wave and step
constexpr int kWaves = 4;

int row_tiles(int max_q, int group, int rows) { return (int)(((long long)max_q * group + rows - 1) / rows); }
// Blocks of a grid with `rtiles` row tiles for each of B * per units, which come in eights.
long long tile_blocks(int B, int per, int rtiles) { return ((long long)B * per + 7) / 8 * 8 * rtiles; }

struct AttnKernelArgs {
  AttentionArgs a;
  FixedDiv by_page, by_group;
  int group, rtiles, split;
  uint32_t* counters;
  float* part;  // (tiles, split, 16, D) sums, then (tiles, split, 16, 2) maximum and denominator
  float* part_ml;
};

// How a cap is taken. Up to kSmallCap: cap - 2 cap / (1 + e^2x), x = s / cap, whose
// error is a few roundings of the cap's size, 4 cap 2^-24 (2^-16 at 64: a sixteenth of
// the weights' own rounding in fp16). For larger caps, where that would reach the
// weights, a series for |x| < 1/4 and the quotient beyond, so that the error goes with
// the score. In blocks of 128 rows it takes longer, hence the two: a prompt of 8192, 32/8
// heads of 128, 700 us with a small cap, 945 us with a larger one.
enum Cap { kNoCap, kSmallCap, kAnyCap };
constexpr float kSmallCapMost = 64.f;

// The score, times log2(e), of a raw product.
struct ScoreRule {
  float scale;    // a product's factor: of the score, with a small cap of the exponent 2x log2(e)
  float inverse;  // any cap: of x
  float cap, slope;
  template <Cap CAP, bool SLOPES>
  __device__ __forceinline__ float score(float dot, int pos, int key) const {
    float s = dot * scale;
    if (CAP == kSmallCap) s = cap - 2 * cap * __builtin_amdgcn_rcpf(1 + __builtin_amdgcn_exp2f(s));  // cap at x = inf, -cap at -inf
    if (CAP == kAnyCap) {
      // tanh x = x (1 - x^2/3 + 2 x^4/15 - 17 x^6/315 + 62 x^8/2835 - ...), the next term below 2^-26 x at 1/4.
      const float x = dot * inverse, u = x * x;
      const float series = fmaf(u, fmaf(u, fmaf(u, fmaf(u, 62.f / 2835, -17.f / 315), 2.f / 15), -1.f / 3), 1.f);
      const float far = cap * fmaf(-2, __builtin_amdgcn_rcpf(1 + __builtin_amdgcn_exp2f(2 * kLog2e * x)), 1.f);
      s = fabsf(x) < 0.25f ? s * series : far;
    }
    return SLOPES ? s - slope * fabsf((float)(pos - key)) : s;
  }
};

inline __host__ __device__ Cap cap_kind(float softcap) {
  return !(softcap > 0) ? kNoCap : softcap <= kSmallCapMost ? kSmallCap : kAnyCap;
}

__device__ __forceinline__ ScoreRule score_rule(const AttentionArgs& a, int head) {
  ScoreRule r;
  // (kept finite where a tiny cap's inverse is not: 0 times it is 0)
  r.inverse = fminf(fmaxf(a.scale / a.softcap, -1e38f), 1e38f);
  r.scale = cap_kind(a.softcap) == kSmallCap ? 2 * kLog2e * r.inverse : kLog2e * a.scale;
  r.cap = kLog2e * a.softcap;
  r.slope = a.slopes ? kLog2e * a.slopes[head] : 0.f;
  return r;
}

// A sequence's query rows [q0, q1) and keys [0, kv) that take part, cut to the call's
// bounds, and its first query's position, which goes by all its queries and keys.
struct Span {
  int q0, q1, kv, first;
};
__device__ __forceinline__ Span span_of(const AttentionArgs& a, int b) {
  Span s;
  s.q0 = min(max(a.q_starts[b], 0), a.T);
  const int queries = min(max(a.q_starts[b + 1], s.q0), a.T) - s.q0, keys = max(a.kv_lens[b], 0);
  s.q1 = s.q0 + min(queries, a.max_q);
  s.kv = min(keys, a.max_kv);
  s.first = keys - queries;
  return s;
}

// Row tiles of a sequence.
__device__ __forceinline__ int row_tiles_of(const Span& s, int group) { return ((s.q1 - s.q0) * group + kRows - 1) / kRows; }

// Zeroes one key head's results of the tokens that no row stands for: those of sequence
// b past its bound, and those before the first sequence and behind the last. Shared out
// over `workers` blocks of 256 threads; as a rule there are none.
template <int D>
__device__ __forceinline__ void zero_rest(const AttnKernelArgs& p, const Span& s, int b, int hk, int worker, int workers) {
  const AttentionArgs& a = p.a;
  const int next = b + 1 < a.B ? min(max(a.q_starts[b + 1], 0), a.T) : a.T;
  if (next <= s.q1 && (b > 0 || s.q0 == 0)) return;
  const int pieces = p.group * D / 8;  // of 16 bytes, per token
  auto zero = [&](int from, int to) {
    for (long long i = worker * 256ll + threadIdx.x; i < (long long)(to - from) * pieces; i += workers * 256ll) {
      const long long t = from + i / pieces;
      *reinterpret_cast<u32x4*>(a.out + (t * a.Hq + hk * p.group) * D + i % pieces * 8) = u32x4{0, 0, 0, 0};
    }
  };
  zero(s.q1, next);
  if (b == 0) zero(0, s.q0);
}

// One row's token (-1: none), head and range of keys.
struct Row {
  int token, head, pos, lo, hi;
};
__device__ __forceinline__ Row row_of(const AttnKernelArgs& p, int r, const Span& s, int hk) {
  const AttentionArgs& a = p.a;
  Row w = {-1, 0, 0, 0, 0};
  const int i = p.by_group(r);
  if (i >= s.q1 - s.q0) return w;
  w.token = s.q0 + i;
  w.head = hk * p.group + r - i * p.group;
  w.pos = s.first + i;
  w.lo = a.first ? max(a.first[w.token], 0) : 0;
  w.hi = max(min(a.end ? a.end[w.token] : w.pos + 1, s.kv), 0);  // not below 0: hi - lo does not overflow
  return w;
}

// Whether the low half is an infinity or a NaN.
template <bool BF>
__device__ __forceinline__ bool not_finite(uint32_t v) {
  constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
  return (v & e) == e;
}

}  // namespace
}  // namespace qmm
