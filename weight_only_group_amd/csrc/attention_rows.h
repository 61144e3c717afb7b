// What the attention kernels over a paged cache have in common: the rows of a tile,
// the keys that they see, the score of a product, the join of partial results.
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
constexpr int kMaxSplit = 64;

struct AttnPlan {
  int group;    // query heads per key head
  int rtiles;   // row tiles of the longest sequence, per key head
  int split;    // blocks along the keys
  size_t tiles;  // all row tiles
};

int row_tiles(int max_q, int group, int rows) { return (int)(((long long)max_q * group + rows - 1) / rows); }
// Blocks of a grid with `rtiles` row tiles for each of B * per units, which come in eights.
long long tile_blocks(int B, int per, int rtiles) { return ((long long)B * per + 7) / 8 * 8 * rtiles; }

AttnPlan attn_plan(int B, int Hq, int Hkv, int max_q, int max_kv, DeviceTopo topo) {
  AttnPlan p;
  p.group = Hq / Hkv;
  p.rtiles = row_tiles(max_q, p.group, kRows);
  p.tiles = (size_t)B * Hkv * p.rtiles;
  const long long want = 4ll * topo.cus / (long long)p.tiles;
  const long long most = (max_kv + kWaves * kChunk - 1ll) / (kWaves * kChunk);
  p.split = (int)(want < most ? want : most);
  if (p.split > kMaxSplit) p.split = kMaxSplit;
  if (p.split < 1 || p.tiles > (size_t)kGemvMaxStrips) p.split = 1;
  return p;
}

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

// The end of a block of 16 rows: its waves' sums (in LDS, with their maxima and
// denominators) in wave order, then the parts along the keys, joined in order by the
// block that arrives last, which writes the results. `pack` rounds two of them.
template <int D, typename PACK>
__device__ __forceinline__ void join_rows(const AttnKernelArgs& p, const float (*so)[kRows][D + 4], const float (*sml)[kRows][2],
                                          int* s_last, const Span& span, int b, int hk, int rt, int part, PACK pack) {
  // Thread: row tid / 16, D / 16 neighbouring dimensions.
  constexpr int E = D / 16;
  const int tid = threadIdx.x, r = tid >> 4, d0 = (tid & 15) * E;
  float m = -INFINITY, l = 0, o[E] = {};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sml[w][r][0]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const float f = sml[w][r][0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(sml[w][r][0] - m);
    l += sml[w][r][1] * f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += so[w][r][d0 + e] * f;
  }
  const AttentionArgs& a = p.a;
  const Row mine = row_of(p, rt * kRows + r, span, hk);
  if (p.split > 1) {
    // Partial sums of the parts, joined in order by the block that arrives last.
    const size_t tile = ((size_t)b * a.Hkv + hk) * p.rtiles + rt;
    // A thread's pairs lie 256 pairs apart: the threads of a store write whole lines. Rows past the
    // sequence's last (12 of 16 with four heads a group and one query) are left out.
    float* po = p.part + (tile * p.split + part) * kRows * D + 2 * tid;
    if (mine.token >= 0) {
#pragma unroll
      for (int e = 0; e < E; e += 2) handoff_store(po + e * 256, o[e], o[e + 1]);
      if ((tid & 15) == 0) handoff_store(p.part_ml + ((tile * p.split + part) * kRows + r) * 2, m, l);
    }
    if (!handoff_last(&p.counters[tile], (uint32_t)p.split, s_last) || mine.token < 0) return;
    const float* qo = p.part + tile * p.split * kRows * D + 2 * tid;
    const float* qm = p.part_ml + (tile * p.split * kRows + r) * 2;
    // Four parts' loads at a time; places past the last part repeat it with a factor of 0.
    constexpr int kBatch = 4;
    m = -INFINITY;
    for (int s0 = 0; s0 < p.split; s0 += kBatch) {
      float ms[kBatch];
#pragma unroll
      for (int s = 0; s < kBatch; ++s) ms[s] = handoff_load(qm + min(s0 + s, p.split - 1) * kRows * 2);
#pragma unroll
      for (int s = 0; s < kBatch; ++s) m = fmaxf(m, ms[s]);
    }
    l = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0;
    for (int s0 = 0; s0 < p.split; s0 += kBatch) {
      float ms[kBatch], ls[kBatch];
      FloatPair os[kBatch][E / 2];
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        const int at = min(s0 + s, p.split - 1);
        const FloatPair ml = handoff_load_pair(qm + at * kRows * 2);
        ms[s] = ml.a;
        ls[s] = ml.b;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) os[s][e] = handoff_load_pair(qo + (size_t)at * kRows * D + 512 * e);
      }
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        const float f = s0 + s >= p.split || ms[s] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ms[s] - m);
        l += ls[s] * f;
        // (a sum that is not finite goes with a finite maximum or a weight that is not: f is not 0 then)
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += f == 0.f ? 0.f : (e & 1 ? os[s][e / 2].b : os[s][e / 2].a) * f;
      }
    }
  }
  if (mine.token < 0) return;
  const float inv = mine.lo < mine.hi ? 1 / l : 0.f;
  uint16_t* dst = a.out + ((long long)mine.token * a.Hq + mine.head) * D + d0;
#pragma unroll
  for (int e = 0; e < E; e += 4)
    *reinterpret_cast<u32x2*>(dst + e) = u32x2{pack(o[e] * inv, o[e + 1] * inv), pack(o[e + 2] * inv, o[e + 3] * inv)};
}

}  // namespace
}  // namespace qmm
