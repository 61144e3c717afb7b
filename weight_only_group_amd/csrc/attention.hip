// Attention of new tokens to the paged cache of their sequences.
//
// For a query row n and keys j: s_j = scale q.k_j (capped, less the distance
// bias), out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), with a running maximum
// m. Scores are kept times log2(e), so that the exponentials are powers of two.
//
// The rows of one key head are the (token, head of the group) pairs of a
// sequence, i * G + g; sixteen rows make a tile, and a wave takes 32 keys of a
// tile at a time (a chunk).
#include <type_traits>

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

AttnPlan attn_plan(int B, int Hq, int Hkv, int max_q, int max_kv, DeviceTopo topo) {
  AttnPlan p;
  p.group = Hq / Hkv;
  p.rtiles = (int)(((long long)max_q * p.group + kRows - 1) / kRows);
  p.tiles = (size_t)B * Hkv * p.rtiles;
  const long long want = 4ll * topo.cus / (long long)p.tiles;
  const long long most = (max_kv + kWaves * kChunk - 1) / (kWaves * kChunk);
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

// The score, times log2(e), of a raw product.
struct ScoreRule {
  float scale;       // without a cap: factor; with one: 2 log2(e) scale / cap, of the exponential in tanh
  float cap;         // cap log2(e), or 0
  float slope;       // slope log2(e) of this lane's head
  __device__ __forceinline__ float operator()(float dot, int pos, int key) const {
    float s;
    // cap tanh(x) = cap - 2 cap / (1 + e^2x): 1 at x = inf, -1 at -inf
    if (cap > 0) s = cap - 2 * cap * __builtin_amdgcn_rcpf(1 + __builtin_amdgcn_exp2f(dot * scale));
    else s = dot * scale;
    return s - slope * fabsf((float)(pos - key));
  }
};

__device__ __forceinline__ ScoreRule score_rule(const AttentionArgs& a, int head) {
  ScoreRule r;
  r.scale = a.softcap > 0 ? 2 * kLog2e * a.scale / a.softcap : kLog2e * a.scale;
  r.cap = kLog2e * a.softcap;
  r.slope = a.slopes ? kLog2e * a.slopes[head] : 0.f;
  return r;
}

// One row's token (-1: none), head and range of keys.
struct Row {
  int token, head, pos, lo, hi;
};
__device__ __forceinline__ Row row_of(const AttnKernelArgs& p, int r, int q0, int q1, int kv, int hk) {
  const AttentionArgs& a = p.a;
  Row w = {-1, 0, 0, 0, 0};
  const int i = p.by_group(r);
  if (i >= q1 - q0) return w;
  w.token = q0 + i;
  w.head = hk * p.group + r - i * p.group;
  w.pos = kv - (q1 - q0) + i;
  w.lo = a.first ? max(a.first[w.token], 0) : 0;
  w.hi = min(a.end ? a.end[w.token] : w.pos + 1, kv);
  return w;
}

// Whether the low half is an infinity or a NaN.
template <bool BF>
__device__ __forceinline__ bool not_finite(uint32_t v) {
  constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
  return (v & e) == e;
}

// Block: one tile of 16 rows, one part of its keys; its waves take the chunks of
// the part in turn and meet in LDS. Bound: HBM, each key and value is read once
// per tile.
//
// Nothing but the final sums passes through LDS: the score product is taken as
// K q^T, whose result has a query per lane column and four neighbouring keys per
// register quad, which is (with the keys of the second 16 behind those of the
// first) the operand layout of the weights in the second product, V^T p^T. Its
// left operand wants eight keys of one dimension per lane: a lane loads 8 (or 4)
// dimensions of its eight keys, whole cache lines per 16 lanes, and pairs them up
// with byte permutes; dimension d = 8 m + i is row m of product i.
template <bool BF, int D>
__global__ void __launch_bounds__(256, D == 256 ? 1 : D == 128 ? 3 : 4) attention_split_kernel(AttnKernelArgs p) {
  constexpr int STEPS = D / 32;
  constexpr int CH = D >= 128 ? 8 : 4;  // dimensions per lane and half
  constexpr int NH = D / (16 * CH);
  constexpr int LD = D + 4;
  __shared__ float so[kWaves][kRows][LD];
  __shared__ float sml[kWaves][kRows][2];
  __shared__ int s_last;
  const AttentionArgs& a = p.a;
  // Blocks of the row tiles that read the same keys follow each other on one XCD.
  const int per = 8 * p.rtiles, w8 = blockIdx.x % per;
  const int rt = w8 / 8, unit = blockIdx.x / per * 8 + w8 % 8;
  if (unit >= a.B * a.Hkv * p.split) return;
  const int part = unit % p.split, hk = unit / p.split % a.Hkv, b = unit / p.split / a.Hkv;
  const int q0 = min(max(a.q_starts[b], 0), a.T), q1 = min(max(a.q_starts[b + 1], q0), min(a.T, q0 + a.max_q));
  const int kv = min(max(a.kv_lens[b], 0), a.max_kv);
  if (rt * kRows >= (q1 - q0) * p.group) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, kg = lane >> 4;
  const Row row = row_of(p, rt * kRows + n, q0, q1, kv, hk);
  const ScoreRule rule = score_rule(a, row.head);

  // The keys that any row sees, and those that all see.
  int lo = row.lo < row.hi ? row.lo : INT32_MAX, hi = row.lo < row.hi ? row.hi : 0;
  int all_lo = row.token < 0 ? 0 : row.lo, all_hi = row.token < 0 ? INT32_MAX : row.hi;  // rows past the last count as seeing all
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor(lo, o));
    hi = max(hi, __shfl_xor(hi, o));
    all_lo = max(all_lo, __shfl_xor(all_lo, o));
    all_hi = min(all_hi, __shfl_xor(all_hi, o));
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  all_lo = __builtin_amdgcn_readfirstlane(all_lo);
  all_hi = __builtin_amdgcn_readfirstlane(all_hi);
  const int c_first = lo < hi ? lo / kChunk : 0, chunks = lo < hi ? (hi + kChunk - 1) / kChunk - c_first : 0;
  const int c0 = c_first + (int)((long long)chunks * part / p.split), c1 = c_first + (int)((long long)chunks * (part + 1) / p.split);

  u32x4 q[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
    q[s] = row.token < 0 ? u32x4{0, 0, 0, 0}
                         : *reinterpret_cast<const u32x4*>(a.q + row.token * a.q_stride + (long long)row.head * D + s * 32 + kg * 8);

  // Row (of D values) of key lane & 31 of a chunk; keys past the last seen one repeat it.
  const int32_t* table = a.page_table + (long long)b * a.table_stride;
  auto key_row = [&](int c) -> uint32_t {
    const int j = min(max(c * kChunk + (lane & 31), lo), hi - 1);
    const int at = p.by_page(j);
    const int page = min(max(table[at], 0), a.pages - 1);
    return ((uint32_t)page * a.Hkv + hk) * a.page_size + (j - at * a.page_size);
  };
  u32x4 k[2][STEPS];
  typedef typename Words<CH / 2>::T VT;
  VT v[NH][8];
  auto load_k = [&](uint32_t rows) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint16_t* src = a.k_cache + (size_t)__shfl(rows, 16 * t + n) * D + kg * 8;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) k[t][s] = *reinterpret_cast<const u32x4*>(src + s * 32);
    }
  };
  auto load_v = [&](uint32_t rows) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const uint16_t* src = a.v_cache + (size_t)__shfl(rows, 16 * (x >> 2) + 4 * kg + (x & 3)) * D + n * CH;
#pragma unroll
      for (int h = 0; h < NH; ++h) v[h][x] = *reinterpret_cast<const VT*>(src + h * 128);
    }
  };

  f32x4 acc[NH][CH] = {};
  float mx = -INFINITY, sum = 0;
  bool any_bad = false;
  uint32_t rows = 0, rows_next = 0;
  // One chunk; with MORE the next one's loads go out as the registers fall free.
  auto step = [&](int c, auto more) {
    constexpr bool MORE = decltype(more)::value;
    f32x4 st[2] = {};
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int t = 0; t < 2; ++t) st[t] = mfma16<BF>(k[t][s], q[s], st[t]);
    if constexpr (MORE) {
      // The page lookup before the keys: loads come back in order, and its row is computed with first.
      const uint32_t next = rows_next;
      rows_next = key_row(c + 2 * kWaves);
      rows = next;
      __builtin_amdgcn_sched_barrier(0);  // the loads take the registers that the products above have read
      load_k(rows);
      __builtin_amdgcn_sched_barrier(0);
    }
    // Scores: keys 32c + 16t + 4kg + r of row n.
    const int j0 = c * kChunk + 4 * kg;
    const bool whole = c * kChunk >= all_lo && (c + 1) * kChunk <= all_hi;  // seen by every row
    float s[8], best = -INFINITY;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int j = j0 + 16 * (x >> 2) + (x & 3);
      s[x] = rule(st[x >> 2][x & 3], row.pos, j);
      if (!whole) s[x] = j >= row.lo && j < row.hi ? s[x] : -INFINITY;
      best = fmaxf(best, s[x]);
    }
    best = fmaxf(best, __shfl_xor(best, 16));
    best = fmaxf(best, __shfl_xor(best, 32));
    if (__any(best > mx)) {
      const float m = fmaxf(mx, best);
      const float f = mx == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx - m);
      sum *= f;
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int i = 0; i < CH; ++i) acc[h][i] *= f;
      mx = m;
    }
    const float off = mx == -INFINITY ? 0.f : mx;
    u32x4 w;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      w[x] = pack_pair<BF>(__builtin_amdgcn_exp2f(s[2 * x] - off), __builtin_amdgcn_exp2f(s[2 * x + 1] - off));
      // The rounded weights make the denominator too: their common rounding cancels.
      sum += bits_to_float<BF>((uint16_t)w[x]) + bits_to_float<BF>((uint16_t)(w[x] >> 16));
    }
    if (!whole) {
      // Places that no row sees may hold anything: they count as 0. So does a value
      // that is not finite, as it must not reach the rows that do not see it (0 times
      // it is NaN); those that do get it back after the loop.
      bool bad = false;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int j = j0 + 16 * (x >> 2) + (x & 3);
        const bool out = j < lo || j >= hi;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int y = 0; y < CH / 2; ++y) {
            if (out) v[h][x][y] = 0;
            bad = bad || not_finite<BF>(v[h][x][y]) || not_finite<BF>(v[h][x][y] >> 16);
          }
      }
      if (__any(bad)) {
        any_bad = true;
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
          for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int y = 0; y < CH / 2; ++y)
              v[h][x][y] &= (not_finite<BF>(v[h][x][y]) ? 0u : 0xFFFFu) | (not_finite<BF>(v[h][x][y] >> 16) ? 0u : 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const uint32_t sel = i & 1 ? 0x07060302u : 0x05040100u;
        u32x4 vt;
#pragma unroll
        for (int x = 0; x < 4; ++x) vt[x] = __builtin_amdgcn_perm(v[h][2 * x + 1][i / 2], v[h][2 * x][i / 2], sel);
        acc[h][i] = mfma16<BF>(vt, w, acc[h][i]);
      }
    if constexpr (MORE) {
      __builtin_amdgcn_sched_barrier(0);
      load_v(rows);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int c = c0 + wave;
  if (c < c1) {
    rows = key_row(c);
    load_k(rows);
    load_v(rows);
    rows_next = key_row(c + kWaves);
    for (; c + kWaves < c1; c += kWaves) step(c, std::true_type{});
    step(c, std::false_type{});
  }

  // The waves' sums meet in LDS, in wave order.
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < CH; i += 4)
        *reinterpret_cast<f32x4*>(&so[wave][n][h * 128 + (4 * kg + r) * CH + i]) =
            f32x4{acc[h][i][r], acc[h][i + 1][r], acc[h][i + 2][r], acc[h][i + 3][r]};
  if (kg == 0) sml[wave][n][0] = mx, sml[wave][n][1] = sum;
  if (any_bad) {
    // Rare: the values left out above, to the rows that see them.
    for (int c = c0 + wave; c < c1; c += kWaves) {
      if (c * kChunk >= all_lo && (c + 1) * kChunk <= all_hi) continue;
      const uint32_t here = key_row(c);
      for (int key = 0; key < kChunk; ++key) {
        const int j = c * kChunk + key;
        const uint16_t* src = a.v_cache + (size_t)__shfl(here, key) * D;
        if (j < row.lo || j >= row.hi) continue;
        for (int d = kg; d < D; d += 4)
          if (not_finite<BF>(src[d])) so[wave][n][d] += bits_to_float<BF>(src[d]);
      }
    }
  }
  __syncthreads();
  // Thread: row tid / 16, D / 16 neighbouring dimensions.
  constexpr int E = D / 16;
  const int r = tid >> 4, d0 = (tid & 15) * E;
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
  const Row mine = row_of(p, rt * kRows + r, q0, q1, kv, hk);
  if (p.split > 1) {
    // Partial sums of the parts, joined in order by the block that arrives last.
    const size_t tile = ((size_t)b * a.Hkv + hk) * p.rtiles + rt;
    float* po = p.part + ((tile * p.split + part) * kRows + r) * D + d0;
#pragma unroll
    for (int e = 0; e < E; e += 2) handoff_store(po + e, o[e], o[e + 1]);
    if ((tid & 15) == 0) handoff_store(p.part_ml + ((tile * p.split + part) * kRows + r) * 2, m, l);
    if (!handoff_last(&p.counters[tile], (uint32_t)p.split, &s_last)) return;
    const float* qo = p.part + (tile * p.split * kRows + r) * D + d0;
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
        for (int e = 0; e < E / 2; ++e) os[s][e] = handoff_load_pair(qo + (size_t)at * kRows * D + 2 * e);
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
    *reinterpret_cast<u32x2*>(dst + e) = u32x2{pack_pair<BF>(o[e] * inv, o[e + 1] * inv), pack_pair<BF>(o[e + 2] * inv, o[e + 3] * inv)};
}

template <bool BF, int D>
hipError_t launch_split(const AttentionArgs& a, hipStream_t stream) {
  const AttnPlan plan = attn_plan(a.B, a.Hq, a.Hkv, a.max_q, a.max_kv, device_topology());
  AttnKernelArgs p = {a, fixed_div(a.page_size), fixed_div(plan.group), plan.group, plan.rtiles, plan.split, reinterpret_cast<uint32_t*>(a.workspace), nullptr, nullptr};
  if (plan.split > 1) {
    p.part = reinterpret_cast<float*>(a.workspace + kWorkspaceHeader);
    p.part_ml = p.part + plan.tiles * plan.split * kRows * D;
  }
  const long long units = (long long)a.B * a.Hkv * plan.split, blocks = (units + 7) / 8 * 8 * plan.rtiles;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  attention_split_kernel<BF, D><<<dim3((unsigned)blocks), 64 * kWaves, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv) {
  const AttnPlan p = attn_plan(B, Hq, Hkv, max_q, max_kv, device_topology());
  return p.split > 1 ? kWorkspaceHeader + p.tiles * p.split * kRows * (D + 2) * sizeof(float) : 0;
}

hipError_t launch_attention(const AttentionArgs& a, bool bf16, hipStream_t stream) {
  if (bf16) {
    if (a.D == 64) return launch_split<true, 64>(a, stream);
    if (a.D == 128) return launch_split<true, 128>(a, stream);
    return launch_split<true, 256>(a, stream);
  }
  if (a.D == 64) return launch_split<false, 64>(a, stream);
  if (a.D == 128) return launch_split<false, 128>(a, stream);
  return launch_split<false, 256>(a, stream);
}

}  // namespace qmm
