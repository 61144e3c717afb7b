// Attention of new tokens to the paged cache of their sequences.
//
// For a query row n and keys j: s_j = scale q.k_j (capped, less the distance
// bias), out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), with a running maximum
// m.
#include <type_traits>

#include "attention_rows.h"

namespace qmm {
namespace {

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
  p.rtiles = row_tiles(max_q, p.group, kRows);
  p.tiles = (size_t)B * Hkv * p.rtiles;
  const long long want = 4ll * topo.cus / (long long)p.tiles;
  const long long most = (max_kv + kWaves * kChunk - 1ll) / (kWaves * kChunk);
  p.split = (int)(want < most ? want : most);
  if (p.split > kMaxSplit) p.split = kMaxSplit;
  if (p.split < 1 || p.tiles > (size_t)kGemvMaxStrips) p.split = 1;
  return p;
}

// Block: one tile of 16 rows, one part of its keys; its waves take the chunks of
// the part in turn and meet in LDS. Bound: HBM, each key and value is read once
// per tile: 48 queries on up to 8192 keys in a window of 4096, 32/8 heads of 128, 74 us,
// 4.4 TB/s. Latency for one sequence: 9.8 us at 1500 keys.
//
// Nothing but the final sums passes through LDS: the score product is taken as
// K q^T, whose result has a query per lane column and four neighbouring keys per
// register quad, which is (with the keys of the second 16 behind those of the
// first) the operand layout of the weights in the second product, V^T p^T. Its
// left operand wants eight keys of one dimension per lane: a lane loads 8 (or 4)
// dimensions of its eight keys, whole cache lines per 16 lanes, and pairs them up
// with byte permutes; dimension d = 8 m + i is row m of product i.
template <bool BF, int D, Cap CAP>
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
  const Span span = span_of(a, b);
  zero_rest<D>(p, span, b, hk, rt * p.split + part, p.rtiles * p.split);
  if (rt * kRows >= (span.q1 - span.q0) * p.group) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, kg = lane >> 4;
  const Row row = row_of(p, rt * kRows + n, span, hk);
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
  auto seen_by_all = [&](int c) { return c * kChunk >= all_lo && (uint32_t)(c + 1) * kChunk <= (uint32_t)all_hi; };
  const int c_first = lo < hi ? lo / kChunk : 0, chunks = lo < hi ? (hi - 1) / kChunk + 1 - c_first : 0;
  const int c0 = c_first + (int)((long long)chunks * part / p.split), c1 = c_first + (int)((long long)chunks * (part + 1) / p.split);

  u32x4 q[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
    q[s] = row.token < 0 ? u32x4{0, 0, 0, 0}
                         : *reinterpret_cast<const u32x4*>(a.q + row.token * a.q_stride + (long long)row.head * D + s * 32 + kg * 8);

  // Row (of D values) of key lane & 31 of a chunk; keys past the last seen one repeat it.
  const int32_t* table = a.page_table + (long long)b * a.table_stride;
  auto key_row = [&](int c) -> uint32_t {  // (the chunks asked for ahead may lie past 2^31)
    const int j = (int)min(max((uint32_t)c * kChunk + (lane & 31), (uint32_t)lo), (uint32_t)hi - 1);
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
  // (the lane's part in one base: added per row it costs the registers that make D 128 spill,
  // one query on 1500 keys 9.5 -> 10.1 us)
  const uint16_t* vbase = a.v_cache + n * CH;
  auto load_v = [&](uint32_t rows) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const uint16_t* src = vbase + (size_t)__shfl(rows, 16 * (x >> 2) + 4 * kg + (x & 3)) * D;
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
    const bool whole = seen_by_all(c);
    float s[8], best = -INFINITY;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int j = j0 + 16 * (x >> 2) + (x & 3);
      s[x] = rule.template score<CAP, true>(st[x >> 2][x & 3], row.pos, j);
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
      if (seen_by_all(c)) continue;
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
    if (!handoff_last(&p.counters[tile], (uint32_t)p.split, &s_last) || mine.token < 0) return;
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
    *reinterpret_cast<u32x2*>(dst + e) = u32x2{pack_pair<BF>(o[e] * inv, o[e + 1] * inv), pack_pair<BF>(o[e + 2] * inv, o[e + 3] * inv)};
}

// Sixteen bytes per lane from its own address to LDS, lane l's to lds_addr + 16 l
// (lds_addr uniform). One asm block, as the compiler would make every later LDS read
// wait for the builtin's; the wait before the barrier that publishes the tile is
// explicit. No vector register is written; m0 is restored.
__device__ __forceinline__ void load_to_lds(uint32_t lds_addr, const void* src) {
  uint32_t saved;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
               : "=&s"(saved)
               : "s"(lds_addr), "v"(src)
               : "memory");
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
// Transposed read: each 16 lanes' 8-byte pieces are four rows of sixteen 16-bit
// values (four lanes a row); lane c of them gets column c of the four rows.
__device__ __forceinline__ u32x2 read_transposed(const void* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

constexpr int kTileRows = 128;                                   // rows per block, 32 per wave
template <int D> constexpr int kTileKeys = D == 256 ? 32 : 64;  // keys per step

// Block: 128 rows of one key head, all their keys in steps that go through two LDS
// buffers, loaded straight from the cache a step ahead. Bound: the exponentials and
// reciprocals (half the vector rate), above all with a cap, then the matrix cores: a
// prompt of 8192 with a cap, 32/8 heads of 128, 700 us, 786 TFLOP/s. 32 rows a wave, so
// that two waves a SIMD fit the registers; 64 keys a step, 32 at D 256.
//
// As above K q^T is taken, whose result has a query per lane column: the softmax
// needs one exchange between lanes, and its weights are the operand of V^T p^T as
// they are, for the four neighbouring keys that a transposed LDS read of V gives.
// The 16-byte pieces of an LDS row are reordered by the row (an exclusive or), so
// that both the rows' reads and the transposed reads fall on distinct banks.
template <bool BF, int D, Cap CAP, bool SLOPES>
__global__ void __launch_bounds__(256, D == 256 ? 1 : 2) attention_tile_kernel(AttnKernelArgs p) {
  constexpr int BN = kTileKeys<D>, SUB = BN / 32, PIECES = D / 8, STEPS = D / 16, MT = D / 32;
  constexpr int OWN = BN / kWaves, LOADS = OWN * D * 2 / 1024, PER_LOAD = 512 / D;  // keys a wave loads, in how many loads
  constexpr int LDO = 36;
  __shared__ __attribute__((aligned(16))) uint16_t kvs[2][2][BN * D];
  __shared__ int range[2][kWaves];
  static_assert(sizeof(kvs) >= kTileRows * LDO * 4, "the result passes through the same LDS");
  const AttentionArgs& a = p.a;
  const int per = 8 * p.rtiles, w8 = blockIdx.x % per;
  const int rt = p.rtiles - 1 - w8 / 8, unit = blockIdx.x / per * 8 + w8 % 8;  // the longest rows of a causal mask first
  if (unit >= a.B * a.Hkv) return;
  const int hk = unit % a.Hkv, b = unit / a.Hkv;
  const Span span = span_of(a, b);
  zero_rest<D>(p, span, b, hk, rt, p.rtiles);
  if ((long long)rt * kTileRows >= (long long)(span.q1 - span.q0) * p.group) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 31, kg = lane >> 5;
  const int r0 = rt * kTileRows + wave * 32;
  const Row row = row_of(p, r0 + n, span, hk);
  // A negative scale turns the queries' signs instead: products are then in the scores' order.
  ScoreRule rule = score_rule(a, row.head);
  const uint32_t q_sign = rule.scale < 0 ? 0x80008000u : 0u;
  rule.scale = fabsf(rule.scale);
  rule.inverse = fabsf(rule.inverse);

  // Keys that any row of the wave sees, and those that all see; the block's from the waves'.
  int lo = row.lo < row.hi ? row.lo : INT32_MAX, hi = row.lo < row.hi ? row.hi : 0;
  int all_lo = row.token < 0 ? 0 : row.lo, all_hi = row.token < 0 ? INT32_MAX : row.hi;  // rows past the last count as seeing all
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor(lo, o));
    hi = max(hi, __shfl_xor(hi, o));
    all_lo = max(all_lo, __shfl_xor(all_lo, o));
    all_hi = min(all_hi, __shfl_xor(all_hi, o));
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  all_lo = __builtin_amdgcn_readfirstlane(all_lo);
  all_hi = __builtin_amdgcn_readfirstlane(all_hi);
  if (lane == 0) range[0][wave] = lo, range[1][wave] = hi;
  __syncthreads();
  int block_lo = INT32_MAX, block_hi = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) block_lo = min(block_lo, range[0][w]), block_hi = max(block_hi, range[1][w]);
  block_lo = __builtin_amdgcn_readfirstlane(block_lo);
  block_hi = __builtin_amdgcn_readfirstlane(block_hi);
  const int t0 = block_lo < block_hi ? block_lo / BN : 0, t1 = block_lo < block_hi ? (block_hi - 1) / BN + 1 : 0;

  u32x4 q[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
    q[s] = row.token < 0 ? u32x4{0, 0, 0, 0}
                         : *reinterpret_cast<const u32x4*>(a.q + row.token * a.q_stride + (long long)row.head * D + s * 16 + kg * 8) ^ q_sign;

  // Reordering of row r's pieces.
  auto turn = [](int r) { return D == 64 ? ((r >> 1) & 1) << 2 | ((r >> 2) & 3) : (r & 3) << 2 | ((r >> 2) & 3); };
  const int32_t* table = a.page_table + (long long)b * a.table_stride;
  auto key_row = [&](uint32_t key) -> uint32_t {  // keys past those seen repeat the nearest
    const int j = (int)min(max(key, (uint32_t)block_lo), (uint32_t)block_hi - 1);
    const int at = p.by_page(j);
    const int page = min(max(table[at], 0), a.pages - 1);
    return ((uint32_t)page * a.Hkv + hk) * a.page_size + (j - at * a.page_size);
  };
  auto own_rows = [&](int t) { return key_row((uint32_t)t * BN + wave * OWN + (lane & (OWN - 1))); };
  auto load_tile = [&](int buf, uint32_t rows) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int local = i * PER_LOAD + lane / PIECES;
      const size_t at = (size_t)__shfl(rows, local) * D + ((lane % PIECES) ^ turn(wave * OWN + local)) * 8;
      const uint32_t to = (uint32_t)(wave * OWN + i * PER_LOAD) * D * 2;
      load_to_lds(lds_offset(kvs[buf][0]) + to, a.k_cache + at);
      load_to_lds(lds_offset(kvs[buf][1]) + to, a.v_cache + at);
    }
  };
  // Whether none of the wave's rows sees a key of the step that starts at key0, and whether all see all.
  auto seen_by_none = [&](int key0) { return (uint32_t)key0 + BN <= (uint32_t)lo || key0 >= hi; };
  auto seen_by_all = [&](int key0) { return key0 >= all_lo && (uint32_t)key0 + BN <= (uint32_t)all_hi; };
  // Byte offsets of this lane's reads: keys' pieces per step, values' per 32 dimensions and four keys.
  uint32_t k_at[STEPS], v_at[MT][2];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) k_at[s] = n * D * 2 + ((2 * s + kg) ^ turn(n)) * 16;
  {
    const int i = (lane & 15) >> 2;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = 4 * kg + 8 * h + i, piece = 4 * m + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
        v_at[m][h] = key * D * 2 + (piece ^ turn(key)) * 16 + (lane & 1) * 8;
      }
  }

  f32x16 o[MT] = {};
  float mx = -INFINITY, sum = 0;
  bool any_bad = false;
  uint32_t rows = 0;
  if (t0 < t1) {
    load_tile(t0 & 1, own_rows(t0));
    rows = own_rows(t0 + 1);
  }
  for (int t = t0; t < t1; ++t) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (t + 1 < t1) {
      load_tile((t + 1) & 1, rows);
      rows = own_rows(t + 2);
    }
    const int key0 = t * BN;
    if (seen_by_none(key0)) continue;
    const char* ks = reinterpret_cast<const char*>(kvs[t & 1][0]);
    const char* vs = reinterpret_cast<const char*>(kvs[t & 1][1]);
    // Products of keys and queries, the keys' pieces read kAhead steps before.
    constexpr int kAhead = 3;
    f32x16 st[SUB] = {};
    u32x4 kf[kAhead + 1][SUB];
    auto read_keys = [&](int s) {
#pragma unroll
      for (int u = 0; u < SUB; ++u) kf[s % (kAhead + 1)][u] = *reinterpret_cast<const u32x4*>(ks + k_at[s] + u * 32 * D * 2);
    };
#pragma unroll
    for (int s = 0; s < kAhead; ++s) read_keys(s);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (s + kAhead < STEPS) read_keys(s + kAhead);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < SUB; ++u) st[u] = mfma32<BF>(kf[s % (kAhead + 1)][u], q[s], st[u]);
    }
    const bool whole = seen_by_all(key0);
    auto key_of = [&](int u, int i) { return key0 + 32 * u + 8 * (i >> 2) + 4 * kg + (i & 3); };
    // The largest score of the row; where a score is more than a multiply-add or a small cap of its
    // product the scores are taken first, else only that of the largest product.
    constexpr bool FIRST = SLOPES || CAP == kAnyCap;
    float best = -INFINITY;
    uint32_t seen = ~0u;  // bit 16 u + i: the row sees key_of(u, i)
    if (FIRST) {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) st[u][i] = rule.template score<CAP, SLOPES>(st[u][i], row.pos, key_of(u, i));
    }
    if (!whole) {
      seen = 0;
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool in = (uint32_t)(key_of(u, i) - row.lo) < (uint32_t)max(row.hi - row.lo, 0);
          seen |= in ? 1u << (16 * u + i) : 0u;
          best = fmaxf(best, in ? st[u][i] : -INFINITY);
        }
    } else {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) best = fmaxf(best, st[u][i]);
    }
    if (!FIRST) best = seen ? rule.template score<CAP, false>(best, 0, 0) : -INFINITY;
    best = fmaxf(best, __shfl_xor(best, 32));
    // A row's maximum is left where it is while no weight passes 2^8: rescaling is rare.
    if (__any(best > mx + 8)) {
      const float m = best > mx + 8 ? best : mx;
      const float f = mx == m ? 1.f : __builtin_amdgcn_exp2f(mx - m);
      sum *= f;
#pragma unroll
      for (int m2 = 0; m2 < MT; ++m2) o[m2] *= f;
      mx = m;
    }
    const float off = mx == -INFINITY ? 0.f : mx;
    // Exponents: the scores less the maximum, in one multiply-add of the product (or, with a cap, of
    // the reciprocal in the tanh).
    if (FIRST) {
#pragma unroll
      for (int u = 0; u < SUB; ++u) st[u] -= off;
    } else if (CAP == kSmallCap) {
      // Stage by stage over sixteen: left to itself the compiler takes two at a time, each
      // waiting for its own exponential and reciprocal.
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
#pragma unroll
        for (int i = 0; i < 16; ++i) st[u][i] *= rule.scale;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 16; ++i) st[u][i] = __builtin_amdgcn_exp2f(st[u][i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 16; ++i) st[u][i] += 1;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 16; ++i) st[u][i] = __builtin_amdgcn_rcpf(st[u][i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 16; ++i) st[u][i] = fmaf(-2 * rule.cap, st[u][i], rule.cap - off);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) st[u][i] = fmaf(st[u][i], rule.scale, -off);
    }
    if (!whole) {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) st[u][i] = seen >> (16 * u + i) & 1 ? st[u][i] : -INFINITY;
    }
    if (!whole) {
      // A value that is not finite must not reach rows that do not see it (0 times it is
      // NaN): the rare step that holds one leaves its values to the end.
      bool bad = false;
#pragma unroll 4
      for (int i = lane; i < BN * D / 8; i += 64) {
        const u32x4 x = reinterpret_cast<const u32x4*>(vs)[i];
#pragma unroll
        for (int y = 0; y < 4; ++y) bad |= (int)not_finite<BF>(x[y]) | (int)not_finite<BF>(x[y] >> 16);
      }
      if (__any(bad)) {
        any_bad = true;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int i = 0; i < 16; i += 2)
            sum = add_pair<BF>(pack_pair<BF>(__builtin_amdgcn_exp2f(st[u][i]), __builtin_amdgcn_exp2f(st[u][i + 1])), sum);
        continue;
      }
    }
    // Weights and their products with the values, sixteen keys at a time: the next ones'
    // exponentials and reads go between the matrix operations.
    constexpr int GROUPS = BN / 16;
    u32x4 vf[2][MT], w[2];
    auto read_values = [&](int g) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32x2 x = read_transposed(vs + v_at[m][0] + g * 16 * D * 2), y = read_transposed(vs + v_at[m][1] + g * 16 * D * 2);
        vf[g & 1][m] = u32x4{x[0], x[1], y[0], y[1]};
      }
    };
    auto weigh = [&](int g) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = 8 * (g & 1) + 2 * x;
        w[g & 1][x] = pack_pair<BF>(__builtin_amdgcn_exp2f(st[g >> 1][i]), __builtin_amdgcn_exp2f(st[g >> 1][i + 1]));
        sum = add_pair<BF>(w[g & 1][x], sum);  // the rounded weights make the denominator too
      }
    };
    read_values(0);
    weigh(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      if (g + 1 < GROUPS) {
        read_values(g + 1);
        weigh(g + 1);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) o[m] = mfma32<BF>(vf[g & 1][m], w[g & 1], o[m]);
      if (g + 1 < GROUPS) {
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * MT, 0);  // LDS reads
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);               // a matrix operation
          __builtin_amdgcn_sched_group_barrier(0x402, (16 + MT - 1) / MT, 0);  // vector operations
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Results leave by LDS, 32 dimensions at a time, each wave for its own rows.
  sum += __shfl_xor(sum, 32);
  const float inv = row.lo < row.hi ? 1 / sum : 0.f;
  __syncthreads();
  float* so = reinterpret_cast<float*>(&kvs[0][0][0]) + wave * 32 * LDO;
  const Row mine = row_of(p, r0 + (lane >> 1), span, hk);
  // Rare: dimensions 32 m on of the steps left out above, key by key, with their scores anew.
  auto add_left_out = [&](int m) {
    for (int t = t0; t < t1; ++t) {
      const int key0 = t * BN;
      if (seen_by_none(key0) || seen_by_all(key0)) continue;
      const uint32_t here = key_row(key0 + (lane & (BN - 1)));
      bool bad = false;
      for (int d = lane / BN; d < D; d += 64 / BN) bad |= not_finite<BF>(a.v_cache[(size_t)here * D + d]);
      if (!__any(bad)) continue;
      for (int key = 0; key < BN; ++key) {
        const size_t at = (size_t)__shfl(here, key) * D;
        const bool in = key0 + key >= row.lo && key0 + key < row.hi;
        if (!in) continue;
        const uint16_t* qr = a.q + row.token * a.q_stride + (long long)row.head * D;
        float dot = 0;
        for (int d = 0; d < D; ++d) dot += bits_to_float<BF>((uint16_t)(qr[d] ^ q_sign)) * bits_to_float<BF>(a.k_cache[at + d]);
        const float s = rule.template score<CAP, SLOPES>(dot, row.pos, key0 + key);
        const float weight = bits_to_float<BF>(float_to_bits<BF>(__builtin_amdgcn_exp2f(s - (mx == -INFINITY ? 0.f : mx))));
        for (int d = kg; d < 32; d += 2) so[n * LDO + d] += weight * inv * bits_to_float<BF>(a.v_cache[at + 32 * m + d]);
      }
    }
  };
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<f32x4*>(so + n * LDO + 8 * g + 4 * kg) =
          f32x4{o[m][4 * g] * inv, o[m][4 * g + 1] * inv, o[m][4 * g + 2] * inv, o[m][4 * g + 3] * inv};
    if (any_bad) add_left_out(m);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (mine.token >= 0) {
      const float* src = so + (lane >> 1) * LDO + 16 * (lane & 1);
      uint16_t* dst = a.out + ((long long)mine.token * a.Hq + mine.head) * D + 32 * m + 16 * (lane & 1);
#pragma unroll
      for (int e = 0; e < 16; e += 8)
        *reinterpret_cast<u32x4*>(dst + e) = u32x4{pack_pair<BF>(src[e], src[e + 1]), pack_pair<BF>(src[e + 2], src[e + 3]),
                                                   pack_pair<BF>(src[e + 4], src[e + 5]), pack_pair<BF>(src[e + 6], src[e + 7])};
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// Blocks of 128 rows where they are enough for a third of the CUs, else tiles of 16
// split over the keys. The blocks' time over the tiles', causal prompts of 64 to 2048,
// 32/8, 16/2 and 8/8 heads of 64, 128 and 256, 256 CUs: with 8 to 32 blocks 0.6 to 2.4,
// above 1 in 23 cases of 27; with 64 0.4 to 1.4; with 128 0.3 to 1.2; with 256 and more
// 0.3 to 0.7, a prompt of 8192 0.3. Few heads a key head are the tiles' side, many the
// blocks'. Where most blocks are short the tiles win beyond that: six ragged sequences of
// documents, 24 heads of 64, up to 2600 tokens 61 us in blocks, 55 in tiles; up to 512
// tokens 15 and 9.
bool use_tiles(int B, int Hq, int Hkv, int max_q, DeviceTopo topo) {
  const long long rows = (long long)max_q * (Hq / Hkv);
  return rows > 64 && (long long)B * Hkv * ((rows + kTileRows - 1) / kTileRows) * 3 >= topo.cus;
}

template <bool BF, int D>
hipError_t launch_tiles(const AttentionArgs& a, hipStream_t stream) {
  const int group = a.Hq / a.Hkv, rtiles = row_tiles(a.max_q, group, kTileRows);
  const AttnKernelArgs p = {a, fixed_div(a.page_size), fixed_div(group), group, rtiles, 1, nullptr, nullptr, nullptr};
  const dim3 grid((unsigned)tile_blocks(a.B, a.Hkv, rtiles));
  const auto run = [&](auto kernel) { kernel<<<grid, 64 * kWaves, 0, stream>>>(p); };
  switch (cap_kind(a.softcap)) {
    case kNoCap: run(a.slopes ? attention_tile_kernel<BF, D, kNoCap, true> : attention_tile_kernel<BF, D, kNoCap, false>); break;
    case kSmallCap: run(a.slopes ? attention_tile_kernel<BF, D, kSmallCap, true> : attention_tile_kernel<BF, D, kSmallCap, false>); break;
    case kAnyCap: run(a.slopes ? attention_tile_kernel<BF, D, kAnyCap, true> : attention_tile_kernel<BF, D, kAnyCap, false>); break;
  }
  return hipGetLastError();
}

template <bool BF, int D>
hipError_t launch_split(const AttentionArgs& a, hipStream_t stream) {
  const AttnPlan plan = attn_plan(a.B, a.Hq, a.Hkv, a.max_q, a.max_kv, device_topology());
  AttnKernelArgs p = {a, fixed_div(a.page_size), fixed_div(plan.group), plan.group, plan.rtiles, plan.split, reinterpret_cast<uint32_t*>(a.workspace), nullptr, nullptr};
  if (plan.split > 1) {
    p.part = reinterpret_cast<float*>(a.workspace + kWorkspaceHeader);
    p.part_ml = p.part + plan.tiles * plan.split * kRows * D;
  }
  const dim3 grid((unsigned)tile_blocks(a.B, a.Hkv * plan.split, plan.rtiles));
  const auto run = [&](auto kernel) { kernel<<<grid, 64 * kWaves, 0, stream>>>(p); };
  switch (cap_kind(a.softcap)) {
    case kNoCap: run(attention_split_kernel<BF, D, kNoCap>); break;
    case kSmallCap: run(attention_split_kernel<BF, D, kSmallCap>); break;
    case kAnyCap: run(attention_split_kernel<BF, D, kAnyCap>); break;
  }
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv) {
  if (use_tiles(B, Hq, Hkv, max_q, device_topology())) return 0;
  const AttnPlan p = attn_plan(B, Hq, Hkv, max_q, max_kv, device_topology());
  return p.split > 1 ? kWorkspaceHeader + p.tiles * p.split * kRows * (D + 2) * sizeof(float) : 0;
}

long long attention_blocks(int B, int Hq, int Hkv, int max_q, int max_kv) {
  const DeviceTopo topo = device_topology();
  if (use_tiles(B, Hq, Hkv, max_q, topo)) return tile_blocks(B, Hkv, row_tiles(max_q, Hq / Hkv, kTileRows));
  const AttnPlan p = attn_plan(B, Hq, Hkv, max_q, max_kv, topo);
  return tile_blocks(B, Hkv * p.split, p.rtiles);
}

template <bool BF>
hipError_t launch_dim(const AttentionArgs& a, hipStream_t stream) {
  if (use_tiles(a.B, a.Hq, a.Hkv, a.max_q, device_topology())) {
    if (a.D == 64) return launch_tiles<BF, 64>(a, stream);
    if (a.D == 128) return launch_tiles<BF, 128>(a, stream);
    return launch_tiles<BF, 256>(a, stream);
  }
  if (a.D == 64) return launch_split<BF, 64>(a, stream);
  if (a.D == 128) return launch_split<BF, 128>(a, stream);
  return launch_split<BF, 256>(a, stream);
}

hipError_t launch_attention(const AttentionArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_dim<true>(a, stream) : launch_dim<false>(a, stream);
}

}  // namespace qmm
