// Attention to the 4-bit cache for prompts: blocks of many rows, whose keys and values
// are decoded once into LDS.
#pragma once

#include <type_traits>

#include "kv4_attention.h"

namespace qmm {

struct Kv4TileArgs {
  AttentionArgs a;
  bool bf16;
};
// One launch per head dimension, each in a translation unit of its own.
template <int D> hipError_t launch_kv4_tiles(const Kv4TileArgs& t, int group_size, hipStream_t stream);
template <int D> constexpr int kKv4TileWaves = D == 256 ? 4 : 8;
template <int D> constexpr int kKv4TileRows = 32 * kKv4TileWaves<D>;

namespace {

// How a score follows from its product: a factor; a small cap; a large cap or a distance bias too.
enum ScoreKind { kPlainScore, kCappedScore, kAnyScore };

struct Kv4TileKernelArgs {
  AttnKernelArgs r;
  bool bf16;
};

// Block: 32 rows a wave of one key head, all their keys in steps of BN that go through two
// LDS buffers. The first half of the waves decodes the values of the next step, the second half
// the keys, from words asked for a step before that; then all take the step's products.
// Bound: the vector ALUs (exponentials, with a cap reciprocals too, and the decoding, which is why a
// block has as many rows as registers allow).
//
// K q^T has a query per lane column; its row m of a 32 x 32 product is key 16 (m / 16) +
// 8 (m / 4 % 2) + 4 (m / 8 % 2) + m % 4 of those 32, so that eight neighbouring registers of a lane are the
// eight tokens of a block, in order: the layout in which the weights are the second operand of V^T p^T,
// and in which a lane that decodes eight tokens' words of four channels writes four whole pieces of V^T.
// The 16-byte pieces of an LDS row are reordered by the row (an exclusive or) so that the reads and the
// writes of eight neighbouring lanes fall on distinct banks.
template <int D, int G, ScoreKind KIND>
__global__ void __launch_bounds__(64 * kKv4TileWaves<D>, D == 256 ? 1 : 2) kv4_tile_kernel(Kv4TileKernelArgs t) {
  constexpr int WAVES = kKv4TileWaves<D>, ROWS = kKv4TileRows<D>, GS = D / G, BLOCK = kv4_block_bytes(D, G);
  constexpr int BN = D == 256 ? 32 : 64, SUB = BN / 32, STEPS = D / 16, MT = D / 32, BLOCKS = BN / 8;
  constexpr int QUADS = D / 4, UNITS = BLOCKS * QUADS;        // eight tokens of four channels
  constexpr int HALF = 32 * WAVES, VU = (UNITS + HALF - 1) / HALF;  // threads of a half, units of one
  static_assert(BN * 4 <= HALF, "a thread decodes a fourth of a key");
  constexpr int K_BYTES = BN * D * 2, MID_BYTES = BN * 16, VM_BYTES = 8 * BN * 2, BUFFER = 2 * K_BYTES + MID_BYTES + VM_BYTES;
  constexpr int LDO = 36, OUT_BYTES = ROWS * LDO * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * BUFFER > OUT_BYTES ? 2 * BUFFER : OUT_BYTES];
  __shared__ int range[2][WAVES], s_bad;
  const AttnKernelArgs& p = t.r;
  const AttentionArgs& a = p.a;
  const uint8_t* k_cache = reinterpret_cast<const uint8_t*>(a.k_cache);
  const uint8_t* v_cache = reinterpret_cast<const uint8_t*>(a.v_cache);
  const int per = 8 * p.rtiles, w8 = blockIdx.x % per;
  const int rt = p.rtiles - 1 - w8 / 8, unit = blockIdx.x / per * 8 + w8 % 8;  // the longest rows of a causal mask first
  if (unit >= a.B * a.Hkv) return;
  const int hk = unit % a.Hkv, b = unit / a.Hkv;
  const Span span = span_of(a, b);
  zero_rest<D>(p, span, b, hk, rt, p.rtiles);
  if ((long long)rt * ROWS >= (long long)(span.q1 - span.q0) * p.group) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 31, kg = lane >> 5;
  const int r0 = rt * ROWS + wave * 32;
  const Row row = row_of(p, r0 + n, span, hk);
  ScoreRule rule = score_rule(a, row.head);

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
  if (tid == 0) s_bad = 0;
  __syncthreads();
  int block_lo = INT32_MAX, block_hi = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) block_lo = min(block_lo, range[0][w]), block_hi = max(block_hi, range[1][w]);
  block_lo = __builtin_amdgcn_readfirstlane(block_lo);
  block_hi = __builtin_amdgcn_readfirstlane(block_hi);
  const int t0 = block_lo < block_hi ? block_lo / BN : 0, t1 = block_lo < block_hi ? (block_hi - 1) / BN + 1 : 0;

  // The row's query, and its groups' sums in two parts (one a lane group).
  u32x4 q[STEPS], qsum = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
    q[s] = row.token < 0 ? u32x4{0, 0, 0, 0}
                         : *reinterpret_cast<const u32x4*>(a.q + row.token * a.q_stride + (long long)row.head * D + s * 16 + kg * 8);
  {
    const float back = scale_query<2>(q, t.bf16);
    // A negative scale turns the queries' signs instead: products are then in the scores' order.
    const uint32_t sign = rule.scale < 0 ? 0x80008000u : 0u;
    rule.scale = fminf(fabsf(rule.scale) * back, 3e38f);
    rule.inverse = fminf(fabsf(rule.inverse) * back, 3e38f);
    f16 part_of[8] = {};
#pragma unroll
    for (int s = 0; s < STEPS; ++s) q[s] ^= sign;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      f32x16 sums = {};  // in every lane of a column
#pragma unroll
      for (int s = g * GS / 16; s < (g + 1) * GS / 16; ++s) sums = mfma32<false>(u32x4{kOnes, kOnes, kOnes, kOnes}, q[s], sums);
      const f16 first = (f16)sums[0], second = (f16)(sums[0] - (float)first);
      part_of[g] = kg == 0 ? first : second;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) qsum[x] = as_u32(f16x2{part_of[2 * x], part_of[2 * x + 1]});
  }

  // ---- decoding -----------------------------------------------------------------------
  const DecodeMasks masks;
  const bool on_values = wave < WAVES / 2;
  const int dt = tid & (HALF - 1);  // a thread's number within its half
  const int32_t* table = a.page_table + (long long)b * a.table_stride;
  // Number of the block of eight tokens, i in the step; past the seen keys' ends the nearest.
  auto token_block = [&](int step, int i) -> uint32_t {
    const int j = (int)min(max((uint32_t)step * BN + 8 * i, (uint32_t)block_lo), (uint32_t)block_hi - 1);
    const int at = p.by_page(j);
    const int page = min(max(table[at], 0), a.pages - 1);
    return (((uint32_t)page * a.Hkv + hk) * a.page_size + (j - at * a.page_size)) / kBlockTokens;
  };
  // Keys: thread 4 key + g has words (D / 32) g on of the key. Values: unit (block, quad), quads first.
  constexpr int KW = D / 32;
  const int key = dt >> 2, kquarter = dt & 3;
  // What a thread has asked for: its key's words, then scales and middles; or per unit words, scales and middles.
  constexpr int RAW = KW + G > 12 * VU ? KW + G : 12 * VU;
  uint32_t raw[RAW], at_block[VU];  // at_block: of the next load
  auto raw4 = [&](int i) { return u32x4{raw[4 * i], raw[4 * i + 1], raw[4 * i + 2], raw[4 * i + 3]}; };
  auto find = [&](int step) {
    if (on_values) {
#pragma unroll
      for (int i = 0; i < VU; ++i) at_block[i] = token_block(step, (dt + i * HALF) / QUADS % BLOCKS);
    } else {
      at_block[0] = token_block(step, key / 8 % BLOCKS);
    }
  };
  auto load = [&]() {
    if (on_values) {
#pragma unroll
      for (int i = 0; i < VU; ++i) {
        const int quad = (dt + i * HALF) % QUADS;
        const uint8_t* src = v_cache + (size_t)at_block[i] * BLOCK;
        load_words<16>(raw + 12 * i, src + quad * 16);
        load_words<32>(raw + 12 * i + 4, src + 4 * D + quad * 4 / GS * 32);
      }
    } else {
      const uint8_t* src = k_cache + (size_t)at_block[0] * BLOCK + (key & 7) * (D / 2);
      load_words<D / 8>(raw, src + kquarter * (D / 8));
      load_words<4 * G>(raw + KW, k_cache + (size_t)at_block[0] * BLOCK + 4 * D + (key & 7) * 4 * G);
    }
  };
  auto key_turn = [](int k) { return (k >> 1 & 1) | (k >> 3 & 1) << 1 | (k & 1) << 2; };
  auto channel_turn = [](int c) { return BN == 32 ? c >> 1 & 3 : ((c ^ c >> 3) & 3) | (c & 4); };
  auto decode_step = [&](int step) {
    uint8_t* buffer = lds + (step & 1) * BUFFER;
    if (on_values) {
#pragma unroll
      for (int i = 0; i < VU; ++i) {
        const int u = dt + i * HALF, quad = u % QUADS, blk = u / QUADS;
        if (UNITS % HALF && u >= UNITS) continue;
        // Tokens that no row sees may hold anything: their scales and middles count as 0. So do those of a seen one
        // that are not finite, as they must not reach the rows that do not see it (0 times NaN is NaN); those that
        // do get a NaN at the end.
        const int j0 = step * BN + 8 * blk;
        const u32x4 words = raw4(3 * i);
        u32x4 sv = raw4(3 * i + 1), mv = raw4(3 * i + 2);
        uint32_t bad = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int j = j0 + 2 * x;
          const uint32_t in = (j >= block_lo && j < block_hi ? 0xFFFFu : 0u) | (j + 1 >= block_lo && j + 1 < block_hi ? 0xFFFF0000u : 0u);
          const uint32_t nf = (not_finite_halves(sv[x]) | not_finite_halves(mv[x])) & in;
          bad |= nf;
          sv[x] &= in & ~nf;
          mv[x] &= in & ~nf;
        }
        if (bad) s_bad = 1;
        f16x2 ss[4], c24[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          ss[x] = as_f16x2(sv[x]);
          c24[x] = times_24(ss[x]);
        }
        uint8_t* to = buffer + K_BYTES;
        auto channel = [&](auto r) {
          constexpr int R = decltype(r)::value;
          const int c = 4 * quad + R;
          *reinterpret_cast<u32x4*>(to + c * (2 * BN) + ((blk ^ channel_turn(c)) * 16)) =
              u32x4{decode<R>(words[0], ss[0], c24[0], masks), decode<R>(words[1], ss[1], c24[1], masks),
                    decode<R>(words[2], ss[2], c24[2], masks), decode<R>(words[3], ss[3], c24[3], masks)};
        };
        channel(std::integral_constant<int, 0>{});
        channel(std::integral_constant<int, 1>{});
        channel(std::integral_constant<int, 2>{});
        channel(std::integral_constant<int, 3>{});
        if (quad * 4 % GS == 0) *reinterpret_cast<u32x4*>(buffer + 2 * K_BYTES + MID_BYTES + quad * 4 / GS * (2 * BN) + blk * 16) = mv;
      }
    } else if (BN * 4 == HALF || dt < BN * 4) {
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const int g = i * 32 / GS;
        const f16 sg = as_f16x2(raw[KW + g / 2])[g % 2];
        const f16x2 ss = {sg, sg}, c24 = times_24(ss);
        *reinterpret_cast<u32x4*>(buffer + key * (2 * D) + (((4 * i + kquarter) ^ key_turn(key)) * 16)) =
            u32x4{decode<0>(raw[i], ss, c24, masks), decode<1>(raw[i], ss, c24, masks), decode<2>(raw[i], ss, c24, masks),
                  decode<3>(raw[i], ss, c24, masks)};
      }
      if (kquarter == 0) {
        u32x4 middles = {0, 0, 0, 0};
        if constexpr (G == 1) {
          middles[0] = raw[KW] >> 16;
        } else {
#pragma unroll
          for (int x = 0; x < G / 2; ++x) middles[x] = raw[KW + G / 2 + x];
        }
        *reinterpret_cast<u32x4*>(buffer + 2 * K_BYTES + key * 16) = middles;
      }
    }
  };

  // ---- products -------------------------------------------------------------------------
  auto seen_by_none = [&](int key0) { return (uint32_t)key0 + BN <= (uint32_t)lo || key0 >= hi; };
  auto seen_by_all = [&](int key0) { return key0 >= all_lo && (uint32_t)key0 + BN <= (uint32_t)all_hi; };
  const int my_key = (n & 19) | (n & 4) << 1 | (n & 8) >> 1;  // of the 32 of row n: bits 2 and 3 change places
  uint32_t k_at[STEPS], v_at[MT];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) k_at[s] = my_key * (2 * D) + (((2 * s + kg) ^ key_turn(my_key)) * 16);
#pragma unroll
  for (int m = 0; m < MT; ++m) v_at[m] = (32 * m + n) * (2 * BN);
  const int my_turn = channel_turn(n);  // (the same for channels 32 apart)

  f32x16 o[MT] = {}, rest = {};  // rest: rows g < 8 the sums of p m_g, row 8 the sum of p
  float mx = -INFINITY;
  if (t0 < t1) {
    find(t0);
    load();
    find(t0 + 1);
    decode_step(t0);
    load();
    find(t0 + 2);
  }
  for (int step = t0; step < t1; ++step) {
    __syncthreads();  // the step's keys and values are there; those of the step before are done with
    if (step + 1 < t1) {
      decode_step(step + 1);
      load();
      find(step + 3);
    }
    const int key0 = step * BN;
    if (seen_by_none(key0)) continue;
    const uint8_t* ks = lds + (step & 1) * BUFFER;
    const uint8_t* vs8 = ks + K_BYTES;
    const uint8_t* mids = ks + 2 * K_BYTES;
    const uint8_t* vmids = mids + MID_BYTES;
    // Products of keys and queries, the keys' pieces read kAhead steps before.
    constexpr int kAhead = 3;
    f32x16 st[SUB] = {};
    u32x4 kf[kAhead + 1][SUB];
    auto read_keys = [&](int s) {
#pragma unroll
      for (int u = 0; u < SUB; ++u) kf[s % (kAhead + 1)][u] = *reinterpret_cast<const u32x4*>(ks + k_at[s] + u * 32 * D * 2);
    };
    u32x4 km[SUB];
#pragma unroll
    for (int u = 0; u < SUB; ++u) km[u] = *reinterpret_cast<const u32x4*>(mids + (32 * u + my_key) * 16);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) read_keys(s);
#pragma unroll
    for (int u = 0; u < SUB; ++u) st[u] = mfma32<false>(km[u], qsum, st[u]);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (s + kAhead < STEPS) read_keys(s + kAhead);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < SUB; ++u) st[u] = mfma32<false>(kf[s % (kAhead + 1)][u], q[s], st[u]);
    }
    const bool whole = seen_by_all(key0);
    auto key_of = [&](int u, int i) { return key0 + 32 * u + 16 * (i >> 3) + 8 * kg + (i & 7); };
    // The largest score of the row; where a score is more than a multiply-add or a small cap of its
    // product the scores are taken first, else only that of the largest product.
    float best = -INFINITY;
    uint32_t seen = ~0u;  // bit 16 u + i: the row sees key_of(u, i)
    if (KIND == kAnyScore) {
      const bool slopes = a.slopes != nullptr;
      const Cap cap = cap_kind(a.softcap);
      if (cap == kSmallCap) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            st[u][i] = rule.template score<kSmallCap, false>(st[u][i], 0, 0);
            if (i % 8 == 7) __builtin_amdgcn_sched_barrier(0);
          }
      } else if (cap == kAnyCap) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            st[u][i] = rule.template score<kAnyCap, false>(st[u][i], 0, 0);
            if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // (or the registers do not suffice)
          }
      } else {
#pragma unroll
        for (int u = 0; u < SUB; ++u) st[u] *= rule.scale;
      }
      if (slopes) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) st[u][i] -= rule.slope * fabsf((float)(row.pos - key_of(u, i)));
      }
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
    if (KIND == kPlainScore) best = seen ? rule.template score<kNoCap, false>(best, 0, 0) : -INFINITY;
    if (KIND == kCappedScore) best = seen ? rule.template score<kSmallCap, false>(best, 0, 0) : -INFINITY;
    best = fmaxf(best, __shfl_xor(best, 32));
    if (__any(best > mx + kSlack)) {
      const float m = best > mx + kSlack ? best : mx;
      const float f = mx == m ? 1.f : __builtin_amdgcn_exp2f(mx - m);
      rest *= f;
#pragma unroll
      for (int m2 = 0; m2 < MT; ++m2) o[m2] *= f;
      mx = m;
    }
    const float off = mx == -INFINITY ? 0.f : mx - kLift;
    // Exponents: the scores less the maximum, in one multiply-add of the product (or, with a cap, of
    // the reciprocal in the tanh).
    if (KIND == kAnyScore) {
#pragma unroll
      for (int u = 0; u < SUB; ++u) st[u] -= off;
    } else if (KIND == kCappedScore) {
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
    // Weights and their products with the values, sixteen keys at a time: the next ones'
    // exponentials and reads go between the matrix operations.
    constexpr int GROUPS = BN / 16;
    u32x4 vf[2][MT + 1], w[2];
    auto read_values = [&](int g) {
      const int piece = 2 * g + kg;
#pragma unroll
      for (int m = 0; m < MT; ++m) vf[g & 1][m] = *reinterpret_cast<const u32x4*>(vs8 + v_at[m] + ((piece ^ my_turn) * 16));
      const u32x4 x = *reinterpret_cast<const u32x4*>(vmids + min(n, G - 1) * (2 * BN) + piece * 16);
#pragma unroll
      for (int y = 0; y < 4; ++y) vf[g & 1][MT][y] = n < G ? x[y] : n == 8 ? kOnes : 0u;
    };
    auto weigh = [&](int g) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = 8 * (g & 1) + 2 * x;
        w[g & 1][x] = pack_pair<false>(__builtin_amdgcn_exp2f(st[g >> 1][i]), __builtin_amdgcn_exp2f(st[g >> 1][i + 1]));
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
      for (int m = 0; m < MT; ++m) o[m] = mfma32<false>(vf[g & 1][m], w[g & 1], o[m]);
      rest = mfma32<false>(vf[g & 1][MT], w[g & 1], rest);
      if (g + 1 < GROUPS) {
        __builtin_amdgcn_sched_group_barrier(0x100, MT + 1, 0);  // LDS reads
#pragma unroll
        for (int m = 0; m < MT + 1; ++m) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);               // a matrix operation
          __builtin_amdgcn_sched_group_barrier(0x402, (16 + MT) / (MT + 1), 0);  // vector operations
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Results leave by LDS, 32 dimensions at a time, each wave for its own rows.
  const float sum = __shfl(rest[4], n);
  const float inv = row.lo < row.hi ? 1 / sum : 0.f;
  __syncthreads();
  const bool any_bad = s_bad != 0;
  float* so = reinterpret_cast<float*>(lds) + wave * 32 * LDO;
  const Row mine = row_of(p, r0 + (lane >> 1), span, hk);
  // Rare: NaN in dimensions 32 m on for the groups left out above, to the rows that see them.
  auto add_left_out = [&](int m) {
    const int g = 32 * m / GS;
    for (int step = t0; step < t1; ++step) {
      const uint32_t here = token_block(step, lane & (BLOCKS - 1));
      for (int j = 0; j < BN; ++j) {
        const uint16_t* params = reinterpret_cast<const uint16_t*>(v_cache + (size_t)__shfl(here, j >> 3) * BLOCK + 4 * D) + g * 16 + (j & 7);
        if (step * BN + j < row.lo || step * BN + j >= row.hi) continue;
        if (not_finite<false>(params[0]) || not_finite<false>(params[8]))
          for (int d = kg; d < 32; d += 2) so[n * LDO + d] = NAN;
      }
    }
  };
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int g = 32 * m / GS;
    const float middle = __shfl(rest[g & 3], (g >> 2) * 32 + n) * inv;
#pragma unroll
    for (int y = 0; y < 4; ++y)
      *reinterpret_cast<f32x4*>(so + n * LDO + 8 * y + 4 * kg) =
          f32x4{fmaf(o[m][4 * y], inv, middle), fmaf(o[m][4 * y + 1], inv, middle), fmaf(o[m][4 * y + 2], inv, middle),
                fmaf(o[m][4 * y + 3], inv, middle)};
    if (any_bad) add_left_out(m);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (mine.token >= 0) {
      const float* src = so + (lane >> 1) * LDO + 16 * (lane & 1);
      uint16_t* dst = a.out + ((long long)mine.token * a.Hq + mine.head) * D + 32 * m + 16 * (lane & 1);
#pragma unroll
      for (int e = 0; e < 16; e += 8) {
        u32x4 v;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          v[x] = t.bf16 ? pack_pair<true>(src[e + 2 * x], src[e + 2 * x + 1]) : pack_pair<false>(src[e + 2 * x], src[e + 2 * x + 1]);
        *reinterpret_cast<u32x4*>(dst + e) = v;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <int D, int G>
hipError_t launch_tiles_of(const Kv4TileArgs& t, hipStream_t stream) {
  const AttentionArgs& a = t.a;
  const int group = a.Hq / a.Hkv, rtiles = row_tiles(a.max_q, group, kKv4TileRows<D>);
  const Kv4TileKernelArgs p = {{a, fixed_div(a.page_size), fixed_div(group), group, rtiles, 1, nullptr, nullptr, nullptr}, t.bf16};
  const dim3 grid((unsigned)tile_blocks(a.B, a.Hkv, rtiles));
  const auto run = [&](auto kernel) { kernel<<<grid, 64 * kKv4TileWaves<D>, 0, stream>>>(p); };
  const Cap cap = cap_kind(a.softcap);
  if (a.slopes || cap == kAnyCap) run(kv4_tile_kernel<D, G, kAnyScore>);
  else if (cap == kSmallCap) run(kv4_tile_kernel<D, G, kCappedScore>);
  else run(kv4_tile_kernel<D, G, kPlainScore>);
  return hipGetLastError();
}

}  // namespace
}  // namespace qmm
