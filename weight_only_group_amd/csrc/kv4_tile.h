// Attention to the 4-bit cache for prompts: blocks of many rows, whose keys and values
// are decoded once into LDS.
//
// A block has 256 rows (128 where D is 256), 32 a wave, and takes 64 keys a step (32). While a wave has its matrix
// operations in hand (the step before's values, the step's keys; 32x32x16, keys and channels in the rows, the wave's
// queries in the columns, so that a softmax is two lanes' affair) it decodes its part of the next step's keys and values
// between them; the other wave of its SIMD, a phase behind, takes its softmax meanwhile.
// Bound by the vector ALUs: a prompt of 8192 with a cap (32 heads of 128 over 8) takes 737 us, 746 TFLOP/s (the first
// thirty after a pause up to 970: the clock settles), with the vector ALUs busy 67% of the cycles (of a score two
// exponentials and a reciprocal, each as long as two other operations) and the matrix cores 39%. The 16-bit cache's kernel
// takes 690 to 750 us for it.
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

// (lambdas that hold registers by reference: left as calls they would put them to memory)
#define QMM_INLINE __attribute__((always_inline))

// How a score follows from its product: a factor; a small cap; a factor and a distance bias; any cap and a
// bias. (Apart, as branches between them in a step make the compiler spill hundreds of registers.)
enum ScoreKind { kPlainScore, kCappedScore, kBiasedScore, kAnyScore };

// f of 0, 1, ... N - 1 as compile-time constants.
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

struct Kv4TileKernelArgs {
  AttnKernelArgs r;
  bool bf16;
};

// Block: 32 rows a wave of one key head, all their keys in steps of BN. Step s has two phases, each ended by a barrier (meet):
//   products   V^T p^T of step s - 1, then K q^T of s; between them each wave decodes its own part of the keys and values of
//              step s + 1, from words asked for a step before, and asks for those of s + 2
//   softmax    of step s: the weights p stay in registers for the next products
// Of eight waves those of the second half are a phase behind (one barrier more ahead of the loop, one less behind it), so that
// a SIMD has one wave in each phase; four waves, one a SIMD, go together.
// Buffers in LDS: keys of s are read in the products of s, while s + 1 is written: two, by the parity of the step. Values of s
// are written in the products of s - 1 and read in those of s + 1, so that three steps' are there at a time: s - 1 read, s
// whole or (by the half behind) still being written, s + 1 written. A buffer is written anew two (three) steps later, one barrier at
// least after the half behind has read it.
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
  constexpr int THREADS = 64 * WAVES, KW = BN * D / 8 / THREADS;  // words of keys a thread decodes
  constexpr int QUADS = D / 4, UNITS = 2 * BLOCKS * QUADS;       // of values: four tokens of four channels
  constexpr int VU = (UNITS + THREADS - 1) / THREADS;            // of a thread
  // Two buffers of keys, each with its keys' middles; three of values, each with rows of middles: the groups', one of ones,
  // one of zeros.
  constexpr int TILE = BN * D * 2, K_BUFFER = TILE + BN * 16, VM_ROW = BN * 2, V_BUFFER = TILE + ((G + 2) * VM_ROW + 511) / 512 * 512;
  constexpr int LDO = 36, OUT_BYTES = ROWS * LDO * 4, KV_BYTES = 2 * K_BUFFER + 3 * V_BUFFER;
  __shared__ __attribute__((aligned(16))) uint8_t lds[KV_BYTES > OUT_BYTES ? KV_BYTES : OUT_BYTES];
  constexpr int V_LDS = 2 * K_BUFFER;  // place of the first of them
  __shared__ int range[4][WAVES], s_bad;
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
  if (KIND == kAnyScore) rule.scale = kLog2e * a.scale;  // (a small cap's has another factor)

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
  if (lane == 0) range[0][wave] = lo, range[1][wave] = hi, range[2][wave] = all_lo, range[3][wave] = all_hi;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  int block_lo = INT32_MAX, block_hi = 0, block_all_lo = 0, block_all_hi = INT32_MAX;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    block_lo = min(block_lo, range[0][w]), block_hi = max(block_hi, range[1][w]);
    block_all_lo = max(block_all_lo, range[2][w]), block_all_hi = min(block_all_hi, range[3][w]);
  }
  block_lo = __builtin_amdgcn_readfirstlane(block_lo);
  block_hi = __builtin_amdgcn_readfirstlane(block_hi);
  block_all_lo = __builtin_amdgcn_readfirstlane(block_all_lo);
  block_all_hi = __builtin_amdgcn_readfirstlane(block_all_hi);
  const int t0 = block_lo < block_hi ? block_lo / BN : 0, t1 = block_lo < block_hi ? (block_hi - 1) / BN + 1 : 0;

  // The row's query, and its groups' sums in two parts (one a lane group): 2^-22 of a sum off, as four roundings of its product in fp32.
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
  const int32_t* table = a.page_table + (long long)b * a.table_stride;
  // Number of the block of eight tokens, i in the step; past the seen keys' ends the nearest.
  auto token_block = [&](int step, int i) QMM_INLINE -> uint32_t {
    const int j = (int)min(max((uint32_t)step * BN + 8 * i, (uint32_t)block_lo), (uint32_t)block_hi - 1);
    const int at = p.by_page(j);
    const int page = min(max(table[at], 0), a.pages - 1);
    return (((uint32_t)page * a.Hkv + hk) * a.page_size + (j - at * a.page_size)) / kBlockTokens;
  };
  // A thread's part of a step: KW neighbouring words of a key, and of the values units: words of four
  // tokens (of a block's halves) of a quad of channels, with their scales and middles.
  constexpr int PER_KEY = D / 8 / KW;  // threads of a key
  const int key = tid / PER_KEY, word0 = tid % PER_KEY * KW;
  auto unit_of = [&](int i) QMM_INLINE { return (tid + i * THREADS) % UNITS; };
  // (of sixteen neighbouring pairs of threads eight quads of two blocks)
  auto quad_of = [&](int i) QMM_INLINE { return (unit_of(i) >> 1 & 7) | unit_of(i) / (16 * BLOCKS) << 3; };
  auto blk_of = [&](int i) QMM_INLINE { return (unit_of(i) >> 4) % BLOCKS; };
  const bool no_values = UNITS < THREADS && tid >= UNITS;
  uint32_t kw[KW], kp[G], vw[VU][2], vs[VU][2], vm[VU][2], k_block, v_block[VU];  // blocks: of the next load
  auto find = [&](int step) QMM_INLINE {
    k_block = token_block(step, key / 8);
#pragma unroll
    for (int i = 0; i < VU; ++i) v_block[i] = token_block(step, blk_of(i));
  };
  auto load = [&]() QMM_INLINE {
    const uint8_t* src = k_cache + (size_t)k_block * BLOCK;
    load_words<4 * KW>(kw, src + (key & 7) * (D / 2) + word0 * 4);
    load_words<4 * G>(kp, src + 4 * D + (key & 7) * 4 * G);
#pragma unroll
    for (int i = 0; i < VU; ++i) {
      const int half = unit_of(i) & 1, quad = quad_of(i);
      const uint8_t* from = v_cache + (size_t)v_block[i] * BLOCK + half * 8;
      load_words<8>(vw[i], from + quad * 16);
      load_words<8>(vs[i], from + 4 * D + quad * 4 / GS * 32);
      load_words<8>(vm[i], from + 4 * D + quad * 4 / GS * 32 + 16);
    }
  };
  // Byte offsets in the buffer of piece (eight channels) `piece` of a key, and of block blk of a channel.
  auto key_place = [](int k, int piece) {
    const int turn = D == 64 ? (k >> 1 & 1) << 2 | (k >> 2 & 3) : (k & 3) << 2 | (k >> 2 & 3);
    return k * (2 * D) + (piece ^ turn) * 16;
  };
  auto value_place = [](int c, int blk) {
    if constexpr (BN == 32) return (c >> 2) * 256 + (((c & 3) ^ (c >> 4 & 1)) * 4 + (blk ^ (c >> 2 & 3))) * 16;
    else return (c >> 1) * 256 + (((c ^ c >> 4) & 1) * 8 + (blk ^ (c >> 1 & 7))) * 16;
  };
  auto seen_by_whole_block = [&](int step) {
    return (uint32_t)step * BN >= (uint32_t)block_all_lo && (uint32_t)(step + 1) * BN <= (uint32_t)block_all_hi;
  };
  // Before the decoding. Tokens that no row sees may hold anything: their scales and middles count as 0. So
  // do those of a seen one that stands for NaN, as they must not reach the rows that do not see it (0 times NaN
  // is NaN); those that do get a NaN at the end.
  auto clean = [&](int step) QMM_INLINE {
    if (seen_by_whole_block(step)) return;
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < VU; ++i) {
      const uint32_t j0 = (uint32_t)step * BN + 8 * blk_of(i) + 4 * (unit_of(i) & 1);  // (a step asked for ahead may begin at 2^31)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t j = j0 + 2 * x, lo = block_lo, hi = block_hi;
        const uint32_t in = (j >= lo && j < hi ? 0xFFFFu : 0u) | (j + 1 >= lo && j + 1 < hi ? 0xFFFF0000u : 0u);
        const uint32_t nan = (bad_scales(vs[i][x]) | bad_middles(vm[i][x])) & in;
        bad |= nan;
        vs[i][x] &= in & ~nan;
        vm[i][x] &= in & ~nan;
      }
    }
    if (bad) s_bad = 1;
  };
  // The middles (apart from the slices, which are to be without branches).
  auto put_middles = [&](int k_to, int v_to) QMM_INLINE {
    if (word0 == 0) {
      u32x4 middles = {0, 0, 0, 0};
      if constexpr (G == 1) {
        middles[0] = middles_or_nan(kp[0] >> 16, kp[0] & 0xFFFF);
      } else {
#pragma unroll
        for (int x = 0; x < G / 2; ++x) middles[x] = middles_or_nan(kp[G / 2 + x], kp[x]);
      }
      *reinterpret_cast<u32x4*>(lds + k_to + TILE + key * 16) = middles;
    }
#pragma unroll
    for (int i = 0; i < VU; ++i)
      if (quad_of(i) * 4 % GS == 0 && !no_values)
        *reinterpret_cast<u32x2*>(lds + v_to + TILE + quad_of(i) * 4 / GS * VM_ROW + blk_of(i) * 16 + (unit_of(i) & 1) * 8) = u32x2{middles_or_nan(vm[i][0], vs[i][0]), middles_or_nan(vm[i][1], vs[i][1])};
  };
  // The decoding in slices: the key's words, then four channels of each unit.
  constexpr int SLICES = KW + 4 * VU;
  const int key_at = key_place(key, 4 * (word0 % (D / 32)) + word0 / (D / 32));
  int unit_at[VU];
#pragma unroll
  for (int i = 0; i < VU; ++i) unit_at[i] = value_place(4 * quad_of(i), blk_of(i)) + (unit_of(i) & 1) * 8;
  auto decode_slice = [&](int k_to, int v_to, auto slice) QMM_INLINE {
    constexpr int I = decltype(slice)::value;
    if constexpr (I < KW) {
      const int g = (word0 + I) % (D / 32) * 32 / GS;
      uint32_t pair = kp[0];
      if constexpr (G > 2) {
#pragma unroll
        for (int x = 1; x < G / 2; ++x) pair = g / 2 == x ? kp[x] : pair;
      }
      const f16 sg = G == 1 ? as_f16x2(pair)[0] : g % 2 ? as_f16x2(pair)[1] : as_f16x2(pair)[0];
      const f16x2 s2 = {sg, sg}, c2 = times_24(s2);
      // (the places of a thread's pieces differ in bits that the buffers' places leave 0)
      *reinterpret_cast<u32x4*>(lds + ((k_to + key_at) ^ I * 64)) =
          u32x4{decode<0>(kw[I], s2, c2, masks), decode<1>(kw[I], s2, c2, masks), decode<2>(kw[I], s2, c2, masks), decode<3>(kw[I], s2, c2, masks)};
    } else {
      constexpr int U = (I - KW) / 4, R = (I - KW) % 4;
      u32x2 v;
#pragma unroll
      for (int x = 0; x < 2; ++x) v[x] = decode<R>(vw[U][x], as_f16x2(vs[U][x]), times_24(as_f16x2(vs[U][x])), masks);
      constexpr int there = BN == 32 ? R * 64 : (R & 1) * 128 | (R >> 1) * (256 | 16);
      if (UNITS >= THREADS || !no_values) *reinterpret_cast<u32x2*>(lds + ((v_to + unit_at[U]) ^ there)) = v;
    }
  };

  // ---- products -------------------------------------------------------------------------
  auto seen_by_all = [&](int key0) { return key0 >= all_lo && (uint32_t)key0 + BN <= (uint32_t)all_hi; };
  const int my_key = (n & 19) | (n & 4) << 1 | (n & 8) >> 1;  // of the 32 of row n: bits 2 and 3 change places
  const int k_at = key_place(my_key, kg);  // (two pieces on: an exclusive or with 32)
  const int v_at = value_place(n, kg);  // (two blocks on: an exclusive or with 32; 32 channels on: the same place, 64 BN further)

  const int my_middles = TILE + (n < G ? n : n == 8 ? G : G + 1) * VM_ROW + kg * 16;
  for (int i = tid; i < 3 * V_BUFFER / 16; i += THREADS) {  // the rows of ones and zeros; values of 0 in all, for the weights of 0 ahead of the first step
    const int at = i * 16 % V_BUFFER - TILE - G * VM_ROW;
    const uint32_t x = at >= 0 && at < VM_ROW ? kOnes : 0u;
    reinterpret_cast<u32x4*>(lds + V_LDS)[i] = u32x4{x, x, x, x};
  }
  __syncthreads();

  f32x16 o[MT] = {}, rest = {};  // rest: rows g < 8 the sums of p m_g, row 8 the sum of p
  float mx = -INFINITY;
  u32x4 w[BN / 16] = {};  // the weights of the step before, sixteen keys a piece
  // A step's matrix operations: the step before's weights times its values, sixteen keys (MT products and one for the
  // middles) after another; then the step's keys, their middles first, times the queries. Their left operands come from LDS
  // AHEAD operations before. (A prompt of 8192, 32 heads of 128 over 8: with 3 859 us, side by side with 5 762, with 7 784 and with 9
  // 779: there is no room for their registers.)
  constexpr int GROUPS = BN / 16, VALUE_OPS = GROUPS * (MT + 1), OPS = VALUE_OPS + SUB * (STEPS + 1), AHEAD = 5;
  f32x16 st[SUB];
  u32x4 operand[AHEAD + 1];
  auto read = [&](int vb, int kb, auto op) QMM_INLINE {
    constexpr int I = decltype(op)::value;
    int from;
    if constexpr (I < VALUE_OPS) {
      constexpr int g = I / (MT + 1), m = I % (MT + 1);
      from = m < MT ? ((vb + v_at) ^ g * 32) + m * (64 * BN) : vb + my_middles + g * 32;
    } else if constexpr (I < VALUE_OPS + SUB) {
      from = kb + TILE + (32 * (I - VALUE_OPS) + my_key) * 16;
    } else {
      constexpr int s = (I - VALUE_OPS - SUB) / SUB, u = (I - VALUE_OPS - SUB) % SUB;
      from = ((kb + k_at) ^ s * 32) + u * (64 * D);
    }
    operand[I % (AHEAD + 1)] = *reinterpret_cast<const u32x4*>(lds + from);
  };
  auto multiply = [&](auto op) QMM_INLINE {
    constexpr int I = decltype(op)::value;
    const u32x4 x = operand[I % (AHEAD + 1)];
    if constexpr (I < VALUE_OPS) {
      constexpr int g = I / (MT + 1), m = I % (MT + 1);
      if constexpr (m < MT) o[m] = mfma32<false>(x, w[g], o[m]);
      else rest = mfma32<false>(x, w[g], rest);
    } else if constexpr (I < VALUE_OPS + SUB) {
      st[I - VALUE_OPS] = mfma32<false>(x, qsum, f32x16{});
    } else {
      constexpr int s = (I - VALUE_OPS - SUB) / SUB, u = (I - VALUE_OPS - SUB) % SUB;
      st[u] = mfma32<false>(x, q[s], st[u]);
    }
  };
  // Everything that a wave has put to LDS is there, for all. (A fence would wait for the loads asked for ahead too.)
  auto meet = [&]() QMM_INLINE {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // Two waves share a SIMD: while one takes its matrix operations (the step before's values, the
  // step's keys), the other takes its softmax. The second half of the waves is a phase behind.
  const bool behind = WAVES == 8 && wave >= 4;
  if (t0 < t1) {
    find(t0);
    load();
    find(t0 + 1);
    clean(t0);
    put_middles((t0 & 1) * K_BUFFER, V_LDS + V_BUFFER);
    each<SLICES>([&](auto i) QMM_INLINE { decode_slice((t0 & 1) * K_BUFFER, V_LDS + V_BUFFER, i); });
    load();
    find(t0 + 2);
    meet();
    if (behind) meet();
  }
  int v_last = 0, v_next = 2;  // buffers of the values of the step before and of the one after (the step's own is the third)
  for (int step = t0; step < t1; ++step) {
    const int key0 = step * BN;
    const int ks = (step & 1) * K_BUFFER, vb = V_LDS + v_last * V_BUFFER;
    // The next step's decoding goes between the matrix operations. (of the steps asked for ahead those past the last are
    // decoded too, to buffers that are not read)
    const int k_to = (~step & 1) * K_BUFFER, v_to = V_LDS + v_next * V_BUFFER;
    each<AHEAD>([&](auto op) QMM_INLINE { read(vb, ks, op); });
    clean(step + 1);
    put_middles(k_to, v_to);
    auto slices = [&](auto i, auto all) QMM_INLINE {  // those of place i of all
      constexpr int from = decltype(i)::value * SLICES / decltype(all)::value, to = (decltype(i)::value + 1) * SLICES / decltype(all)::value;
      each<to - from>([&](auto x) QMM_INLINE { decode_slice(k_to, v_to, std::integral_constant<int, from + decltype(x)::value>{}); });
    };
    each<OPS>([&](auto op) QMM_INLINE {
      constexpr int I = decltype(op)::value;
      if constexpr (I + AHEAD < OPS) read(vb, ks, std::integral_constant<int, I + AHEAD>{});
      __builtin_amdgcn_sched_barrier(0);
      multiply(op);
      slices(op, std::integral_constant<int, OPS>{});
    });
    load();
    find(step + 3);
    meet();
    // The softmax (with weights of 0 where the wave's rows see none of the step's keys).
    const bool whole = seen_by_all(key0);
    auto key_of = [&](int u, int i) { return key0 + 32 * u + 16 * (i >> 3) + 8 * kg + (i & 7); };
    // The largest score of the row; where a score is more than a multiply-add or a small cap of its
    // product the scores are taken first, else only that of the largest product.
    float best = -INFINITY;
    uint32_t seen = ~0u;  // bit 16 u + i: the row sees key_of(u, i)
    if (KIND >= kBiasedScore) {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          st[u][i] = rule.template score<KIND == kAnyScore ? kAnyCap : kNoCap, true>(st[u][i], row.pos, key_of(u, i));
          if (KIND == kAnyScore && i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // (or the registers do not suffice)
        }
    }
    if (!whole) {
      asm volatile("");  // (keeps the masks of whole steps from being computed along)
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
    if (KIND >= kBiasedScore) {
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
      asm volatile("");
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) st[u][i] = seen >> (16 * u + i) & 1 ? st[u][i] : -INFINITY;
    }
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = 8 * (g & 1) + 2 * x;
        w[g][x] = pack_pair<false>(__builtin_amdgcn_exp2f(st[g >> 1][i]), __builtin_amdgcn_exp2f(st[g >> 1][i + 1]));
      }
    v_last = v_last == 2 ? 0 : v_last + 1;
    v_next = v_next == 2 ? 0 : v_next + 1;
    meet();
  }
  if (t0 < t1) {
    if (WAVES == 8 && !behind) meet();
    const int vb = V_LDS + v_last * V_BUFFER;
    each<AHEAD>([&](auto op) QMM_INLINE { read(vb, 0, op); });
    each<VALUE_OPS>([&](auto op) QMM_INLINE {
      constexpr int I = decltype(op)::value;
      if constexpr (I + AHEAD < VALUE_OPS) read(vb, 0, std::integral_constant<int, I + AHEAD>{});
      multiply(op);
    });
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
        if (bad_scale(params[0]) || bad_middle(params[8]))
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
  if (cap == kAnyCap || (a.slopes && cap == kSmallCap)) run(kv4_tile_kernel<D, G, kAnyScore>);
  else if (a.slopes) run(kv4_tile_kernel<D, G, kBiasedScore>);
  else if (cap == kSmallCap) run(kv4_tile_kernel<D, G, kCappedScore>);
  else run(kv4_tile_kernel<D, G, kPlainScore>);
  return hipGetLastError();
}

}  // namespace
}  // namespace qmm
