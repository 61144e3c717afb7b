// Attention of new tokens to their sequences' cache in 4 bits: single tokens and few rows.
#include <algorithm>
#include <type_traits>

#include "kv4_attention.h"
#include "kv4_tile.h"

namespace qmm {
namespace {

// Lane exchanges within rows of sixteen: a value of the lane R to the right (round the
// row; or, of lanes past its end, anything).
template <int R>
__device__ __forceinline__ float rotated(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + 16 - R, 0xF, 0xF, true));
}
template <int R>
__device__ __forceinline__ uint32_t shifted(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x100 + R, 0xF, 0xF, true);
}
// Of the row's first four lanes a, b, c and d, side by side.
__device__ __forceinline__ float spread(float a, float b, float c, float d) {
  int v = __builtin_bit_cast(int, a);
  v = __builtin_amdgcn_update_dpp(v, __builtin_bit_cast(int, b), 0x114, 0xF, 0x2, false);
  v = __builtin_amdgcn_update_dpp(v, __builtin_bit_cast(int, c), 0x118, 0xF, 0x4, false);
  v = __builtin_amdgcn_update_dpp(v, __builtin_bit_cast(int, d), 0x11C, 0xF, 0x8, false);
  return __builtin_bit_cast(float, v);
}
// Running sums over a wave's lanes.
template <int CTRL, int ROWS>
__device__ __forceinline__ int plus_dpp(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int running_sum(int v) {
  v = plus_dpp<0x111, 0xF>(v);
  v = plus_dpp<0x112, 0xF>(v);
  v = plus_dpp<0x114, 0xF>(v);
  v = plus_dpp<0x118, 0xF>(v);
  v = plus_dpp<0x142, 0xA>(v);  // a row's last lane to the next row
  return plus_dpp<0x143, 0xC>(v);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float plus_dpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float sum_of_wave(float v) {
  v = plus_dpp<0x111, 0xF>(v);
  v = plus_dpp<0x112, 0xF>(v);
  v = plus_dpp<0x114, 0xF>(v);
  v = plus_dpp<0x118, 0xF>(v);
  v = plus_dpp<0x142, 0xA>(v);
  v = plus_dpp<0x143, 0xC>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
// The least and the largest over a row's sixteen lanes, of integers.
template <int CTRL>
__device__ __forceinline__ int across(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ int least_of_row(int v) {
  v = min(v, across<0x128>(v));
  v = min(v, across<0x124>(v));
  v = min(v, across<0x122>(v));
  return min(v, across<0x121>(v));
}
__device__ __forceinline__ int largest_of_row(int v) {
  v = max(v, across<0x128>(v));
  v = max(v, across<0x124>(v));
  v = max(v, across<0x122>(v));
  return max(v, across<0x121>(v));
}
// The largest of the four rows' values.
__device__ __forceinline__ float max_of_rows(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

// How many parts the keys of each tile are split into, so that the parts are alike
// whatever the sequences' lengths, and so many as run at a time: a block's start and end
// take 10 us. With c chunks a part, sum ceil(chunks / c) is at most sum chunks / c + tiles, so c =
// sum chunks / parts gives no more blocks than parts + tiles; smaller ones are tried first.
// A sequence's chunks are those of its first and last query.
// One part each where that is faster: a share, its hand-over and the join cost 5 us and more a block, against the time of
// the longest tile alone. Measured, the time in parts over that without (profiles/cache_attention_choices.txt, means), single
// tokens: up to 16 tiles of D 64, 128 and 256 on 400 keys 1.57, 1.37 and 1.19, on 1000 1.20, 1.09 and 0.84, on 3000 0.66, 0.61
// and 0.48; 256 to 4096 tiles on less than four keys a tile 1.97 (one at 6.2), and where one sequence among short ones has eight keys a
// tile and more 0.43. Sequences of more than 128 rows are split up to kMostTiles tiles and from half as many keys on: their
// last ones see the most keys. A prompt of 3000 alone takes 0.57 of the time in parts, of 2000 0.71, of 1000 1.06; two
// to four of them 0.98 to 1.25, and prompts of 150 to 500, which are not split, would take 2.2 to 1.7.
// Of several tiles of a sequence a block then takes two, so that its keys and values are decoded once for both: 1.08 times as fast
// as one tile a block with 17 to 32 rows, 1.16 with 33 to 64, 1.05 with 65 to 128. D 256 has no registers for it (0.6).
constexpr int kMostSequences = 1024;  // of a split launch
constexpr int kMostTiles = 4096, kPartsFrom = 192 * 1024;  // keys, with D: 1536, 1024, 614
constexpr int kMostParts = 256;       // of a tile
constexpr int kLeastChunks = kWaves;  // of a part

// Blocks of a split launch that run at a time.
inline int resident_blocks(int D, DeviceTopo topo) { return topo.cus * (D == 64 ? 4 : D == 128 ? 3 : 2); }

struct Kv4Plan {
  int group, rtiles;
  int fit;    // blocks that run at a time
  int parts;  // parts beyond one a tile that there may be; 0: one a tile
  bool wide;  // a block takes two tiles
  long long blocks;
};
Kv4Plan kv4_plan(int B, int Hq, int Hkv, int D, int max_q, int max_kv, DeviceTopo topo) {
  Kv4Plan p;
  p.group = Hq / Hkv;
  p.rtiles = row_tiles(max_q, p.group, kRows);
  const long long tiles = (long long)B * Hkv * p.rtiles;
  p.fit = resident_blocks(D, topo);
  p.parts = 0;
  const long long rows = (long long)max_q * p.group;
  const bool prompts = rows > 8 * kRows;
  const bool worth_it = max_kv > kPartsFrom / (D + 64) / (prompts ? 2 : 1) && (prompts || max_kv > 4 * tiles);
  if (B <= kMostSequences && tiles <= kMostTiles && worth_it)
    p.parts = (int)std::max(p.fit - tiles, p.fit / 2ll);
  const long long most = ((long long)max_kv + kLeastChunks * kChunk - 1) / (kLeastChunks * kChunk);
  p.wide = rows > kRows && !p.parts && D <= 128;
  if (p.wide) p.rtiles = row_tiles(max_q, p.group, 2 * kRows);
  p.blocks = p.parts ? std::min(tiles + p.parts, tiles * most) : tile_blocks(B, Hkv, p.rtiles);
  return p;
}

struct Kv4KernelArgs {
  AttnKernelArgs r;
  int fit, parts;
  Cap cap;
  bool bf16;
};

// A block's share: part `part` of `parts` of tile (b, hk, rt); first: the block of
// the tile's part 0, step: blocks from part to part. b -1: none.
struct Share {
  int b, hk, rt, part, parts, first, step;
  Span span;
};

// n / d rounded up, 0 <= n < 2^27 (d's inverse given), for quotients below 2^20.
__device__ __forceinline__ int divided_up(int n, int d, float inverse) {
  int q = (int)((float)n * inverse);  // off by one at most
  q -= (long long)q * d > n;
  q += (long long)q * d < n;
  return q + ((long long)q * d < n);
}

struct Sequence {
  Span span;
  int tiles, chunks;  // tiles of all key heads
};
__device__ __forceinline__ Sequence sequence_of(const AttnKernelArgs& p, int b) {
  const AttentionArgs& a = p.a;
  Sequence s = {{0, 0, 0, 0}, 0, 0};
  if (b >= a.B) return s;
  s.span = span_of(a, b);
  s.tiles = max(row_tiles_of(s.span, p.group), 1) * a.Hkv;
  if (s.span.q1 == s.span.q0) return s;
  int lo = 0, hi = s.span.kv;
  if (a.first) lo = max(min(a.first[s.span.q0], a.first[s.span.q1 - 1]), 0);
  if (a.end) hi = min(max(a.end[s.span.q0], a.end[s.span.q1 - 1]), hi);
  s.chunks = lo < hi ? (hi - 1) / kChunk + 1 - lo / kChunk : 0;
  return s;
}

// Blocks: per sequence its parts, of each the key heads, of each the row tiles. Every wave finds the
// block's share by itself.
__device__ __forceinline__ Share share_of(const Kv4KernelArgs& p) {
  const AttentionArgs& a = p.r.a;
  const int lane = threadIdx.x & 63, id = blockIdx.x;
  const int per = (a.B + 63) / 64;  // neighbouring sequences of a lane
  Sequence own = sequence_of(p.r, lane * per);
  float work = (float)own.tiles * (float)own.chunks;
#pragma unroll 1
  for (int i = 1; i < per; ++i) {
    const Sequence s = sequence_of(p.r, lane * per + i);
    work += (float)s.tiles * (float)s.chunks;
  }
  work = sum_of_wave(work);
  // Chunks a part: from the fewest that fit on, as long as they make more blocks than run at a
  // time; after some tries those that surely make few enough. (a little more than the quotient: the
  // sums are rounded)
  int c = 0, parts = 0, blocks = 0;
  float inverse = 0, wanted = work / (float)p.fit;
  auto parts_of = [&](const Sequence& s) { return min(max(divided_up(s.chunks, c, inverse), 1), kMostParts); };
#pragma unroll 1
  for (int i = 0; i < 5; ++i) {
    if (i == 4) wanted = work / (float)p.parts;
    c = max((int)(wanted * 1.00001f) + 1, kLeastChunks);
    inverse = 1 / (float)c;
    parts = parts_of(own);
    blocks = parts * own.tiles;
#pragma unroll 1
    for (int i = 1; i < per; ++i) {
      const Sequence s = sequence_of(p.r, lane * per + i);
      blocks += parts_of(s) * s.tiles;
    }
    const int all = __builtin_amdgcn_readlane(running_sum(blocks), 63);
    if (all <= p.fit) break;
    wanted = (float)c * fmaxf((float)all / (float)p.fit, 1.03f);
  }
  int at = running_sum(blocks) - blocks, b = lane * per;
  const uint64_t here = __ballot(id >= at && id < at + blocks);
  Share r;
  r.b = -1;
  if (here == 0) return r;
#pragma unroll 1
  for (int i = 1; i < per && id >= at + parts * own.tiles; ++i) {  // (the lane found gets to its sequence)
    at += parts * own.tiles;
    own = sequence_of(p.r, ++b);
    parts = parts_of(own);
  }
  const int from = __builtin_ctzll(here);
  auto get = [&](int v) { return __builtin_amdgcn_readlane(v, from); };
  r.b = get(b);
  r.parts = get(parts);
  r.span = {get(own.span.q0), get(own.span.q1), get(own.span.kv), get(own.span.first)};
  const int off = id - get(at), rtiles = get(own.tiles) / a.Hkv;
  r.step = rtiles * a.Hkv;
  r.part = off / r.step;
  const int rest = off - r.part * r.step;
  r.hk = rest / rtiles;
  r.rt = rest - r.hk * rtiles;
  r.first = id - r.part * r.step;
  return r;
}

// What a tile's end needs to know of a row: where its result goes (the element's index; -1: no
// such row), and whether it sees a key.
struct RowEnd {
  long long at;
  int some;
};

// Joins a tile's parts: the block that arrives last. scratch: LDS of 16 D + 2 * kWaves * kRows floats.
// A wave takes every fourth part, four rows at a time.
template <int D, typename PACK>
__device__ __forceinline__ void join_parts(const Kv4KernelArgs& p, const Share& sh, const RowEnd* ends, int rows, float* scratch, PACK pack) {
  constexpr int E = D / 16, BATCH = 64 / E;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  float* red = scratch;             // (wave, E, lane)
  float* wave_ml = scratch + 16 * D;  // (wave, row): maximum, sum
  for (int r0 = 0; r0 < rows; r0 += 4) {
    // Lane: row r0 + lane / 16, E neighbouring dimensions; BATCH parts at a time.
    const int r = r0 + (lane >> 4);
    const bool live = r < rows;
    const int row = min(r, rows - 1);
    float m = -INFINITY, l = 0, o[E] = {};
    for (int q0 = wave; q0 < sh.parts; q0 += kWaves * BATCH) {
      FloatPair v[BATCH][E / 2], ml[BATCH];
#pragma unroll
      for (int y = 0; y < BATCH; ++y) {
        const int part = min(q0 + y * kWaves, sh.parts - 1);
        const size_t slot = (size_t)(sh.first + part * sh.step) * kRows;
        ml[y] = handoff_load_pair(p.r.part_ml + (slot + row) * 2);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) v[y][e] = handoff_load_pair(p.r.part + slot * D + (row * 16 + (lane & 15)) * 2 + 512 * e);
      }
      float n = m;
#pragma unroll
      for (int y = 0; y < BATCH; ++y) n = fmaxf(n, ml[y].a);
      const float off = n == -INFINITY ? 0.f : n, f = __builtin_amdgcn_exp2f(m - off);
      m = n;
      l *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
      for (int y = 0; y < BATCH; ++y) {
        if (q0 + y * kWaves >= sh.parts) break;  // (the last part again)
        const float w = __builtin_amdgcn_exp2f(ml[y].a - off);
        l += ml[y].b * w;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          o[2 * e] += v[y][e].a * w;
          o[2 * e + 1] += v[y][e].b * w;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) red[(wave * E + e) * 64 + lane] = o[e];
    if ((lane & 15) == 0) wave_ml[(wave * 4 + (lane >> 4)) * 2] = m, wave_ml[(wave * 4 + (lane >> 4)) * 2 + 1] = l;
    __syncthreads();
    constexpr int PER = E / 4 > 2 ? E / 4 : 2;  // dimensions a wave finishes
    if (live && wave * PER < E) {
      float f[kWaves], n = -INFINITY, sum = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) n = fmaxf(n, wave_ml[(w * 4 + (lane >> 4)) * 2]);
      const float off = n == -INFINITY ? 0.f : n;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        f[w] = __builtin_amdgcn_exp2f(wave_ml[(w * 4 + (lane >> 4)) * 2] - off);
        sum += wave_ml[(w * 4 + (lane >> 4)) * 2 + 1] * f[w];
      }
      const RowEnd end = ends[r];
      const float inv = end.some ? 1 / sum : 0.f;
      uint16_t* dst = p.r.a.out + end.at + (lane & 15) * E + wave * PER;
#pragma unroll
      for (int e = 0; e < PER; e += 2) {
        float x = 0, y = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          x += red[(w * E + wave * PER + e) * 64 + lane] * f[w];
          y += red[(w * E + wave * PER + e + 1) * 64 + lane] * f[w];
        }
        *reinterpret_cast<uint32_t*>(dst + e) = pack(x * inv, y * inv);
      }
    }
    __syncthreads();
  }
}

// Block: a tile of 16 rows (or RT of them), one part of its keys, in chunks of 32 keys a wave, as for the
// cache of 16-bit values. The products are K q^T and V^T p^T. Row i of a chunk's t-th
// sixteen is key 8 (i / 4) + 4 t + i % 4, so that a lane's scores are those of one block of
// eight tokens, whose values' words hold two tokens each: they need no exchange.
//
// No operand passes through LDS: a wave's 32 keys are read once, by the lanes that need them, and the next ones are
// asked for as the registers fall free. Few rows are bound by memory and by a block's start and end (the share of the work,
// page, keys; the join of the parts: 10 us together): 48 decodes of 128 to 8192 keys (32 heads of 128 over 8, 92 MB) 29 us,
// three on up to 131071 (157 MB) 42 us, 3.7 TB/s; one on 1500 keys 11 us, all of it latency. Tiles of sixteen rows are bound by
// the vector ALUs, 77% busy over documents of 24 heads of 64 (49 us): codes are decoded again in each. Two tiles a block: 47.5 us.
//
// RT: tiles of a block, one behind another (a wave's operands serve both); with parts one.
//
// NARROW: no more than four rows (one token of up to four heads a key head). Twelve of
// a product's sixteen columns are then free: the scores of the eight keys of a lane are spread
// over them, two a lane, for the softmax.
template <int D, int G, bool NARROW, int RT>
__global__ void __launch_bounds__(256, D == 256 || (D == 128 && RT == 2) ? 2 : 3) kv4_split_kernel(Kv4KernelArgs k) {
  constexpr int STEPS = D / 32, U = D / 64, GS = D / G, BLOCK = kv4_block_bytes(D, G);
  constexpr int NS = GS == 32 ? U : G;  // sets of scales that a lane needs for its values
  constexpr int LD = D + 4;
  __shared__ __attribute__((aligned(16))) float shared[kWaves * kRows * (LD + 2)];  // (the join of parts needs less)
  __shared__ RowEnd ends[kRows];
  __shared__ int s_last;
  float (*so)[kRows][LD] = reinterpret_cast<float (*)[kRows][LD]>(shared);
  float (*sml)[kRows][2] = reinterpret_cast<float (*)[kRows][2]>(shared + kWaves * kRows * LD);
  const AttnKernelArgs& p = k.r;
  const AttentionArgs& a = p.a;
  const bool bf16_data = k.bf16;
  const uint8_t* k_cache = reinterpret_cast<const uint8_t*>(a.k_cache);
  const uint8_t* v_cache = reinterpret_cast<const uint8_t*>(a.v_cache);
  Share share;
  if (RT == 1 && k.parts) {
    share = share_of(k);
    if (share.b < 0) return;
  } else {
    // Blocks of the row tiles that read the same keys follow each other on one XCD.
    const int per = 8 * p.rtiles, w8 = blockIdx.x % per, unit = blockIdx.x / per * 8 + w8 % 8;
    if (unit >= a.B * a.Hkv) return;
    share = {unit / a.Hkv, unit % a.Hkv, w8 / 8, 0, 1, 0, 0, span_of(a, unit / a.Hkv)};
  }
  const int b = share.b, hk = share.hk, rt = share.rt;
  const Span span = share.span;
  const int rtiles = max((row_tiles_of(span, p.group) + RT - 1) / RT, 1);
  zero_rest<D>(p, span, b, hk, rt * share.parts + share.part, rtiles * share.parts);
  const int rows_left = (span.q1 - span.q0) * p.group - rt * RT * kRows;
  if (rows_left <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, kg = lane >> 4;
  Row row[RT];
  ScoreRule rule[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    row[r] = row_of(p, (rt * RT + r) * kRows + (NARROW ? n & 3 : n), span, hk);
    rule[r] = score_rule(a, row[r].head);
  }

  // The keys that any row sees, and those that all see (rows past the last count as seeing all).
  int lo = INT32_MAX, hi = 0, all_lo = 0, all_hi = INT32_MAX;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (row[r].lo < row[r].hi) lo = min(lo, row[r].lo), hi = max(hi, row[r].hi);
    if (row[r].token >= 0) all_lo = max(all_lo, row[r].lo), all_hi = min(all_hi, row[r].hi);
  }
  lo = __builtin_amdgcn_readfirstlane(least_of_row(lo));
  hi = __builtin_amdgcn_readfirstlane(largest_of_row(hi));
  all_lo = __builtin_amdgcn_readfirstlane(largest_of_row(all_lo));
  all_hi = __builtin_amdgcn_readfirstlane(least_of_row(all_hi));
  auto seen_by_all = [&](int c) { return c * kChunk >= all_lo && (uint32_t)(c + 1) * kChunk <= (uint32_t)all_hi; };
  const int c_first = lo < hi ? lo / kChunk : 0, chunks = lo < hi ? (hi - 1) / kChunk + 1 - c_first : 0;
  const int c0 = c_first + (int)((long long)chunks * share.part / share.parts), c1 = c_first + (int)((long long)chunks * (share.part + 1) / share.parts);

  // The row's query, asked for ahead of the keys that its use waits for too.
  u32x4 q[RT][STEPS];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      q[r][s] = row[r].token < 0 ? u32x4{0, 0, 0, 0}
                                 : *reinterpret_cast<const u32x4*>(a.q + row[r].token * a.q_stride + (long long)row[r].head * D + s * 32 + kg * 8);

  // Number of the block of eight tokens that holds tokens 8 (lane & 3) on of a chunk; past
  // the seen keys' ends the nearest.
  const int32_t* table = a.page_table + (long long)b * a.table_stride;
  auto token_block = [&](int c) -> uint32_t {  // (the chunks asked for ahead may lie past 2^31)
    const int j = (int)min(max((uint32_t)c * kChunk + 8 * (lane & 3), (uint32_t)lo), (uint32_t)hi - 1);
    const int at = p.by_page(j);
    const int page = min(max(table[at], 0), a.pages - 1);
    return (((uint32_t)page * a.Hkv + hk) * a.page_size + (j - at * a.page_size)) / kBlockTokens;
  };
  uint32_t kw[2][STEPS], kp[2][G];  // a key's words and its scales and middles
  u32x4 vw[U], vs[NS], vm;          // eight tokens' words, scales and middles
  const uint8_t* kbase = k_cache + (n & 3) * (D / 2) + kg * (D / 8);
  const uint8_t* kparams = k_cache + 4 * D + (n & 3) * 4 * G;
  auto load_k = [&](uint32_t blocks) {
    const size_t at = (size_t)__shfl(blocks, n >> 2) * BLOCK;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      load_words<D / 8>(kw[t], kbase + at + t * (2 * D));
      load_words<4 * G>(kp[t], kparams + at + t * (16 * G));
    }
  };
  const uint8_t* vbase = v_cache + n * 16;
  const uint8_t* vscales = v_cache + 4 * D + (GS == 32 ? n >> 3 : 0) * 32;
  const uint8_t* vmiddles = v_cache + 4 * D + min(n, G - 1) * 32 + 16;
  auto load_v = [&](uint32_t blocks) {
    const size_t at = (size_t)__shfl(blocks, kg) * BLOCK;
#pragma unroll
    for (int u = 0; u < U; ++u) vw[u] = *reinterpret_cast<const u32x4*>(vbase + at + u * 256);
#pragma unroll
    for (int i = 0; i < NS; ++i) vs[i] = *reinterpret_cast<const u32x4*>(vscales + at + i * (GS == 32 ? 64 : 32));
    vm = *reinterpret_cast<const u32x4*>(vmiddles + at);
  };

  uint32_t blocks = 0, blocks_next = 0;
  int c = c0 + wave;
  if (c < c1) {
    blocks = token_block(c);
    load_k(blocks);
    load_v(blocks);
    blocks_next = token_block(c + kWaves);
  }

  // The row's query in fp16, and its groups' sums in three parts (lane group 0: the first, ...).
  u32x4 qsum[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float back = scale_query<4>(q[r], bf16_data);
    rule[r].scale = fminf(fmaxf(rule[r].scale * back, -3e38f), 3e38f);
    rule[r].inverse = fminf(fmaxf(rule[r].inverse * back, -3e38f), 3e38f);
    f16 part_of[8] = {};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      f32x4 sums = {};  // in every lane of a column
#pragma unroll
      for (int s = g * GS / 32; s < (g + 1) * GS / 32; ++s) sums = mfma16<false>(u32x4{kOnes, kOnes, kOnes, kOnes}, q[r][s], sums);
      const float s = sums[0];
      const f16 first = (f16)s, second = (f16)(s - (float)first), third = (f16)(s - (float)first - (float)second);
      part_of[g] = kg == 0 ? first : kg == 1 ? second : kg == 2 ? third : (f16)0.f;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) qsum[r][x] = as_u32(f16x2{part_of[2 * x], part_of[2 * x + 1]});
  }

  const DecodeMasks masks;
  f32x4 acc[RT][U][4] = {}, rest[RT] = {};  // rest: rows g the sums of p m_g, row 15 the sum of p
  float mx[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) mx[r] = -INFINITY;
  bool any_bad = false;
  // One chunk; with MORE the next one's loads go out as the registers fall free.
  auto step = [&](int c, auto more) {
    constexpr bool MORE = decltype(more)::value;
    f32x4 st[RT][2] = {};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      // Halves [s of all groups][m of all groups].
      u32x4 middles = {0, 0, 0, 0};
      if constexpr (G == 1) {
        middles[0] = middles_or_nan(kp[t][0] >> 16, kp[t][0] & 0xFFFF);
      } else {
#pragma unroll
        for (int x = 0; x < G / 2; ++x) middles[x] = middles_or_nan(kp[t][G / 2 + x], kp[t][x]);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) st[r][t] = mfma16<false>(middles, qsum[r], st[r][t]);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int g = s * 32 / GS;
        const uint32_t pair = kp[t][g / 2];
        const f16 sg = as_f16x2(pair)[g % 2];
        const f16x2 ss = {sg, sg}, c24 = times_24(ss);
        const uint32_t w = kw[t][s];
        const u32x4 keys = {decode<0>(w, ss, c24, masks), decode<1>(w, ss, c24, masks), decode<2>(w, ss, c24, masks), decode<3>(w, ss, c24, masks)};
#pragma unroll
        for (int r = 0; r < RT; ++r) st[r][t] = mfma16<false>(keys, q[r][s], st[r][t]);
      }
    }
    if constexpr (MORE) {
      // The page lookup before the keys: loads come back in order, and its block is computed with first.
      const uint32_t next = blocks_next;
      blocks_next = token_block(c + 2 * kWaves);
      blocks = next;
      __builtin_amdgcn_sched_barrier(0);  // the loads take the registers that the products above have read
      load_k(blocks);
      __builtin_amdgcn_sched_barrier(0);
    }
    // Scores: key j0 + x of the row.
    constexpr int NX = NARROW ? 2 : 8;
    const int j0 = c * kChunk + 8 * kg + (NARROW ? 2 * (n >> 2) : 0);
    const bool whole = seen_by_all(c);
    u32x4 w[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float s[NX], best = -INFINITY;
      if constexpr (NARROW) {
        s[0] = spread(st[r][0][0], st[r][0][2], st[r][1][0], st[r][1][2]);
        s[1] = spread(st[r][0][1], st[r][0][3], st[r][1][1], st[r][1][3]);
      } else {
#pragma unroll
        for (int x = 0; x < NX; ++x) s[x] = st[r][x >> 2][x & 3];
      }
      if (k.cap == kNoCap) {
#pragma unroll
        for (int x = 0; x < NX; ++x) s[x] = rule[r].template score<kNoCap, false>(s[x], 0, 0);
      } else if (k.cap == kSmallCap) {
#pragma unroll
        for (int x = 0; x < NX; ++x) s[x] = rule[r].template score<kSmallCap, false>(s[x], 0, 0);
      } else {
#pragma unroll
        for (int x = 0; x < NX; ++x) s[x] = rule[r].template score<kAnyCap, false>(s[x], 0, 0);
      }
      if (a.slopes) {
#pragma unroll
        for (int x = 0; x < NX; ++x) s[x] -= rule[r].slope * fabsf((float)(row[r].pos - (j0 + x)));
      }
      if (!whole) {
#pragma unroll
        for (int x = 0; x < NX; ++x) s[x] = j0 + x >= row[r].lo && j0 + x < row[r].hi ? s[x] : -INFINITY;
      }
#pragma unroll
      for (int x = 0; x < NX; ++x) best = fmaxf(best, s[x]);
      if (NARROW) {
        best = fmaxf(best, rotated<4>(best));
        best = fmaxf(best, rotated<8>(best));
      }
      best = max_of_rows(best);
      if (__any(best > mx[r] + kSlack)) {
        const float m = best > mx[r] + kSlack ? best : mx[r];
        const float f = mx[r] == m ? 1.f : __builtin_amdgcn_exp2f(mx[r] - m);
        rest[r] *= f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][u][i] *= f;
        mx[r] = m;
      }
      const float off = mx[r] == -INFINITY ? 0.f : mx[r] - kLift;
#pragma unroll
      for (int x = 0; x < NX / 2; ++x)
        w[r][x] = pack_pair<false>(__builtin_amdgcn_exp2f(s[2 * x] - off), __builtin_amdgcn_exp2f(s[2 * x + 1] - off));
      if constexpr (NARROW) {  // (what columns past the fourth get is in no result)
        w[r][1] = shifted<4>(w[r][0]);
        w[r][2] = shifted<8>(w[r][0]);
        w[r][3] = shifted<12>(w[r][0]);
      }
    }
    if (!whole) {
      // Places that no row sees may hold anything: their scales and middles count as 0. So do those
      // of a seen place that stands for NaN, as they must not reach the rows that do not see it (0
      // times NaN is NaN); those that do get a NaN after the loop.
      uint32_t bad = 0;
      auto clean = [&](u32x4& v, auto bad_of) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int j = c * kChunk + 8 * kg + 2 * x;
          const uint32_t in = (j >= lo && j < hi ? 0xFFFFu : 0u) | (j + 1 >= lo && j + 1 < hi ? 0xFFFF0000u : 0u);
          const uint32_t nan = bad_of(v[x]) & in;
          bad |= nan;
          v[x] &= in & ~nan;
        }
      };
#pragma unroll
      for (int i = 0; i < NS; ++i) clean(vs[i], bad_scales);
      clean(vm, bad_middles);
      if (__any(bad != 0)) any_bad = true;
    }
    {
      u32x4 m = vm;
#pragma unroll
      for (int x = 0; x < 4; ++x) m[x] = n < G ? m[x] : n == 15 ? kOnes : 0u;
#pragma unroll
      for (int r = 0; r < RT; ++r) rest[r] = mfma16<false>(m, w[r], rest[r]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const u32x4 sv = vs[GS == 32 ? u : u * 64 / GS];
      f16x2 ss[4], c24[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        ss[x] = as_f16x2(sv[x]);
        c24[x] = times_24(ss[x]);
      }
      auto product = [&](auto r) {
        constexpr int R = decltype(r)::value;
        u32x4 vt;
#pragma unroll
        for (int x = 0; x < 4; ++x) vt[x] = decode<R>(vw[u][x], ss[x], c24[x], masks);
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r][u][R] = mfma16<false>(vt, w[r], acc[r][u][R]);
      };
      product(std::integral_constant<int, 0>{});
      product(std::integral_constant<int, 1>{});
      product(std::integral_constant<int, 2>{});
      product(std::integral_constant<int, 3>{});
    }
    if constexpr (MORE) {
      __builtin_amdgcn_sched_barrier(0);
      load_v(blocks);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (c < c1) {
    for (; c + kWaves < c1; c += kWaves) step(c, std::true_type{});
    step(c, std::false_type{});
  }

  // The waves' sums meet in LDS, sixteen rows at a time. Register r of acc[t][u][i] is channel 64 u + 16 kg + 4 r + i.
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (t > 0) __syncthreads();
    const float sum = __shfl(rest[t][3], 48 + n);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float middle;
      if constexpr (GS == 32) {  // of group 2 u + kg / 2
        const float m0 = __shfl(rest[t][2 * u & 3], (2 * u >> 2) * 16 + n), m1 = __shfl(rest[t][(2 * u + 1) & 3], ((2 * u + 1) >> 2) * 16 + n);
        middle = kg >> 1 ? m1 : m0;
      } else {
        constexpr int PER = GS / 64;
        middle = __shfl(rest[t][u / PER & 3], (u / PER >> 2) * 16 + n);
      }
      // From a group that stands for NaN: its middle is infinite or, the scale being too large, every code.
      if (fabsf(middle) == INFINITY || fabsf(acc[t][u][0][0]) == INFINITY) middle = NAN;
      if (NARROW && n >= 4) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<f32x4*>(&so[wave][n][u * 64 + kg * 16 + r * 4]) =
            f32x4{acc[t][u][0][r], acc[t][u][1][r], acc[t][u][2][r], acc[t][u][3][r]} + middle;
    }
    if (kg == 0) sml[wave][n][0] = mx[t], sml[wave][n][1] = sum;
    if (tid < kRows) ends[tid] = {row[t].token < 0 ? -1 : ((long long)row[t].token * a.Hq + row[t].head) * D, row[t].lo < row[t].hi};
    if (any_bad) {
      // Rare: the groups left out above, to the rows that see them.
      for (int c = c0 + wave; c < c1; c += kWaves) {
        if (seen_by_all(c)) continue;
        const uint32_t here = token_block(c);
        for (int key = 0; key < kChunk; ++key) {
          const int j = c * kChunk + key;
          const uint16_t* params = reinterpret_cast<const uint16_t*>(v_cache + (size_t)__shfl(here, key >> 3) * BLOCK + 4 * D) + (key & 7);
          if (j < row[t].lo || j >= row[t].hi) continue;
          for (int g = kg; g < G; g += 4)
            if (bad_scale(params[g * 16]) || bad_middle(params[g * 16 + 8]))
              for (int d = 0; d < GS; ++d) so[wave][n][g * GS + d] = NAN;
        }
      }
    }
    __syncthreads();
    // Thread: row tid / 16, D / 16 neighbouring dimensions.
    const auto pack = [=](float x, float y) { return bf16_data ? pack_pair<true>(x, y) : pack_pair<false>(x, y); };
    constexpr int E = D / 16;
    const int r = tid >> 4, d0 = (tid & 15) * E, rows = min(rows_left - t * kRows, kRows);
    float m = -INFINITY, l = 0, o[E] = {};
    if (r < rows) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sml[w][r][0]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = sml[w][r][0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(sml[w][r][0] - m);
        l += sml[w][r][1] * f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += so[w][r][d0 + e] * f;
      }
    }
    if (RT == 1 && share.parts > 1) {
      if (r < rows) {
        // A thread's pairs lie 256 pairs apart: the threads of a store write whole lines.
        float* to = p.part + (size_t)blockIdx.x * kRows * D + 2 * tid;
#pragma unroll
        for (int e = 0; e < E; e += 2) handoff_store(to + e * 256, o[e], o[e + 1]);
        if ((tid & 15) == 0) handoff_store(p.part_ml + ((size_t)blockIdx.x * kRows + r) * 2, m, l);
      }
      const size_t tile = ((size_t)b * a.Hkv + hk) * p.rtiles + rt;
      if (handoff_last(&p.counters[tile], (uint32_t)share.parts, &s_last)) join_parts<D>(k, share, ends, rows, shared, pack);
      return;
    }
    if (r >= rows) continue;
    const float inv = ends[r].some ? 1 / l : 0.f;
    uint16_t* dst = a.out + ends[r].at + d0;
#pragma unroll
    for (int e = 0; e < E; e += 4)
      *reinterpret_cast<u32x2*>(dst + e) = u32x2{pack(o[e] * inv, o[e + 1] * inv), pack(o[e + 2] * inv, o[e + 3] * inv)};
  }
}

template <int D, int G>
hipError_t launch_split(const AttentionArgs& a, bool bf16, hipStream_t stream) {
  const Kv4Plan plan = kv4_plan(a.B, a.Hq, a.Hkv, D, a.max_q, a.max_kv, device_topology());
  Kv4KernelArgs p = {{a, fixed_div(a.page_size), fixed_div(plan.group), plan.group, plan.rtiles, 1, reinterpret_cast<uint32_t*>(a.workspace), nullptr, nullptr},
                     plan.fit, plan.parts, cap_kind(a.softcap), bf16};
  if (plan.parts) {
    p.r.part = reinterpret_cast<float*>(a.workspace + kWorkspaceHeader);
    p.r.part_ml = p.r.part + plan.blocks * kRows * D;
  }
  const dim3 grid((unsigned)plan.blocks);
  if ((long long)a.max_q * plan.group <= 4) kv4_split_kernel<D, G, true, 1><<<grid, 64 * kWaves, 0, stream>>>(p);
  else if (!plan.wide) kv4_split_kernel<D, G, false, 1><<<grid, 64 * kWaves, 0, stream>>>(p);
  else if constexpr (D <= 128) kv4_split_kernel<D, G, false, 2><<<grid, 64 * kWaves, 0, stream>>>(p);
  return hipGetLastError();
}

// Blocks of many rows, whose keys are not split, where their waves (32 rows each) fill the CUs' SIMDs and the sequences
// have half a block of rows on average. Measured, time of the other kernel over that of the blocks, 24 to 32 heads over 8 to 32,
// dimensions of 128: half as many waves 0.5 to 0.7; as many 0.85 to 1.3; many 1.5 to 1.8; sequences of a quarter of a
// block 0.45 to 0.7 with one query head a key head.
// There a block spans the most positions, so that its rows see the fewest keys in common: prompts of 500 to 8000 without masks, with
// windows, documents and distances (756 shapes, the middle 80 of 100) 0.7 to 1.06 with D 64, 0.9 on average; 0.8 to 1.04 with D 256 and
// distances, 0.92; but 0.9 to 1.3 with D 128 and 1.0 to 1.15 with D 256 otherwise. Prompts of few tiles, whose keys would be
// in parts, 0.8 to 1.5 whatever D, 1.2 on average. (Several query heads a key head: 1.0 to 1.6, D 64 1.2 on average, D 128 1.5.)
bool use_tiles(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv, bool biased, DeviceTopo topo) {
  const long long tokens = std::min<long long>(T, (long long)B * max_q), rows = tokens * (Hq / Hkv);
  if (rows < 128ll * B || (rows + 31) / 32 * Hkv < 4ll * topo.cus) return false;
  return Hq != Hkv || !(D == 64 || (D == 256 && biased)) || kv4_plan(B, Hq, Hkv, D, max_q, max_kv, topo).parts > 0;
}

}  // namespace

size_t kv4_attention_workspace(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv) {
  if (use_tiles(B, T, Hq, Hkv, D, max_q, max_kv, true, device_topology())) return 0;
  const Kv4Plan p = kv4_plan(B, Hq, Hkv, D, max_q, max_kv, device_topology());
  return p.parts ? kWorkspaceHeader + p.blocks * kRows * (D + 2) * sizeof(float) : 0;
}

Kv4Launch kv4_attention_launch(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv, bool biased) {
  const DeviceTopo topo = device_topology();
  if (use_tiles(B, T, Hq, Hkv, D, max_q, max_kv, biased, topo)) {
    const int rows = D == 256 ? kKv4TileRows<256> : kKv4TileRows<128>, waves = D == 256 ? kKv4TileWaves<256> : kKv4TileWaves<128>;
    return {kKv4Blocks, rows, tile_blocks(B, Hkv, row_tiles(max_q, Hq / Hkv, rows)), 0, 0, 64 * waves};
  }
  const Kv4Plan p = kv4_plan(B, Hq, Hkv, D, max_q, max_kv, topo);
  return {p.parts ? kKv4Parts : p.wide ? kKv4Pair : kKv4Tile, p.wide ? 2 * kRows : kRows, p.blocks, p.parts ? p.fit : 0, p.parts,
          64 * kWaves};
}

hipError_t launch_kv4_attention(const AttentionArgs& a, int group_size, bool bf16, hipStream_t stream) {
  if (kv4_attention_launch(a.B, a.T, a.Hq, a.Hkv, a.D, a.max_q, a.max_kv, a.slopes).kernel == kKv4Blocks) {
    const Kv4TileArgs t = {a, bf16};
    return a.D == 64 ? launch_kv4_tiles<64>(t, group_size, stream)
           : a.D == 128 ? launch_kv4_tiles<128>(t, group_size, stream) : launch_kv4_tiles<256>(t, group_size, stream);
  }
  if (a.D == 64) return group_size == 32 ? launch_split<64, 2>(a, bf16, stream) : launch_split<64, 1>(a, bf16, stream);
  if (a.D == 128)
    return group_size == 32 ? launch_split<128, 4>(a, bf16, stream)
           : group_size == 64 ? launch_split<128, 2>(a, bf16, stream) : launch_split<128, 1>(a, bf16, stream);
  return group_size == 32 ? launch_split<256, 8>(a, bf16, stream)
         : group_size == 64 ? launch_split<256, 4>(a, bf16, stream) : launch_split<256, 2>(a, bf16, stream);
}

}  // namespace qmm
