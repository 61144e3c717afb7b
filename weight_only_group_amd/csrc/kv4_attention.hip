// Attention of new tokens to their sequences' cache in 4 bits.
//
// The formulas of the attention to a cache of 16-bit values, with k_j = m + s (c - 8) per
// group of channels, taken apart so that what the matrix cores see is exact in fp16:
//   q.k_j = sum_d q_d [s_j (c_jd - 8)] + sum_g m_jg Q_g,     Q_g = sum of the group's q_d
//   sum_j p_j v_j = sum_j p_j [s_j (c_jd - 8)] + sum_j p_j m_jg
// s has 8 significant bits and c - 8 three and a sign, so the brackets are fp16 numbers.
// A code becomes one by an AND, an OR and half a packed multiply-add: the half 16 + c
// has it in the top of its mantissa, and s (16 + c) - 24 s is rounded once, so not at all.
// The second sums are one matrix operation more for all channels together, with
// the middles as further channels; Q goes in three fp16 parts (33 bits). A row of ones among
// the value's middles gives the weights' sum.
//
// Queries are scaled by a power of two, so that a row's largest is in [1, 2) and fp16
// holds them whatever their type. The weights p are fp16, 2^14 for a row's largest key so
// far, so that those down to 2^-28 of it keep all their bits.
#include <type_traits>

#include "attention_rows.h"
#include "cache.h"

namespace qmm {
namespace {

constexpr float kLift = 14.f;  // log2 of the largest weight

// Two of a word's codes, nibbles r and r + 4, as s (c - 8); c24 = -24 s.
template <int R>
__device__ __forceinline__ uint32_t decode(uint32_t w, f16x2 s, f16x2 c24) {
  constexpr uint32_t mask = 0x03C003C0u, sixteen = 0x4C004C00u;
  const uint32_t at = R == 0 ? w << 6 : R == 1 ? w << 2 : R == 2 ? w >> 2 : w >> 6;
  return as_u32(__builtin_elementwise_fma(as_f16x2((at & mask) | sixteen), s, c24));
}
__device__ __forceinline__ f16x2 times_24(f16x2 s) { return s * f16x2{(f16)-24.f, (f16)-24.f}; }  // exact: 10 bits

// Whether a half of the pair is an infinity or a NaN, as a mask of those halves.
__device__ __forceinline__ uint32_t not_finite_halves(uint32_t v) {
  return (not_finite<false>(v) ? 0xFFFFu : 0u) | (not_finite<false>(v >> 16) ? 0xFFFF0000u : 0u);
}

// BYTES (a multiple of 4, up to 32) from p as 32-bit words.
template <int BYTES>
__device__ __forceinline__ void load_words(uint32_t (&to)[BYTES / 4], const uint8_t* p) {
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

// Block: one tile of 16 rows, one part of its keys, in chunks of 32 keys a wave, as for the
// cache of 16-bit values. The products are K q^T and V^T p^T. Row i of a chunk's t-th
// sixteen is key 8 (i / 4) + 4 t + i % 4, so that a lane's scores are those of one block of
// eight tokens, whose values' words hold two tokens each: they need no exchange.
template <int D, int G, Cap CAP>
__global__ void __launch_bounds__(256, D == 256 ? 2 : 3) kv4_split_kernel(AttnKernelArgs p, bool bf16_data) {
  constexpr int STEPS = D / 32, U = D / 64, GS = D / G, BLOCK = kv4_block_bytes(D, G);
  constexpr int NS = GS == 32 ? U : G;  // sets of scales that a lane needs for its values
  constexpr int LD = D + 4;
  __shared__ float so[kWaves][kRows][LD];
  __shared__ float sml[kWaves][kRows][2];
  __shared__ int s_last;
  const AttentionArgs& a = p.a;
  const uint8_t* k_cache = reinterpret_cast<const uint8_t*>(a.k_cache);
  const uint8_t* v_cache = reinterpret_cast<const uint8_t*>(a.v_cache);
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
  ScoreRule rule = score_rule(a, row.head);

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

  // The row's query in fp16, and its groups' sums in three parts (lane group 0: the first, ...).
  u32x4 q[STEPS], qsum = {0, 0, 0, 0};
  {
    u32x4 raw[STEPS];
    uint32_t most = 0;  // of the values' bits without a sign: in the order of their sizes
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      raw[s] = row.token < 0 ? u32x4{0, 0, 0, 0}
                             : *reinterpret_cast<const u32x4*>(a.q + row.token * a.q_stride + (long long)row.head * D + s * 32 + kg * 8);
#pragma unroll
      for (int x = 0; x < 4; ++x) most = max(most, max(raw[s][x] & 0x7FFFu, raw[s][x] >> 16 & 0x7FFFu));
    }
    most = max(most, (uint32_t)__shfl_xor((int)most, 16));
    most = max(most, (uint32_t)__shfl_xor((int)most, 32));
    const float largest = bf16_data ? bits_to_float<true>((uint16_t)most) : bits_to_float<false>((uint16_t)most);
    const bool finite = largest < INFINITY;
    const int up = min(max(254 - (int)(__builtin_bit_cast(uint32_t, largest) >> 23), 1), 253);  // exponent field of the factor
    const float factor = finite ? __builtin_bit_cast(float, (uint32_t)up << 23) : NAN;
    const float back = __builtin_bit_cast(float, (uint32_t)(254 - up) << 23);
    rule.scale = fminf(fmaxf(rule.scale * back, -3e38f), 3e38f);
    rule.inverse = fminf(fmaxf(rule.inverse * back, -3e38f), 3e38f);
    float sums[G] = {};
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint16_t b0 = (uint16_t)raw[s][x], b1 = (uint16_t)(raw[s][x] >> 16);
        const float f0 = bf16_data ? bits_to_float<true>(b0) : bits_to_float<false>(b0);
        const float f1 = bf16_data ? bits_to_float<true>(b1) : bits_to_float<false>(b1);
        const f16x2 h = {(f16)(f0 * factor), (f16)(f1 * factor)};
        q[s][x] = as_u32(h);
        sums[s * 32 / GS] += (float)h[0] + (float)h[1];
      }
    f16 part_of[8] = {};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float s = sums[g];
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      const f16 first = (f16)s, second = (f16)(s - (float)first), third = (f16)(s - (float)first - (float)second);
      part_of[g] = kg == 0 ? first : kg == 1 ? second : kg == 2 ? third : (f16)0.f;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) qsum[x] = as_u32(f16x2{part_of[2 * x], part_of[2 * x + 1]});
  }

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

  f32x4 acc[U][4] = {}, rest = {};  // rest: rows g the sums of p m_g, row 15 the sum of p
  float mx = -INFINITY;
  bool any_bad = false;
  uint32_t blocks = 0, blocks_next = 0;
  // One chunk; with MORE the next one's loads go out as the registers fall free.
  auto step = [&](int c, auto more) {
    constexpr bool MORE = decltype(more)::value;
    f32x4 st[2] = {};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      // Halves [s of all groups][m of all groups].
      u32x4 middles = {0, 0, 0, 0};
      if constexpr (G == 1) {
        middles[0] = kp[t][0] >> 16;
      } else {
#pragma unroll
        for (int x = 0; x < G / 2; ++x) middles[x] = kp[t][G / 2 + x];
      }
      st[t] = mfma16<false>(middles, qsum, st[t]);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int g = s * 32 / GS;
        const uint32_t pair = kp[t][g / 2];
        const f16 sg = as_f16x2(pair)[g % 2];
        const f16x2 ss = {sg, sg}, c24 = times_24(ss);
        const uint32_t w = kw[t][s];
        st[t] = mfma16<false>(u32x4{decode<0>(w, ss, c24), decode<1>(w, ss, c24), decode<2>(w, ss, c24), decode<3>(w, ss, c24)}, q[s], st[t]);
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
    // Scores: key 32 c + 8 kg + 4 t + r of row n.
    const int j0 = c * kChunk + 8 * kg;
    const bool whole = seen_by_all(c);
    float s[8], best = -INFINITY;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      s[x] = rule.template score<CAP, true>(st[x >> 2][x & 3], row.pos, j0 + x);
      if (!whole) s[x] = j0 + x >= row.lo && j0 + x < row.hi ? s[x] : -INFINITY;
      best = fmaxf(best, s[x]);
    }
    best = fmaxf(best, __shfl_xor(best, 16));
    best = fmaxf(best, __shfl_xor(best, 32));
    if (__any(best > mx)) {
      const float m = fmaxf(mx, best);
      const float f = mx == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mx - m);
      rest *= f;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u][i] *= f;
      mx = m;
    }
    const float off = mx == -INFINITY ? 0.f : mx - kLift;
    u32x4 w;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      w[x] = pack_pair<false>(__builtin_amdgcn_exp2f(s[2 * x] - off), __builtin_amdgcn_exp2f(s[2 * x + 1] - off));
    if (!whole) {
      // Places that no row sees may hold anything: their scales and middles count as 0. So do those
      // of a seen place that are not finite, as they must not reach the rows that do not see it (0
      // times NaN is NaN); those that do get a NaN after the loop.
      uint32_t bad = 0;
      auto clean = [&](u32x4& v) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int j = j0 + 2 * x;
          const uint32_t in = (j >= lo && j < hi ? 0xFFFFu : 0u) | (j + 1 >= lo && j + 1 < hi ? 0xFFFF0000u : 0u);
          const uint32_t nf = not_finite_halves(v[x]) & in;
          bad |= nf;
          v[x] &= in & ~nf;
        }
      };
#pragma unroll
      for (int i = 0; i < NS; ++i) clean(vs[i]);
      clean(vm);
      if (__any(bad != 0)) any_bad = true;
    }
    {
      u32x4 m = vm;
#pragma unroll
      for (int x = 0; x < 4; ++x) m[x] = n < G ? m[x] : n == 15 ? 0x3C003C00u : 0u;
      rest = mfma16<false>(m, w, rest);
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
        for (int x = 0; x < 4; ++x) vt[x] = decode<R>(vw[u][x], ss[x], c24[x]);
        acc[u][R] = mfma16<false>(vt, w, acc[u][R]);
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
  int c = c0 + wave;
  if (c < c1) {
    blocks = token_block(c);
    load_k(blocks);
    load_v(blocks);
    blocks_next = token_block(c + kWaves);
    for (; c + kWaves < c1; c += kWaves) step(c, std::true_type{});
    step(c, std::false_type{});
  }

  // The waves' sums meet in LDS. Register r of acc[u][i] is channel 64 u + 16 kg + 4 r + i.
  const float sum = __shfl(rest[3], 48 + n);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float middle;
    if constexpr (GS == 32) {  // of group 2 u + kg / 2
      const float m0 = __shfl(rest[2 * u & 3], (2 * u >> 2) * 16 + n), m1 = __shfl(rest[(2 * u + 1) & 3], ((2 * u + 1) >> 2) * 16 + n);
      middle = kg >> 1 ? m1 : m0;
    } else {
      constexpr int PER = GS / 64;
      middle = __shfl(rest[u / PER & 3], (u / PER >> 2) * 16 + n);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<f32x4*>(&so[wave][n][u * 64 + kg * 16 + r * 4]) =
          f32x4{acc[u][0][r], acc[u][1][r], acc[u][2][r], acc[u][3][r]} + middle;
  }
  if (kg == 0) sml[wave][n][0] = mx, sml[wave][n][1] = sum;
  if (any_bad) {
    // Rare: the groups left out above, to the rows that see them.
    for (int c = c0 + wave; c < c1; c += kWaves) {
      if (seen_by_all(c)) continue;
      const uint32_t here = token_block(c);
      for (int key = 0; key < kChunk; ++key) {
        const int j = c * kChunk + key;
        const uint16_t* params = reinterpret_cast<const uint16_t*>(v_cache + (size_t)__shfl(here, key >> 3) * BLOCK + 4 * D) + (key & 7);
        if (j < row.lo || j >= row.hi) continue;
        for (int g = kg; g < G; g += 4)
          if (not_finite<false>(params[g * 16]) || not_finite<false>(params[g * 16 + 8]))
            for (int d = 0; d < GS; ++d) so[wave][n][g * GS + d] = NAN;
      }
    }
  }
  __syncthreads();
  join_rows<D>(p, so, sml, &s_last, span, b, hk, rt, part, [=](float x, float y) { return bf16_data ? pack_pair<true>(x, y) : pack_pair<false>(x, y); });
}

template <int D, int G>
hipError_t launch_split(const AttentionArgs& a, bool bf16, hipStream_t stream) {
  const AttnPlan plan = attn_plan(a.B, a.Hq, a.Hkv, a.max_q, a.max_kv, device_topology());
  AttnKernelArgs p = {a, fixed_div(a.page_size), fixed_div(plan.group), plan.group, plan.rtiles, plan.split, reinterpret_cast<uint32_t*>(a.workspace), nullptr, nullptr};
  if (plan.split > 1) {
    p.part = reinterpret_cast<float*>(a.workspace + kWorkspaceHeader);
    p.part_ml = p.part + plan.tiles * plan.split * kRows * D;
  }
  const dim3 grid((unsigned)tile_blocks(a.B, a.Hkv * plan.split, plan.rtiles));
  const auto run = [&](auto kernel) { kernel<<<grid, 64 * kWaves, 0, stream>>>(p, bf16); };
  switch (cap_kind(a.softcap)) {
    case kNoCap: run(kv4_split_kernel<D, G, kNoCap>); break;
    case kSmallCap: run(kv4_split_kernel<D, G, kSmallCap>); break;
    case kAnyCap: run(kv4_split_kernel<D, G, kAnyCap>); break;
  }
  return hipGetLastError();
}

}  // namespace

size_t kv4_attention_workspace(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv) {
  const AttnPlan p = attn_plan(B, Hq, Hkv, max_q, max_kv, device_topology());
  return p.split > 1 ? kWorkspaceHeader + p.tiles * p.split * kRows * (D + 2) * sizeof(float) : 0;
}

long long kv4_attention_blocks(int B, int Hq, int Hkv, int max_q, int max_kv) {
  const AttnPlan p = attn_plan(B, Hq, Hkv, max_q, max_kv, device_topology());
  return tile_blocks(B, Hkv * p.split, p.rtiles);
}

hipError_t launch_kv4_attention(const AttentionArgs& a, int group_size, bool bf16, hipStream_t stream) {
  if (a.D == 64) return group_size == 32 ? launch_split<64, 2>(a, bf16, stream) : launch_split<64, 1>(a, bf16, stream);
  if (a.D == 128)
    return group_size == 32 ? launch_split<128, 4>(a, bf16, stream)
           : group_size == 64 ? launch_split<128, 2>(a, bf16, stream) : launch_split<128, 1>(a, bf16, stream);
  return group_size == 32 ? launch_split<256, 8>(a, bf16, stream)
         : group_size == 64 ? launch_split<256, 4>(a, bf16, stream) : launch_split<256, 2>(a, bf16, stream);
}

}  // namespace qmm
