// The mixture-of-experts layer with quantised experts for a few tokens: the
// routing, then one launch for the gate and up products with the gating, and one
// for the down products with the weighted sum.
//
// An assignment is a (token, choice) pair, t * top_k + j. A group's part of a
// product is s (sum_k x q - z sum_k x): codes go to the matrix cores as they are,
// the scale and zero point are applied to the sums.
#include "gemv_common.h"
#include "handoff.h"
#include "layer.h"
#include "mfma.h"

namespace qmm {
namespace {

// ---- routing -------------------------------------------------------------------

constexpr int kRouteWaves = 8;

// The largest of a wave's values in every lane (bit patterns in the floats' order).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x111, 0xF, 0xF, false));  // row_shr:1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x112, 0xF, 0xF, false));  // row_shr:2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x114, 0xF, 0xF, false));  // row_shr:4
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x118, 0xF, 0xF, false));  // row_shr:8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x142, 0xF, 0xF, false));  // row_bcast:15
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x143, 0xF, 0xF, false));  // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Unsigned order of floats: larger logits larger, NaN above all, -0 as 0; 0 is below every one.
__device__ __forceinline__ uint32_t float_order(float l) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);
  return l != l ? 0xFFFFFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// One wave: the top_k of token t. Each lane holds a run of PER neighbouring
// experts, so that among equal logits the lowest lane has the lowest expert.
template <int PER>
__device__ void route_top(const RouteArgs& a, int t, int lane) {
  const float* l = a.logits + (size_t)t * a.E;
  uint32_t key[PER];
  float mx = 0, total = 0, mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    key[i] = e < a.E ? float_order(handoff_load(&l[e])) : 0;
  }
  auto value = [](uint32_t k) {
    return __builtin_bit_cast(float, k == 0xFFFFFFFFu ? 0x7FC00000u : (k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
  };
  if (!a.renormalize) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) best = max(best, key[i]);
    mx = value(wave_max(best));
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i]) total += __expf(value(key[i]) - mx);
    for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
  }
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (key[i] > best) best = key[i], at = i;
    const uint32_t top = wave_max(best);
    const int from = __builtin_ctzll(__ballot(best == top));
    const int e = __builtin_amdgcn_readlane(lane * PER + at, from);
    if (lane == from) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == at) key[i] = 0;
    }
    if (j == 0) mx = value(top);
    const float p = __expf(value(top) - mx);
    if (a.renormalize) total += p;
    if (lane == j) {
      mine = p;
      a.ids[t * a.top_k + j] = e;
    }
  }
  if (lane < a.top_k) a.weights[t * a.top_k + lane] = mine / total;
}

// Block: the logits of 16 experts for 16 tokens, its waves over H; the block that
// ends a token tile's logits chooses for its tokens. Bound: latency (a few hundred
// KiB of router weights over the CUs).
template <bool BF>
__global__ void __launch_bounds__(64 * kRouteWaves) route_kernel(RouteArgs a) {
  __shared__ float part[kRouteWaves][16][17];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, kg = lane >> 4;
  const int e = min((int)blockIdx.x * 16 + n, a.E - 1), t0 = blockIdx.y * 16, t = min(t0 + n, a.T - 1);
  const u32x4* x = reinterpret_cast<const u32x4*>(a.x + (size_t)t * a.H + kg * 8);
  const u32x4* r = reinterpret_cast<const u32x4*>(a.router + (size_t)e * a.H + kg * 8);
  f32x4 acc = {};
  const int units = a.H / 32;
  constexpr int kBatch = 4;  // units whose loads go out together
  for (int u0 = wave; u0 < units; u0 += kBatch * kRouteWaves) {
    u32x4 xv[kBatch], rv[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int u = min(u0 + i * kRouteWaves, units - 1);
      xv[i] = x[u * 4];
      rv[i] = r[u * 4];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (u0 + i * kRouteWaves < units) acc = mfma16<BF>(xv[i], rv[i], acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][4 * kg + i][n] = acc[i];
  __syncthreads();
  if (tid < 256) {
    const int row = tid >> 4, col = tid & 15;
    float s = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) s += part[w][row][col];
    if (t0 + row < a.T && (int)blockIdx.x * 16 + col < a.E)
      handoff_store(&a.logits[(size_t)(t0 + row) * a.E + blockIdx.x * 16 + col], s);
  }
  if (!handoff_last(&a.counters[blockIdx.y], gridDim.x, &s_last)) return;
  for (int i = t0 + wave; i < min(t0 + 16, a.T); i += kRouteWaves) {
    if (a.E <= 64) route_top<1>(a, i, lane);
    else if (a.E <= 128) route_top<2>(a, i, lane);
    else if (a.E <= 256) route_top<4>(a, i, lane);
    else route_top<16>(a, i, lane);
  }
}

// ---- codes as matrix operands --------------------------------------------------------

// Eight codes of lane group j, in decode8's element order, as 16-bit numbers:
// fp16: q 2^-24 (a subnormal half, exact); bf16: 128 + q for up to 4 bits (the
// code in the mantissa's low bits), q for 8 bits (exact in 8 significant bits).
template <int BITS, bool BF>
__device__ __forceinline__ u32x4 codes8(uint32_t w0, uint32_t w1, int j) {
  u32x4 b;
  constexpr uint32_t kOr = BF ? 0x43004300u : 0u;
  if constexpr (BITS == 4) {
#pragma unroll
    for (int p = 0; p < 4; ++p) b[p] = ((w0 >> (4 * p)) & 0x000F000Fu) | kOr;
  } else if constexpr (BITS == 8) {
    if constexpr (BF) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t w = p < 2 ? w0 : w1;
        const float lo = (float)((w >> (16 * (p & 1))) & 0xFF), hi = (float)((w >> (16 * (p & 1) + 8)) & 0xFF);
        b[p] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
      }
    } else {
      b[0] = __builtin_amdgcn_perm(0u, w0, 0x0C010C00u);
      b[1] = __builtin_amdgcn_perm(0u, w0, 0x0C030C02u);
      b[2] = __builtin_amdgcn_perm(0u, w1, 0x0C010C00u);
      b[3] = __builtin_amdgcn_perm(0u, w1, 0x0C030C02u);
    }
  } else if constexpr (BITS == 2) {
    const uint32_t t = w0 >> (8 * (j & 1));
#pragma unroll
    for (int p = 0; p < 4; ++p) b[p] = ((t >> (2 * p)) & 0x00030003u) | kOr;
  } else if constexpr (BITS == 3) {
    const uint32_t h = w0 >> (8 * (j & 1));
    const uint32_t t = w1 >> (16 * (j >> 1) + 4 * (j & 1));
    const uint32_t l = __builtin_amdgcn_perm(0u, t, 0x0C010C00u);  // bytes (0, -, 1, -) of t
#pragma unroll
    for (int p = 0; p < 4; ++p) b[p] = (((h >> (2 * p)) & 0x00030003u) << 1) | ((l >> p) & 0x00010001u) | kOr;
  } else {
    const uint32_t t = (w0 >> (8 * j)) & 0xFFu, both = t | (t << 12);  // slots p and p + 4 sixteen bits apart
#pragma unroll
    for (int p = 0; p < 4; ++p) b[p] = ((both >> p) & 0x00010001u) | kOr;
  }
  return b;
}
template <int BITS, bool BF> constexpr float kCodeOffset = BF && BITS <= 4 ? 128.f : 0.f;

// Place of k (0..31 of a unit) when the operands of the four lane groups lie one
// behind another, each in decode8's element order.
template <int BITS>
__device__ __forceinline__ int operand_place(int k) {
  if constexpr (BITS == 8) return k;
  else if constexpr (BITS == 4 || BITS == 1) return (k & 24) | ((k & 3) << 1) | ((k >> 2) & 1);
  else return (k & 16) | ((k & 4) << 1) | ((k & 3) << 1) | ((k >> 3) & 1);
}

// Words of one plane for strip columns c0..c0 + 15: word (r, c0 + n) at base[r * stride].
struct PlaneColumn {
  const uint32_t *hi, *lo;
  int stride;
};
template <int BITS>
__device__ __forceinline__ PlaneColumn plane_column(const ExpertPlanes& w, int e, int K, int N, int strips, int col) {
  constexpr int HB = BITS == 3 ? 2 : BITS;
  const int rows = K * HB / 32;
  PlaneColumn p;
  p.stride = plane_row_stride(N, strips);
  p.hi = w.qw + (size_t)e * rows * N + plane_col(col, rows, strips);
  p.lo = BITS == 3 ? w.qlo + (size_t)e * (K / 32) * N + plane_col(col, K / 32, strips) : nullptr;
  return p;
}

// A chunk: four units (32 k each) of one column strip.
constexpr int kUnits = 4;
template <int BITS> struct ChunkWords { uint32_t w[kUnits][Bits<BITS>::NW]; };

template <int BITS>
__device__ __forceinline__ void load_chunk(ChunkWords<BITS>& c, const PlaneColumn& p, int u0, int units, int j) {
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = min(u0 + i, units - 1);
#pragma unroll
    for (int x = 0; x < Bits<BITS>::NW; ++x) {
      const uint32_t* base = BITS == 3 && x == 1 ? p.lo : p.hi;
      c.w[i][x] = __builtin_nontemporal_load(base + (uint32_t)(u * unit_rows<BITS>(x) + lane_row<BITS>(j, x)) * (uint32_t)p.stride);
    }
  }
}

// Scale (low half) and zero point of lane group j's unit of the chunk, for this lane's column.
__device__ __forceinline__ uint32_t load_group(const ExpertPlanes& w, size_t expert_groups, int N, int col, int u, int upg) {
  const size_t at = (expert_groups + (uint32_t)u / (uint32_t)upg) * N + col;
  return (uint32_t)w.scales[at] | (uint32_t)w.zeros[at] << 16;
}

// ---- gate and up products --------------------------------------------------------------

constexpr int kGateWaves = 8;

// The experts in use are numbered by slots: with fewer assignments than experts
// a slot is an assignment (in use where it is the first of its expert), else an
// expert. Per slot: its expert, the number of its assignments and the assignments.
struct Slots {
  int count;
  int* rows;       // (slots) assignments of each; 0: not in use
  uint16_t* list;  // (slots, T)
};

struct MoeKernelArgs {
  MoeArgs a;
  Slots slots;
  uint16_t* h;  // (assignments, 2, I) bf16: high and low parts, each unit in operand order
  int strips;
};

// Row tiles of NT * 16 assignments from `base` on: partial sums of a wave.
template <int BITS, bool BF, int NT>
__device__ __forceinline__ void gate_up_rows(const MoeKernelArgs& p, int e, int strip, const uint16_t* list, int base, int rows,
                                             float (*sums)[2][16 * NT][17]) {
  const MoeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, j = lane >> 4;
  const int units = a.H / 32, upg = a.gs_h / 32, chunks = (units + kUnits - 1) / kUnits, N = 2 * a.I;
  const PlaneColumn col[2] = {plane_column<BITS>(a.gate_up, e, a.H, N, p.strips, strip * 16 + n),
                              plane_column<BITS>(a.gate_up, e, a.H, N, p.strips, a.I + strip * 16 + n)};
  const size_t groups = (size_t)e * (units / upg);
  const uint16_t* x[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int at = list[min(base + 16 * t + n, rows - 1)];
    x[t] = a.x + (size_t)(at / a.top_k) * a.H + x_first<BITS>(j);
  }
  struct Stage {
    ChunkWords<BITS> w[2];
    uint32_t sz[2];
    u32x4 x[NT][kUnits];
  } st[2];
  auto load = [&](Stage& s, int c) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      load_chunk<BITS>(s.w[v], col[v], c * kUnits, units, j);
      s.sz[v] = load_group(a.gate_up, groups, N, v * a.I + strip * 16 + n, min(c * kUnits + j, units - 1), upg);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const uint16_t* src = x[t] + min(c * kUnits + i, units - 1) * 32;
        if constexpr (BITS == 2 || BITS == 3) {
          const u32x2 lo = *reinterpret_cast<const u32x2*>(src), hi = *reinterpret_cast<const u32x2*>(src + 8);
          s.x[t][i] = u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
          s.x[t][i] = *reinterpret_cast<const u32x4*>(src);
        }
      }
  };
  f32x4 total[2][NT] = {};
  constexpr uint32_t kOne = BF ? 0x3F803F80u : 0x3C003C00u;
  auto compute = [&](const Stage& s, int c) {
    f32x4 acc[2][NT] = {}, xs[NT] = {};
    int in_group = (c * kUnits) % upg;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (c * kUnits + i < units) {
        u32x4 xa[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          xa[t] = x_operand<BITS>(s.x[t][i]);
          xs[t] = mfma16<BF>(xa[t], u32x4{kOne, kOne, kOne, kOne}, xs[t]);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const u32x4 b = codes8<BITS, BF>(s.w[v].w[i][0], s.w[v].w[i][Bits<BITS>::NW - 1], j);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[v][t] = mfma16<BF>(xa[t], b, acc[v][t]);
        }
      }
      // The end of a group or of the chunk: scale and zero point, from the lane group that holds the unit's.
      if (++in_group == upg || i == kUnits - 1) {
        if (in_group == upg) in_group = 0;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t sz = __shfl(s.sz[v], 16 * i + n);
          const float sc = bits_to_float<BF>((uint16_t)sz), z = bits_to_float<BF>((uint16_t)(sz >> 16)) + kCodeOffset<BITS, BF>;
          constexpr float kUp = BF ? 1.f : 16777216.f;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) total[v][t][r] += sc * (acc[v][t][r] * kUp - z * xs[t][r]);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[v][t] = f32x4{};
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) xs[t] = f32x4{};
      }
    }
  };
  int c = wave;
  if (c < chunks) load(st[0], c);
  while (c < chunks) {
    if (c + kGateWaves < chunks) load(st[1], c + kGateWaves);
    compute(st[0], c);
    c += kGateWaves;
    if (c >= chunks) break;
    if (c + kGateWaves < chunks) load(st[0], c + kGateWaves);
    compute(st[1], c);
    c += kGateWaves;
  }
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wave][v][16 * t + 4 * j + r][n] = total[v][t][r];
  __syncthreads();
  for (int o = tid; o < 16 * NT * 16; o += 64 * kGateWaves) {
    const int row = o >> 4, cc = o & 15;
    float g = 0, u = 0;
#pragma unroll
    for (int w = 0; w < kGateWaves; ++w) g += sums[w][0][row][cc], u += sums[w][1][row][cc];
    if (base + row >= rows) continue;
    const float h = g / (1 + __expf(-g)) * u;
    const bf16 hi = (bf16)h;
    const float rest = h - (float)hi;
    // (an infinite high part takes no low one: inf - inf is NaN)
    const bf16 lo = (bf16)(fabsf((float)hi) == INFINITY ? 0.f : rest);
    const int i = strip * 16 + cc, place = (i & ~31) | operand_place<BITS>(i & 31);
    uint16_t* dst = p.h + (size_t)list[base + row] * 2 * a.I + place;
    dst[0] = __builtin_bit_cast(uint16_t, hi);
    dst[a.I] = __builtin_bit_cast(uint16_t, lo);
  }
  __syncthreads();
}

// Block: 16 gate and the 16 up columns of one expert, its waves over H. Bound: HBM,
// an expert's words are read once for all its tokens (twice from 33 on).
template <int BITS, bool BF>
__global__ void __launch_bounds__(64 * kGateWaves, 2) gate_up_kernel(MoeKernelArgs p) {
  __shared__ float sums[kGateWaves][2][32][17];
  __shared__ uint16_t list[kMoeTokens];
  __shared__ int counts[2][kGateWaves];
  const MoeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, strip = blockIdx.x, slot = blockIdx.y;
  const int assignments = a.T * a.top_k;
  const bool by_assignment = p.slots.count == assignments;
  const int e = by_assignment ? a.ids[slot] : slot;
  // The expert's assignments, in order; a slot whose expert came before is not in use.
  bool dup = false;
  int rows = 0;
  for (int base = 0; base < assignments; base += 64 * kGateWaves) {
    const int i = base + tid;
    const bool mine = i < assignments && a.ids[i] == e;
    dup |= mine && by_assignment && i < slot;
    const uint64_t hits = __ballot(mine);
    int* count = counts[(base / (64 * kGateWaves)) & 1];
    if (lane == 0) count[wave] = __builtin_popcountll(hits);
    __syncthreads();
    int before = rows;
    for (int w = 0; w < kGateWaves; ++w) {
      if (w < wave) before += count[w];
      rows += count[w];
    }
    before += __builtin_popcountll(hits & ((1ull << lane) - 1));
    if (mine && before < a.T) list[before] = (uint16_t)i;
  }
  const bool unused = __syncthreads_or(dup) || e < 0 || e >= a.E || rows == 0;
  rows = unused ? 0 : min(rows, a.T);
  if (strip == 0) {
    if (tid == 0) p.slots.rows[slot] = rows;
    if (tid < rows) p.slots.list[(size_t)slot * a.T + tid] = list[tid];
  }
  for (int base = 0; base < rows;) {
    if (rows - base <= 16) {
      gate_up_rows<BITS, BF, 1>(p, e, strip, list, base, rows, reinterpret_cast<float (*)[2][16][17]>(sums));
      base += 16;
    } else {
      gate_up_rows<BITS, BF, 2>(p, e, strip, list, base, rows, sums);
      base += 32;
    }
  }
}

// ---- down products and the weighted sum ---------------------------------------------------

constexpr int kDownWaves = 16;

// Block: 16 columns of y for all tokens; its waves take (expert, chunk) pairs in
// turn and add to sums of their own, which meet in wave order. A row tile is 8
// assignments: the high parts of h in rows 0-7, the low parts in rows 8-15.
// Bound: HBM, as above.
template <int BITS, bool BF>
__global__ void __launch_bounds__(64 * kDownWaves) down_kernel(MoeKernelArgs p) {
  extern __shared__ float sums[];  // (waves, T, 16)
  __shared__ uint16_t used[kMoeExperts];
  __shared__ int s_used;
  const MoeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, j = lane >> 4;
  const int strip = blockIdx.x, units = a.I / 32, upg = a.gs_i / 32, chunks = (units + kUnits - 1) / kUnits;
  const bool by_assignment = p.slots.count == a.T * a.top_k;
  if (wave == 0) {
    int total = 0;
    for (int base = 0; base < p.slots.count; base += 64) {
      const bool in_use = base + lane < p.slots.count && p.slots.rows[base + lane] > 0;
      const uint64_t hits = __ballot(in_use);
      if (in_use) used[total + __builtin_popcountll(hits & ((1ull << lane) - 1))] = (uint16_t)(base + lane);
      total += __builtin_popcountll(hits);
    }
    if (lane == 0) s_used = total;
  }
  float* mine = sums + (size_t)wave * a.T * 16;
  for (int i = lane; i < a.T * 16; i += 64) mine[i] = 0;
  __syncthreads();
  const int items = s_used * chunks;
  for (int it = wave; it < items; it += kDownWaves) {
    const int slot = used[it / chunks], c = it % chunks;
    const int e = by_assignment ? a.ids[slot] : slot, rows = p.slots.rows[slot];
    const uint16_t* list = p.slots.list + (size_t)slot * a.T;
    ChunkWords<BITS> w;
    load_chunk<BITS>(w, plane_column<BITS>(a.down, e, a.I, a.H, p.strips, strip * 16 + n), c * kUnits, units, j);
    const uint32_t sz = load_group(a.down, (size_t)e * (units / upg), a.H, strip * 16 + n, min(c * kUnits + j, units - 1), upg);
    for (int base = 0; base < rows; base += 8) {
      const int at = list[min(base + (n & 7), rows - 1)];
      const uint16_t* h = p.h + ((size_t)at * 2 + (n >> 3)) * a.I + j * 8;
      u32x4 ha[kUnits];
#pragma unroll
      for (int i = 0; i < kUnits; ++i) ha[i] = *reinterpret_cast<const u32x4*>(h + min(c * kUnits + i, units - 1) * 32);
      f32x4 total = {}, acc = {}, hs = {};
      int in_group = (c * kUnits) % upg;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        if (c * kUnits + i < units) {
          hs = mfma16<true>(ha[i], u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}, hs);
          acc = mfma16<true>(ha[i], codes8<BITS, true>(w.w[i][0], w.w[i][Bits<BITS>::NW - 1], j), acc);
        }
        if (++in_group == upg || i == kUnits - 1) {
          if (in_group == upg) in_group = 0;
          const uint32_t g = __shfl(sz, 16 * i + n);
          const float sc = bits_to_float<BF>((uint16_t)g), z = bits_to_float<BF>((uint16_t)(g >> 16)) + kCodeOffset<BITS, true>;
#pragma unroll
          for (int r = 0; r < 4; ++r) total[r] += sc * (acc[r] - z * hs[r]);
          acc = hs = f32x4{};
        }
      }
      // Rows 4 j + r of lanes j < 2 are the high parts, of lanes j + 2 the low ones.
#pragma unroll
      for (int r = 0; r < 4; ++r) total[r] += __shfl_xor(total[r], 32);
      if (j < 2) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (base + 4 * j + r < rows) {
            const int as = list[base + 4 * j + r];
            mine[(as / a.top_k) * 16 + n] += a.weights[as] * total[r];
          }
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * 16; i += 64 * kDownWaves) {
    float y = 0;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) y += sums[(size_t)w * a.T * 16 + i];
    a.y[(size_t)(i >> 4) * a.H + strip * 16 + (i & 15)] = float_to_bits<BF>(y);
  }
}

template <int BITS, bool BF>
hipError_t launch_bits(const MoeKernelArgs& p, hipStream_t stream) {
  gate_up_kernel<BITS, BF><<<dim3(p.a.I / 16, p.slots.count), 64 * kGateWaves, 0, stream>>>(p);
  down_kernel<BITS, BF><<<p.a.H / 16, 64 * kDownWaves, (size_t)kDownWaves * p.a.T * 16 * 4, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

size_t moe_route_workspace(int T, int H, int E) { return kWorkspaceHeader; }

hipError_t launch_moe_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid((unsigned)(a.E + 15) / 16, (unsigned)(a.T + 15) / 16);
  if (bf16) route_kernel<true><<<grid, 64 * kRouteWaves, 0, stream>>>(a);
  else route_kernel<false><<<grid, 64 * kRouteWaves, 0, stream>>>(a);
  return hipGetLastError();
}

size_t moe_workspace(int T, int H, int I, int E, int top_k) {
  const size_t slots = cmin(E, T * top_k);
  return kWorkspaceHeader + (size_t)T * top_k * I * 4 + slots * 4 + slots * T * 2;
}

hipError_t launch_moe(const MoeArgs& a, int bits, bool bf16, bool strips, hipStream_t stream) {
  MoeKernelArgs p = {a, {}, nullptr, strips};
  p.slots.count = cmin(a.E, a.T * a.top_k);
  char* at = a.workspace + kWorkspaceHeader;
  p.h = reinterpret_cast<uint16_t*>(at);
  at += (size_t)a.T * a.top_k * a.I * 4;
  p.slots.rows = reinterpret_cast<int*>(at);
  p.slots.list = reinterpret_cast<uint16_t*>(at + (size_t)p.slots.count * 4);
  switch (bits) {
    case 1: return bf16 ? launch_bits<1, true>(p, stream) : launch_bits<1, false>(p, stream);
    case 2: return bf16 ? launch_bits<2, true>(p, stream) : launch_bits<2, false>(p, stream);
    case 3: return bf16 ? launch_bits<3, true>(p, stream) : launch_bits<3, false>(p, stream);
    case 4: return bf16 ? launch_bits<4, true>(p, stream) : launch_bits<4, false>(p, stream);
    default: return bf16 ? launch_bits<8, true>(p, stream) : launch_bits<8, false>(p, stream);
  }
}

}  // namespace qmm
