// The mixture-of-experts layer with quantised experts for a few tokens: the
// routing, then one launch for the gate and up products with the gating, and one
// for the down products with the weighted sum.
//
// An assignment is a (token, choice) pair, t * top_k + j. A group's part of a
// product is s (sum_k x q - z sum_k x): codes go to the matrix cores as they are,
// the scale and zero point are applied to the sums.
#include "fixed_div.h"
#include "gemv_common.h"
#include "handoff.h"
#include "layer.h"
#include "mfma.h"

namespace qmm {
namespace {

// ---- routing -------------------------------------------------------------------

constexpr int kRouteBatch = 8;  // units of H whose loads a wave has on the way together

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
// ends a token tile's logits chooses for its tokens (a choice per block would need the
// logits of all). Bound: latency, a few hundred KiB of router weights over few CUs:
// 7.0 us at one token, H 2048, 64 experts; 10.4 us at 13 tokens, H 4096, 32 experts.
template <bool BF, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) route_kernel(RouteArgs a) {
  __shared__ float part[WAVES][16][17];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = lane & 15, kg = lane >> 4;
  const int e = min((int)blockIdx.x * 16 + n, a.E - 1), t0 = blockIdx.y * 16, t = min(t0 + n, a.T - 1);
  const u32x4* x = reinterpret_cast<const u32x4*>(a.x + (size_t)t * a.H + kg * 8);
  const u32x4* r = reinterpret_cast<const u32x4*>(a.router + (size_t)e * a.H + kg * 8);
  f32x4 acc = {};
  const int units = a.H / 32;
  for (int u0 = wave; u0 < units; u0 += kRouteBatch * WAVES) {
    u32x4 xv[kRouteBatch], rv[kRouteBatch];
#pragma unroll
    for (int i = 0; i < kRouteBatch; ++i) {
      const int u = min(u0 + i * WAVES, units - 1);
      xv[i] = x[u * 4];
      rv[i] = r[u * 4];
    }
#pragma unroll
    for (int i = 0; i < kRouteBatch; ++i)
      if (u0 + i * WAVES < units) acc = mfma16<BF>(xv[i], rv[i], acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][4 * kg + i][n] = acc[i];
  __syncthreads();
  if (tid < 256) {
    const int row = tid >> 4, col = tid & 15;
    float s = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += part[w][row][col];
    if (t0 + row < a.T && (int)blockIdx.x * 16 + col < a.E)
      handoff_store(&a.logits[(size_t)(t0 + row) * a.E + blockIdx.x * 16 + col], s);
  }
  if (!handoff_last(&a.counters[blockIdx.y], gridDim.x, &s_last)) return;
  for (int i = t0 + wave; i < min(t0 + 16, a.T); i += WAVES) {
    if (a.E <= 64) route_top<1>(a, i, lane);
    else if (a.E <= 128) route_top<2>(a, i, lane);
    else if (a.E <= 256) route_top<4>(a, i, lane);
    else route_top<16>(a, i, lane);
  }
}

// ---- codes as matrix operands --------------------------------------------------------

// Eight codes of lane group j, in decode8's element order, as 16-bit numbers. bf16:
// 128 + q for up to 4 bits (the code in the mantissa's low bits), q for 8 bits (exact in
// 8 significant bits). fp16: q 2^(kPlace - 24), the code at bits kPlace on of a half whose
// bits up to 10 read as a plain number (subnormals, and the first normals behind them).
//
// The matrix cores place a product by its operands' exponent fields: of the products of
// a subnormal with nine leading zeros nine bits are cut off at the far end, always
// downwards (sums of 4096 products with codes 0 and 1 at 2^-24: 4.6e-5 off, all to one
// side; at 2^-20 4.2e-7; at 2^-15 and above 7e-8, a rounding in fp32). So the code goes
// as far up as it gets without another operation, and at the top for the narrow ones.
//
// The masks are made once and kept in vector registers, the bits put around the code
// (nothing for fp16) in a scalar one, so that inserting is one operation.
template <int BITS, bool BF> constexpr int kPlace = BF || BITS == 8 ? 0 : BITS == 4 ? 4 : 11 - BITS;
template <int BITS, bool BF> struct CodeMasks {
  uint32_t code, low, around;
  __device__ __forceinline__ CodeMasks()
      : code((BITS == 4 ? 0x000F000Fu : BITS == 3 ? 0x00060006u : BITS == 2 ? 0x00030003u : 0x00010001u) << kPlace<BITS, BF>),
        low(0x00010001u << kPlace<BITS, BF>), around(BF ? 0x43004300u : 0u) {
    if (BITS != 8) asm("" : "+v"(code));
    if (BITS == 3) asm("" : "+v"(low));
    if (BF && BITS != 8) asm("" : "+s"(around));
  }
};
__device__ __forceinline__ uint32_t rotate_right(uint32_t w, int n) { return __builtin_amdgcn_alignbit(w, w, (uint32_t)n); }  // by n mod 32
// w moved up by n bits, down for n < 0.
__device__ __forceinline__ uint32_t moved_up(uint32_t w, int n) { return n >= 0 ? w << n : w >> -n; }
template <int BITS, bool BF>
__device__ __forceinline__ u32x4 codes8(uint32_t w0, uint32_t w1, int j, const CodeMasks<BITS, BF>& m) {
  constexpr int PLACE = kPlace<BITS, BF>;
  u32x4 b;
  if constexpr (BITS == 4) {
#pragma unroll
    for (int p = 0; p < 4; ++p) b[p] = (moved_up(w0, PLACE - 4 * p) & m.code) | m.around;
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
    // Pair p at bits 2 p of t, or (fp16) 2 p + 3: pair 3 is where it goes then.
    const uint32_t t = BF ? w0 >> (8 * (j & 1)) : rotate_right(w0, 8 * (j & 1) - 3);
#pragma unroll
    for (int p = 0; p < 4; ++p) b[p] = (moved_up(t, BF ? -2 * p : 6 - 2 * p) & m.code) | m.around;
  } else if constexpr (BITS == 3) {
    const uint32_t h = BF ? w0 >> (8 * (j & 1)) : rotate_right(w0, 8 * (j & 1) - 3);
    const uint32_t t = w1 >> (16 * (j >> 1) + 4 * (j & 1));
    const uint32_t l = __builtin_amdgcn_perm(0u, t, BF ? 0x0C010C00u : 0x010C000Cu);  // byte 0 of t in one half, 1 in the other
#pragma unroll
    for (int p = 0; p < 4; ++p) b[p] = ((l >> p) & m.low) | ((moved_up(h, BF ? 1 - 2 * p : 6 - 2 * p) & m.code) | m.around);
  } else {
    // Slots p and p + 4 sixteen bits apart, p at bit p, or (fp16) 7 + p.
    const uint32_t t = BF ? (w0 >> (8 * j)) & 0xFFu : rotate_right(w0, 8 * j - 7) & 0x7F80u, both = t | (t << 12);
#pragma unroll
    for (int p = 0; p < 4; ++p) b[p] = (moved_up(both, BF ? -p : 3 - p) & m.code) | m.around;
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

// One expert's weight (K x N) as its kernels address it: byte offsets are 32-bit,
// a lane's part of them fixed, a unit's part uniform.
template <int BITS> struct ExpertView {
  __amdgpu_buffer_rsrc_t hi, lo, scales, zeros;
  int N, rows, rows_lo, stride;  // word rows per plane, words per row step
  int strips;
};
template <int BITS>
__device__ __forceinline__ ExpertView<BITS> expert_view(const ExpertPlanes& w, int e, int K, int N, int groups, int strips) {
  ExpertView<BITS> v;
  v.N = N;
  v.rows = K * (BITS == 3 ? 2 : BITS) / 32;
  v.rows_lo = K / 32;
  v.stride = plane_row_stride(N, strips);
  v.strips = strips;
  const size_t plane = (size_t)v.rows * N, plane_lo = (size_t)v.rows_lo * N, params = (size_t)groups * N;
  v.hi = make_rsrc(w.qw + e * plane, plane * 4);
  v.lo = BITS == 3 ? make_rsrc(w.qlo + e * plane_lo, plane_lo * 4) : v.hi;
  v.scales = make_rsrc(w.scales + e * params, params * 2);
  v.zeros = make_rsrc(w.zeros + e * params, params * 2);
  return v;
}

// A chunk: four units (32 k each) of one column strip, and the scale and zero point
// of lane group j's unit for this lane's column. A wave keeps a run of chunks in
// registers (16 words a lane) and asks for a chunk's successor as it has used it.
constexpr int kUnits = 4;
template <int BITS> constexpr int kRun = 4 / Bits<BITS>::NW;
template <int BITS> struct Chunk {
  uint32_t w[kUnits][Bits<BITS>::NW];
  uint16_t scale, zero;
};

// Chunk c of column col; units past the last repeat it.
template <int BITS>
__device__ __forceinline__ void load_chunk(Chunk<BITS>& r, const ExpertView<BITS>& v, int col, int c, int units, FixedDiv by_upg, int j) {
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t u = (uint32_t)min(c * kUnits + i, units - 1);
#pragma unroll
    for (int x = 0; x < Bits<BITS>::NW; ++x) {
      const bool low = BITS == 3 && x == 1;
      const uint32_t lane = 4u * (plane_col(col, low ? v.rows_lo : v.rows, v.strips) + (uint32_t)lane_row<BITS>(j, x) * (uint32_t)v.stride);
      r.w[i][x] = __builtin_amdgcn_raw_buffer_load_b32(low ? v.lo : v.hi, lane, u * (uint32_t)(4 * unit_rows<BITS>(x)) * (uint32_t)v.stride,
                                                       kNonTemporal);
    }
  }
  const uint32_t at = 2u * ((uint32_t)by_upg(min(c * kUnits + j, units - 1)) * (uint32_t)v.N + (uint32_t)col);
  r.scale = __builtin_amdgcn_raw_buffer_load_b16(v.scales, at, 0, 0);
  r.zero = __builtin_amdgcn_raw_buffer_load_b16(v.zeros, at, 0, 0);
}

// Where groups end within a chunk: every kUnits or kUnits / 2 units, known at
// compile time, or anywhere.
enum Groups { kWholeChunk, kHalfChunk, kAnywhere };
inline Groups groups_of(int upg) { return upg % kUnits == 0 ? kWholeChunk : upg == kUnits / 2 ? kHalfChunk : kAnywhere; }

// total += a (16 rows) @ dequantize(chunk) for COLS strips' chunks; units past the
// last must be 0 in a. BF: of the operands; SBF: of the scales and zero points.
template <int BITS, bool BF, bool SBF, int COLS, Groups G>
__device__ __forceinline__ void chunk_product(f32x4 (&total)[COLS], const u32x4 (&a)[kUnits], const Chunk<BITS>* const (&w)[COLS], int c,
                                              int upg, FixedDiv by_upg, int j, int n, const CodeMasks<BITS, BF>& masks) {
  constexpr uint32_t kOne = BF ? 0x3F803F80u : 0x3C003C00u;
  constexpr float kUp = BF ? 1.f : 1 << (24 - kPlace<BITS, BF>);
  f32x4 acc[COLS] = {}, as = {};
  int in_group = G == kAnywhere ? c * kUnits - by_upg(c * kUnits) * upg : 0;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    as = mfma16<BF>(a[i], u32x4{kOne, kOne, kOne, kOne}, as);
#pragma unroll
    for (int v = 0; v < COLS; ++v)
      acc[v] = mfma16<BF>(a[i], codes8<BITS, BF>(w[v]->w[i][0], w[v]->w[i][Bits<BITS>::NW - 1], j, masks), acc[v]);
    // The end of a group or of the chunk: scale and zero point, from the lane group that
    // holds the unit's (its own where the chunk is of one group).
    if (G == kWholeChunk ? i == kUnits - 1 : G == kHalfChunk ? i % 2 == 1 : ++in_group == upg || i == kUnits - 1) {
      in_group = 0;
#pragma unroll
      for (int v = 0; v < COLS; ++v) {
        float sc = bits_to_float<SBF>(w[v]->scale), z = bits_to_float<SBF>(w[v]->zero);
        if constexpr (G != kWholeChunk) {
          const uint32_t sz = __shfl((uint32_t)w[v]->scale | (uint32_t)w[v]->zero << 16, 16 * i + n);
          sc = bits_to_float<SBF>((uint16_t)sz);
          z = bits_to_float<SBF>((uint16_t)(sz >> 16));
        }
        z += kCodeOffset<BITS, BF>;
#pragma unroll
        for (int r = 0; r < 4; ++r) total[v][r] += sc * (acc[v][r] * kUp - z * as[r]);
        acc[v] = f32x4{};
      }
      as = f32x4{};
    }
  }
}

// Zeroes a chunk's operands of units past the last.
__device__ __forceinline__ void cut_units(u32x4 (&a)[kUnits], int c, int units) {
  if ((c + 1) * kUnits > units) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (c * kUnits + i >= units) a[i] = u32x4{0, 0, 0, 0};
  }
}

// ---- gate and up products --------------------------------------------------------------

constexpr int kGateWaves = 4;
static_assert(64 * kGateWaves == 256, "a thread per element of a block's result");

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
  FixedDiv by_upg_h, by_upg_i, by_top_k, by_runs;  // units per group of both products; choices per token; runs per expert of the second
  Slots slots;
  uint16_t* h;  // (assignments, 2, I) bf16: high and low parts, each unit in operand order
  int strips;
};

// The 16 assignments from `base` on.
template <int BITS, bool BF, Groups G>
__device__ __forceinline__ void gate_up_rows(const MoeKernelArgs& p, int e, int strip, const uint16_t* list, int base, int rows,
                                             float (*sums)[2][16][17]) {
  const MoeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, j = lane >> 4;
  const int units = a.H / 32, upg = a.gs_h / 32, chunks = (units + kUnits - 1) / kUnits;
  const ExpertView<BITS> view = expert_view<BITS>(a.gate_up, e, a.H, 2 * a.I, p.by_upg_h(units), p.strips);
  Chunk<BITS> run[kRun<BITS>][2];
  auto load_words = [&](int k, int c) {
#pragma unroll
    for (int v = 0; v < 2; ++v) load_chunk<BITS>(run[k][v], view, v * a.I + strip * 16 + n, min(c, chunks - 1), units, p.by_upg_h, j);
  };
#pragma unroll
  for (int k = 0; k < kRun<BITS>; ++k)
    if (wave + k * kGateWaves < chunks) load_words(k, wave + k * kGateWaves);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (size_t)a.T * a.H * 2);
  const uint32_t x = 2u * ((uint32_t)p.by_top_k(list[min(base + n, rows - 1)]) * (uint32_t)a.H + (uint32_t)x_first<BITS>(j));
  u32x4 xv[kUnits];
  auto load_x = [&](int c, u32x4 (&to)[kUnits]) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t u = (uint32_t)min(c * kUnits + i, units - 1) * 64u;
      if constexpr (BITS == 2 || BITS == 3) {
        const u32x2 lo = __builtin_amdgcn_raw_buffer_load_b64(xr, x, u, 0), hi = __builtin_amdgcn_raw_buffer_load_b64(xr, x + 16, u, 0);
        to[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
      } else {
        to[i] = __builtin_amdgcn_raw_buffer_load_b128(xr, x, u, 0);
      }
    }
  };
  const CodeMasks<BITS, BF> masks;
  f32x4 total[2] = {};
  int c = wave;
  if (c < chunks) load_x(c, xv);
  while (c < chunks) {
#pragma unroll
    for (int k = 0; k < kRun<BITS>; ++k) {
      if (c >= chunks) break;
      u32x4 xa[kUnits];
#pragma unroll
      for (int i = 0; i < kUnits; ++i) xa[i] = x_operand<BITS>(xv[i]);
      cut_units(xa, c, units);
      const Chunk<BITS>* const w[2] = {&run[k][0], &run[k][1]};
      chunk_product<BITS, BF, BF, 2, G>(total, xa, w, c, upg, p.by_upg_h, j, n, masks);
      __builtin_amdgcn_sched_barrier(0);
      load_x(c + kGateWaves, xv);
      if (c + kRun<BITS> * kGateWaves < chunks) load_words(k, c + kRun<BITS> * kGateWaves);
      __builtin_amdgcn_sched_barrier(0);
      c += kGateWaves;
    }
  }
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int r = 0; r < 4; ++r) sums[wave][v][4 * j + r][n] = total[v][r];
  __syncthreads();
  if (base + (tid >> 4) < rows) {  // a thread per element of 16 x 16
    const int row = tid >> 4, cc = tid & 15;
    float g = 0, u = 0;
#pragma unroll
    for (int w = 0; w < kGateWaves; ++w) g += sums[w][0][row][cc], u += sums[w][1][row][cc];
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

// Block: 16 gate and the 16 up columns of one expert, its waves over H; both, so that
// the gating is the epilogue. An expert's words are read once per 16 of its tokens
// (from the L2 after the first). Four waves: twice the blocks of eight, whose starts
// and ends overlap better (13 tokens 49.8 -> 43.8 us). Bound: HBM in principle; the
// vector ALUs are half busy with codes and addresses. 13 tokens, 32 experts of 4096 x
// 2560 at 4 bits: 43.6 us, 3.6 TB/s; 64 tokens, 16 of 4096 x 2816 at 3 bits: 47.6 us.
template <int BITS, bool BF, Groups G>
__global__ void __launch_bounds__(64 * kGateWaves, 4) gate_up_kernel(MoeKernelArgs p) {
  __shared__ float sums[kGateWaves][2][16][17];
  __shared__ uint16_t list[kMoeTokens];
  __shared__ int counts[2][kGateWaves];
  const MoeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, strip = blockIdx.x, slot = blockIdx.y;
  const int assignments = a.T * a.top_k;
  const bool by_assignment = p.slots.count == assignments;
  const int e = by_assignment ? a.ids[slot] : slot;
  int rows = 0;
  if (a.T == 1 && by_assignment) {  // one token: every choice an expert of its own
    rows = e >= 0 && e < a.E;
    if (tid == 0) {
      list[0] = (uint16_t)slot;
      if (strip == 0) {
        p.slots.rows[slot] = rows;
        p.slots.list[slot] = (uint16_t)slot;
      }
    }
    __syncthreads();
  } else {
    // The expert's assignments, in order; a slot whose expert came before is not in use.
    bool dup = false;
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
    const bool unused = __syncthreads_or(dup) || e < 0 || e >= a.E;
    rows = unused ? 0 : min(rows, a.T);
    if (strip == 0) {
      if (tid == 0) p.slots.rows[slot] = rows;
      if (tid < rows) p.slots.list[(size_t)slot * a.T + tid] = list[tid];
    }
  }
  for (int base = 0; base < rows; base += 16) gate_up_rows<BITS, BF, G>(p, e, strip, list, base, rows, sums);
}

// ---- down products and the weighted sum ---------------------------------------------------

constexpr int kDownWaves = 16;

// Block: 16 columns of y for all tokens; its waves take (expert, run of chunks)
// pairs in turn, the next one's words on the way as the current ones are used, and
// add to sums of their own, which meet in wave order. A row tile is 8 assignments: the high
// parts of h in rows 0-7, the low parts in rows 8-15. Bound: as above, and
// latency at one token. One token, 8 experts of 1024 x 2048 at 4 bits: 9.6 us; 13 tokens,
// 32 of 1280 x 4096: 34.8 us, 2.2 TB/s; 64 tokens, 16 of 1408 x 4096 at 3 bits: 40.3 us.
template <int BITS, bool BF, Groups G>
__global__ void __launch_bounds__(64 * kDownWaves) down_kernel(MoeKernelArgs p) {
  extern __shared__ float sums[];  // (waves, T, 16)
  __shared__ uint16_t used_slot[kMoeExperts], used_expert[kMoeExperts], used_first[kMoeExperts + 1], list[kMoeAssignments];
  __shared__ float weight[kMoeAssignments];
  __shared__ int s_used;
  const MoeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15, j = lane >> 4;
  const int strip = blockIdx.x, units = a.I / 32, upg = a.gs_i / 32, chunks = (units + kUnits - 1) / kUnits;
  const int runs = (chunks + kRun<BITS> - 1) / kRun<BITS>;
  const bool by_assignment = p.slots.count == a.T * a.top_k;
  // The slots in use, their experts and assignments (used_first[u] on in the list), all in LDS.
  for (int i = tid; i < a.T * a.top_k; i += 64 * kDownWaves) weight[i] = a.weights[i];
  if (wave == 0) {
    int total = 0, first = 0;
    for (int base = 0; base < p.slots.count; base += 64) {
      const int slot = base + lane;
      const bool in = slot < p.slots.count;
      const int e = !in ? -1 : by_assignment ? a.ids[slot] : slot;
      int rows = !in ? 0 : p.slots.rows[slot], upto = rows;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int before = __shfl_up(upto, o);
        if (lane >= o) upto += before;
      }
      const uint64_t hits = __ballot(rows > 0);
      if (rows > 0) {
        const int u = total + __builtin_popcountll(hits & ((1ull << lane) - 1));
        used_slot[u] = (uint16_t)slot;
        used_expert[u] = (uint16_t)e;
        used_first[u] = (uint16_t)(first + upto - rows);
      }
      total += __builtin_popcountll(hits);
      first += __shfl(upto, 63);
    }
    if (lane == 0) {
      s_used = total;
      used_first[total] = (uint16_t)first;
    }
  }
  float* mine = sums + (size_t)wave * a.T * 16;
  for (int i = lane; i < a.T * 16; i += 64) mine[i] = 0;
  __syncthreads();
  for (int u = wave; u < s_used; u += kDownWaves) {
    const int first = used_first[u];
    if (lane < used_first[u + 1] - first) list[first + lane] = p.slots.list[(size_t)used_slot[u] * a.T + lane];
  }
  // Items: runs of one expert's chunks.
  const int items = s_used * runs;
  struct Item {
    int u, c0;
  };
  auto item = [&](int it) {
    const int u = p.by_runs(it);
    return Item{u, (it - u * runs) * kRun<BITS>};
  };
  Chunk<BITS> run[kRun<BITS>];
  auto load = [&](int k, const Item& x) {
    const int e = __builtin_amdgcn_readfirstlane(used_expert[x.u]);
    load_chunk<BITS>(run[k], expert_view<BITS>(a.down, e, a.I, a.H, p.by_upg_i(units), p.strips), strip * 16 + n,
                     min(x.c0 + k, chunks - 1), units, p.by_upg_i, j);
  };
  int it = wave;
  Item x = item(min(it, max(items - 1, 0)));
  if (it < items) {
#pragma unroll
    for (int k = 0; k < kRun<BITS>; ++k) load(k, x);
  }
  __syncthreads();
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(p.h, (size_t)a.T * a.top_k * a.I * 4);
  const CodeMasks<BITS, true> masks;
  // h of chunk c for the 8 assignments from `at` on of an item.
  auto load_h = [&](const Item& x, int base, int c, u32x4 (&h)[kUnits]) {
    const int first = used_first[x.u], rows = used_first[x.u + 1] - first;
    const uint32_t as = list[first + min(base + (n & 7), rows - 1)];
    const uint32_t off = 2u * ((as * 2u + (uint32_t)(n >> 3)) * (uint32_t)a.I + (uint32_t)j * 8u);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) h[i] = __builtin_amdgcn_raw_buffer_load_b128(hr, off, (uint32_t)min(c * kUnits + i, units - 1) * 64u, 0);
  };
  u32x4 ha[kUnits];
  if (it < items) load_h(x, 0, x.c0, ha);
  for (; it < items; it += kDownWaves) {
    const Item next = item(min(it + kDownWaves, items - 1));
    const int first = used_first[x.u], rows = used_first[x.u + 1] - first;
#pragma unroll
    for (int k = 0; k < kRun<BITS>; ++k) {
      const int c = x.c0 + k;
      if (c < chunks) {
        for (int base = 0; base < rows; base += 8) {
          if (base > 0) load_h(x, base, c, ha);
          cut_units(ha, c, units);
          f32x4 total[1] = {};
          const Chunk<BITS>* const w[1] = {&run[k]};
          chunk_product<BITS, true, BF, 1, G>(total, ha, w, c, upg, p.by_upg_i, j, n, masks);
          // Rows 4 j + r of lanes j < 2 are the high parts, of lanes j + 2 the low ones.
#pragma unroll
          for (int r = 0; r < 4; ++r) total[0][r] += __shfl_xor(total[0][r], 32);
          if (j < 2) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (base + 4 * j + r < rows) {
                const int as = list[first + base + 4 * j + r];
                mine[p.by_top_k(as) * 16 + n] += weight[as] * total[0][r];
              }
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (k + 1 < kRun<BITS>) load_h(x, 0, min(c + 1, chunks - 1), ha);
      else load_h(next, 0, next.c0, ha);
      load(k, next);
      __builtin_amdgcn_sched_barrier(0);
    }
    x = next;
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
  const dim3 gate_grid(p.a.I / 16, p.slots.count), down_grid(p.a.H / 16);
  const size_t lds = (size_t)kDownWaves * p.a.T * 16 * 4;
  const auto run = [&](auto gate, auto down) {
    gate<<<gate_grid, 64 * kGateWaves, 0, stream>>>(p);
    down<<<down_grid, 64 * kDownWaves, lds, stream>>>(p);
  };
  const auto down_for = [&](auto gate) {
    switch (groups_of(p.a.gs_i / 32)) {
      case kWholeChunk: return run(gate, down_kernel<BITS, BF, kWholeChunk>);
      case kHalfChunk: return run(gate, down_kernel<BITS, BF, kHalfChunk>);
      default: return run(gate, down_kernel<BITS, BF, kAnywhere>);
    }
  };
  switch (groups_of(p.a.gs_h / 32)) {
    case kWholeChunk: down_for(gate_up_kernel<BITS, BF, kWholeChunk>); break;
    case kHalfChunk: down_for(gate_up_kernel<BITS, BF, kHalfChunk>); break;
    default: down_for(gate_up_kernel<BITS, BF, kAnywhere>); break;
  }
  return hipGetLastError();
}

}  // namespace

size_t moe_route_workspace(int T, int H, int E) { return kWorkspaceHeader; }

hipError_t launch_moe_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid((unsigned)(a.E + 15) / 16, (unsigned)(a.T + 15) / 16);
  // Eight waves where a batch of each covers H, else sixteen (whose join takes longer:
  // 7.0 against 9.3 us at one token and H 2048, 11.7 against 10.4 at 13 and 4096).
  const bool few = a.H <= 8 * 32 * kRouteBatch;
  if (bf16 && few) route_kernel<true, 8><<<grid, 512, 0, stream>>>(a);
  else if (bf16) route_kernel<true, 16><<<grid, 1024, 0, stream>>>(a);
  else if (few) route_kernel<false, 8><<<grid, 512, 0, stream>>>(a);
  else route_kernel<false, 16><<<grid, 1024, 0, stream>>>(a);
  return hipGetLastError();
}

size_t moe_workspace(int T, int H, int I, int E, int top_k) {
  const size_t slots = cmin(E, T * top_k);
  return kWorkspaceHeader + (size_t)T * top_k * I * 4 + slots * 4 + slots * T * 2;
}

hipError_t launch_moe(const MoeArgs& a, int bits, bool bf16, bool strips, hipStream_t stream) {
  const int run = 4 / (bits == 3 || bits == 8 ? 2 : 1), chunks = (a.I / 32 + 3) / 4;
  MoeKernelArgs p = {a, fixed_div(a.gs_h / 32), fixed_div(a.gs_i / 32), fixed_div(a.top_k), fixed_div((chunks + run - 1) / run), {}, nullptr, strips};
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
