// The mixture-of-experts layer with quantised experts for a few tokens.
#include "layer.h"

namespace qmm {
namespace {

// ---- routing -------------------------------------------------------------------

// One wave per logit.
template <bool BF>
__global__ void __launch_bounds__(64) route_logits_kernel(RouteArgs a) {
  const int e = blockIdx.x, t = blockIdx.y, lane = threadIdx.x;
  float s = 0;
  for (int h = lane; h < a.H; h += 64)
    s += bits_to_float<BF>(a.x[(long long)t * a.H + h]) * bits_to_float<BF>(a.router[(long long)e * a.H + h]);
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0) a.logits[(long long)t * a.E + e] = s;
}

// A total order: larger logits first, NaN above all, equal ones by the lower expert.
__device__ __forceinline__ uint64_t route_key(float l, int e) {
  uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);  // -0 counts as 0
  b = l != l ? 0xFFFFFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return (uint64_t)b << 32 | (uint32_t)~e;
}

// One wave per token.
__global__ void __launch_bounds__(64) route_top_kernel(RouteArgs a) {
  const int t = blockIdx.x, lane = threadIdx.x;
  const float* l = a.logits + (long long)t * a.E;
  uint64_t below = ~0ull;
  float mx = 0, sum = 0, mine = 0;
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t best = 0;
    for (int e = lane; e < a.E; e += 64) {
      const uint64_t k = route_key(l[e], e);
      if (k < below && k > best) best = k;
    }
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t w = __shfl_xor(best, o);
      best = w > best ? w : best;
    }
    below = best;
    const int e = (int)~(uint32_t)best;
    if (j == 0) mx = l[e];
    const float p = __expf(l[e] - mx);
    sum += p;
    if (lane == j) mine = p;
    if (lane == 0) a.ids[t * a.top_k + j] = e;
  }
  if (!a.renormalize) {
    sum = 0;
    for (int e = lane; e < a.E; e += 64) sum += __expf(l[e] - mx);
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  }
  if (lane < a.top_k) a.weights[t * a.top_k + lane] = mine / sum;
}

// ---- the experts' products ---------------------------------------------------------

// Code (k, n) of an expert's plane.
template <int BITS>
__device__ __forceinline__ int code_at(const uint32_t* qw, const uint32_t* qlo, int K, int N, int strips, int k, int n) {
  if constexpr (BITS == 3) {
    const int hi = (int)(qw[plane_col(n, K / 16, strips) + (uint32_t)(k / 16) * plane_row_stride(N, strips)] >> (2 * (k % 16))) & 3;
    const int lo = (int)(qlo[plane_col(n, K / 32, strips) + (uint32_t)(k / 32) * plane_row_stride(N, strips)] >> (k % 32)) & 1;
    return 2 * hi + lo;
  } else {
    constexpr int EPS = 32 / BITS;
    return (int)(qw[plane_col(n, K / EPS, strips) + (uint32_t)(k / EPS) * plane_row_stride(N, strips)] >> (BITS * (k % EPS))) &
           ((1 << BITS) - 1);
  }
}

// Column n of (row of K floats or 16-bit values) @ dequantize(expert e).
template <int BITS, bool BF, typename X>
__device__ __forceinline__ float expert_column(const X* x, const ExpertPlanes& w, int e, int K, int N, int gs, int strips, int n) {
  constexpr int HI = BITS == 3 ? 2 : BITS;
  const uint32_t* qw = w.qw + (size_t)e * (K * HI / 32) * N;
  const uint32_t* qlo = BITS == 3 ? w.qlo + (size_t)e * (K / 32) * N : nullptr;
  const size_t groups = K / gs;
  float total = 0;
  for (int g = 0; g < (int)groups; ++g) {
    const float z = bits_to_float<BF>(w.zeros[(e * groups + g) * N + n]), s = bits_to_float<BF>(w.scales[(e * groups + g) * N + n]);
    float acc = 0;
    for (int k = g * gs; k < (g + 1) * gs; ++k) {
      float xv;
      if constexpr (sizeof(X) == 2) xv = bits_to_float<BF>(x[k]);
      else xv = x[k];
      acc += xv * ((float)code_at<BITS>(qw, qlo, K, N, strips, k, n) - z);
    }
    total += s * acc;
  }
  return total;
}

template <int BITS, bool BF>
__global__ void __launch_bounds__(64) gate_up_kernel(MoeArgs a, float* h, int strips) {
  const int n = blockIdx.x * 64 + threadIdx.x, at = blockIdx.y, e = a.ids[at];
  if (n >= a.I || e < 0 || e >= a.E) return;
  const uint16_t* x = a.x + (long long)(at / a.top_k) * a.H;
  const float g = expert_column<BITS, BF>(x, a.gate_up, e, a.H, 2 * a.I, a.gs_h, strips, n);
  const float u = expert_column<BITS, BF>(x, a.gate_up, e, a.H, 2 * a.I, a.gs_h, strips, n + a.I);
  h[(long long)at * a.I + n] = g / (1 + __expf(-g)) * u;
}

template <int BITS, bool BF>
__global__ void __launch_bounds__(64) down_kernel(MoeArgs a, const float* h, int strips) {
  const int n = blockIdx.x * 64 + threadIdx.x, t = blockIdx.y;
  if (n >= a.H) return;
  float y = 0;
  for (int j = 0; j < a.top_k; ++j) {
    const int at = t * a.top_k + j, e = a.ids[at];
    if (e < 0 || e >= a.E) continue;
    y += a.weights[at] * expert_column<BITS, BF>(h + (long long)at * a.I, a.down, e, a.I, a.H, a.gs_i, strips, n);
  }
  a.y[(long long)t * a.H + n] = float_to_bits<BF>(y);
}

template <int BITS, bool BF>
hipError_t launch_bits(const MoeArgs& a, bool strips, hipStream_t stream) {
  float* h = reinterpret_cast<float*>(a.workspace + kWorkspaceHeader);
  gate_up_kernel<BITS, BF><<<dim3((a.I + 63) / 64, a.T * a.top_k), 64, 0, stream>>>(a, h, strips);
  down_kernel<BITS, BF><<<dim3((a.H + 63) / 64, a.T), 64, 0, stream>>>(a, h, strips);
  return hipGetLastError();
}

}  // namespace

size_t moe_route_workspace(int T, int H, int E) { return kWorkspaceHeader; }

hipError_t launch_moe_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid((unsigned)a.E, (unsigned)a.T);
  if (bf16) route_logits_kernel<true><<<grid, 64, 0, stream>>>(a);
  else route_logits_kernel<false><<<grid, 64, 0, stream>>>(a);
  route_top_kernel<<<a.T, 64, 0, stream>>>(a);
  return hipGetLastError();
}

size_t moe_workspace(int T, int H, int I, int E, int top_k) { return kWorkspaceHeader + (size_t)T * top_k * I * 4; }

hipError_t launch_moe(const MoeArgs& a, int bits, bool bf16, bool strips, hipStream_t stream) {
  switch (bits) {
    case 1: return bf16 ? launch_bits<1, true>(a, strips, stream) : launch_bits<1, false>(a, strips, stream);
    case 2: return bf16 ? launch_bits<2, true>(a, strips, stream) : launch_bits<2, false>(a, strips, stream);
    case 3: return bf16 ? launch_bits<3, true>(a, strips, stream) : launch_bits<3, false>(a, strips, stream);
    case 4: return bf16 ? launch_bits<4, true>(a, strips, stream) : launch_bits<4, false>(a, strips, stream);
    default: return bf16 ? launch_bits<8, true>(a, strips, stream) : launch_bits<8, false>(a, strips, stream);
  }
}

}  // namespace qmm
