// Log probabilities of given tokens, entropy and the largest alternatives of
// rows of logits. lse = m + ln S with m = max l, S = sum e^(l - m); entropy =
// ln S - sum e^(l - m) (l - m) / S.
#include "layer.h"

namespace qmm {
namespace {

template <LogitType TYPE>
__device__ __forceinline__ float load_logit(const void* row, long long i) {
  if constexpr (TYPE == LogitType::kFp32) return static_cast<const float*>(row)[i];
  else return bits_to_float<TYPE == LogitType::kBf16>(static_cast<const uint16_t*>(row)[i]);
}

// A total order: larger logits first, NaN above all, equal ones by index.
__device__ __forceinline__ uint64_t order_key(float l, int index) {
  uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);  // -0 counts as 0
  b = l != l ? 0xFFFFFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return (uint64_t)b << 32 | (uint32_t)~index;
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor(v, o);
    v = w > v ? w : v;
  }
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// One block per row: a pass for the maximum, one for the sums, one per alternative.
template <LogitType TYPE>
__global__ void __launch_bounds__(256) logprobs_kernel(LogprobArgs a) {
  __shared__ uint64_t keys[4];
  __shared__ float sums[2][4];
  const int m = blockIdx.x, tid = threadIdx.x, wave = tid >> 6;
  const char* row = static_cast<const char*>(a.logits) + (long long)m * a.row_stride * (TYPE == LogitType::kFp32 ? 4 : 2);
  auto block_largest = [&](uint64_t below) {
    uint64_t best = 0;
    for (int i = tid; i < a.V; i += 256) {
      const uint64_t k = order_key(load_logit<TYPE>(row, i), i);
      if (k < below && k > best) best = k;
    }
    best = wave_max(best);
    __syncthreads();
    if ((tid & 63) == 0) keys[wave] = best;
    __syncthreads();
    best = keys[0];
    for (int w = 1; w < 4; ++w) best = keys[w] > best ? keys[w] : best;
    return best;
  };
  const uint64_t first = block_largest(~0ull);
  const float mx = load_logit<TYPE>(row, (int)~(uint32_t)first);
  float s = 0, e = 0;
  for (int i = tid; i < a.V; i += 256) {
    const float d = load_logit<TYPE>(row, i) - mx, p = __expf(d);
    s += p;
    if (d != -INFINITY) e += p * d;
  }
  s = wave_sum(s);
  e = wave_sum(e);
  if ((tid & 63) == 0) sums[0][wave] = s, sums[1][wave] = e;
  __syncthreads();
  s = sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3];
  e = sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3];
  const float lse = mx + logf(s);
  if (tid == 0) {
    a.entropy[m] = logf(s) - e / s;
    if (a.targets) {
      const int64_t t = a.targets[m];
      a.logprob[m] = t < 0 ? 0.f : t >= a.V ? NAN : load_logit<TYPE>(row, t) - lse;
    }
  }
  uint64_t k = ~0ull;
  for (int j = 0; j < a.top; ++j) {
    k = block_largest(k);
    if (tid == 0) {
      const int id = (int)~(uint32_t)k;
      a.top_ids[(long long)m * a.top + j] = id;
      a.top_logprobs[(long long)m * a.top + j] = load_logit<TYPE>(row, id) - lse;
    }
  }
}

}  // namespace

size_t logprobs_workspace(int M, int V, int top) { return 0; }

hipError_t launch_logprobs(const LogprobArgs& a, LogitType type, hipStream_t stream) {
  const dim3 grid((unsigned)a.M);
  if (type == LogitType::kFp32) logprobs_kernel<LogitType::kFp32><<<grid, 256, 0, stream>>>(a);
  else if (type == LogitType::kBf16) logprobs_kernel<LogitType::kBf16><<<grid, 256, 0, stream>>>(a);
  else logprobs_kernel<LogitType::kFp16><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace qmm
