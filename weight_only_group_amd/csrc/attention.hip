// Attention of new tokens to the paged cache of their sequences.
#include "layer.h"

namespace qmm {
namespace {

// One wave per query row and head; each lane holds D / 64 values, the keys are
// taken one by one with a running maximum and sum.
template <bool BF, int D>
__global__ void __launch_bounds__(64) attention_kernel(AttentionArgs a) {
  constexpr int N = D / 64;
  const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x;
  const int q0 = min(max(a.q_starts[b], 0), a.T), q1 = min(max(a.q_starts[b + 1], q0), a.T);
  const int i = blockIdx.x, t = q0 + i;
  if (t >= q1) return;
  const int kv = min(max(a.kv_lens[b], 0), a.max_kv);
  const int pos = kv - (q1 - q0) + i;
  const int lo = a.first ? max(a.first[t], 0) : 0, hi = min(a.end ? a.end[t] : pos + 1, kv);
  const int hk = h / (a.Hq / a.Hkv);
  float q[N], o[N] = {};
  for (int d = 0; d < N; ++d) q[d] = bits_to_float<BF>(a.q[t * a.q_stride + (long long)h * D + lane * N + d]);
  float mx = -INFINITY, sum = 0;
  for (int j = lo; j < hi; ++j) {
    const int page = min(max(a.page_table[(long long)b * a.table_stride + j / a.page_size], 0), a.pages - 1);
    const long long at = (((long long)page * a.Hkv + hk) * a.page_size + j % a.page_size) * D + lane * N;
    float s = 0;
    for (int d = 0; d < N; ++d) s += q[d] * bits_to_float<BF>(a.k_cache[at + d]);
    for (int x = 32; x > 0; x >>= 1) s += __shfl_xor(s, x);
    s *= a.scale;
    if (a.softcap > 0) s = a.softcap * tanhf(s / a.softcap);
    if (a.slopes) s -= a.slopes[h] * fabsf((float)(pos - j));
    const float m = fmaxf(mx, s), f = __expf(mx - m), p = __expf(s - m);
    sum = sum * f + p;
    for (int d = 0; d < N; ++d) o[d] = o[d] * f + p * bits_to_float<BF>(a.v_cache[at + d]);
    mx = m;
  }
  for (int d = 0; d < N; ++d)
    a.out[((long long)t * a.Hq + h) * D + lane * N + d] = float_to_bits<BF>(hi > lo ? o[d] / sum : 0.f);
}

}  // namespace

size_t attention_workspace(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv) { return 0; }

hipError_t launch_attention(const AttentionArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid((unsigned)a.max_q, (unsigned)a.Hq, (unsigned)a.B);
  if (bf16) {
    if (a.D == 64) attention_kernel<true, 64><<<grid, 64, 0, stream>>>(a);
    else if (a.D == 128) attention_kernel<true, 128><<<grid, 64, 0, stream>>>(a);
    else attention_kernel<true, 256><<<grid, 64, 0, stream>>>(a);
  } else {
    if (a.D == 64) attention_kernel<false, 64><<<grid, 64, 0, stream>>>(a);
    else if (a.D == 128) attention_kernel<false, 128><<<grid, 64, 0, stream>>>(a);
    else attention_kernel<false, 256><<<grid, 64, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace qmm
