// The append to the paged cache: queries and keys rotated by their positions,
// keys and values stored at their slots.
//
// For a pair (a, b) of a head and the angle's (c, s): (a c - b s, b c + a s), in
// fp32, rounded once. Bound: HBM, every value is read and written once, the table
// rows of a token come from the caches for all its heads but the first. 16381 tokens of
// 24 + 2 x 4 heads of 64: 30.8 us, 4.4 TB/s (a plain copy reaches 4.9); 7 tokens of
// 32 + 2 x 8 heads of 128: 3.3 us, a launch's latency.
#include "layer.h"

namespace qmm {
namespace {

// Eight values of one head per thread. With half-split pairs (i, i + R / 2) a
// thread takes values [8c, 8c + 8) of the first half and their partners.
template <bool BF, bool ADJ>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a) {
  const int chunks = a.D / 8;
  const int heads = a.Hq + 2 * a.Hkv;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int c = (int)(i % chunks);
  const long long th = i / chunks;
  const int h = (int)(th % heads);
  const long long t = th / heads;
  if (t >= a.T) return;

  const uint16_t* src;
  uint16_t* dst;
  const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
  if (is_q) {
    src = a.q + t * a.q_stride + (long long)h * a.D;
    dst = a.q_out + (t * a.Hq + h) * a.D;
  } else {
    const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= (long long)a.pages * a.page_size) return;
    const long long page = slot / a.page_size;
    const int at = (int)(slot - page * a.page_size);
    src = (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + (long long)hk * a.D;
    dst = (is_v ? a.v_cache : a.k_cache) + ((page * a.Hkv + hk) * a.page_size + at) * a.D;
  }
  if (is_v || 8 * c >= a.R) {
    *reinterpret_cast<u32x4*>(dst + 8 * c) = *reinterpret_cast<const u32x4*>(src + 8 * c);
    return;
  }
  if (!ADJ && 16 * c >= a.R) return;  // the second half goes with its partners
  const int pos = min(max(a.positions[t], 0), a.P - 1);
  const float* cs = a.cos + (long long)pos * (a.R / 2);
  const float* sn = a.sin + (long long)pos * (a.R / 2);
  if constexpr (ADJ) {
    u32x4 x = *reinterpret_cast<const u32x4*>(src + 8 * c), y;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float u = bits_to_float<BF>((uint16_t)x[p]), w = bits_to_float<BF>((uint16_t)(x[p] >> 16));
      const float co = cs[4 * c + p], si = sn[4 * c + p];
      y[p] = float_to_bits<BF>(u * co - w * si) | (uint32_t)float_to_bits<BF>(w * co + u * si) << 16;
    }
    *reinterpret_cast<u32x4*>(dst + 8 * c) = y;
  } else {
    const int half = a.R / 2;
    const u32x4 x = *reinterpret_cast<const u32x4*>(src + 8 * c);
    const u32x4 z = *reinterpret_cast<const u32x4*>(src + 8 * c + half);
    u32x4 xo, zo;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t lo[2], hi[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float u = bits_to_float<BF>((uint16_t)(x[p] >> (16 * e))), w = bits_to_float<BF>((uint16_t)(z[p] >> (16 * e)));
        const float co = cs[8 * c + 2 * p + e], si = sn[8 * c + 2 * p + e];
        lo[e] = float_to_bits<BF>(u * co - w * si);
        hi[e] = float_to_bits<BF>(w * co + u * si);
      }
      xo[p] = lo[0] | lo[1] << 16;
      zo[p] = hi[0] | hi[1] << 16;
    }
    *reinterpret_cast<u32x4*>(dst + 8 * c) = xo;
    *reinterpret_cast<u32x4*>(dst + 8 * c + half) = zo;
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, bool bf16, bool adjacent, hipStream_t stream) {
  const long long n = (long long)a.T * (a.Hq + 2 * a.Hkv) * (a.D / 8);
  const dim3 grid((unsigned)((n + 255) / 256));
  if (bf16 && adjacent) kv_append_kernel<true, true><<<grid, 256, 0, stream>>>(a);
  else if (bf16) kv_append_kernel<true, false><<<grid, 256, 0, stream>>>(a);
  else if (adjacent) kv_append_kernel<false, true><<<grid, 256, 0, stream>>>(a);
  else kv_append_kernel<false, false><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace qmm
