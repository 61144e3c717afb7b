// Log probabilities of given tokens, entropy and the largest alternatives of rows
// of logits, in one pass over them.
//
// With a running maximum m: S = sum e^(l - m), A = sum e^(l - m) (l - m); lse = m +
// ln S, entropy = ln S - A / S. A change of m to n scales S by f = e^(m - n) and
// makes A f (A + (m - n) S).
//
// Alternatives: a logit's key is its order in the upper and the complement of its
// index in the lower half, so that keys differ, and larger keys come first. A wave
// keeps the largest key that each lane has seen: the top-th largest of those is no
// larger than the wave's top-th key, and few keys reach it. They go to a list.
#include "handoff.h"
#include "layer.h"

namespace qmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPer = 16;                // logits per thread and step
constexpr int kStep = kThreads * kPer;  // logits per block and step
constexpr int kList = 1024;             // keys a wave's list holds
constexpr int kMaxSplit = 64;

template <LogitType TYPE> constexpr int kSize = TYPE == LogitType::kFp32 ? 4 : 2;

template <LogitType TYPE>
__device__ __forceinline__ float load_logit(const char* row, long long i) {
  if constexpr (TYPE == LogitType::kFp32) return reinterpret_cast<const float*>(row)[i];
  else return bits_to_float<TYPE == LogitType::kBf16>(reinterpret_cast<const uint16_t*>(row)[i]);
}

// Unsigned order of floats, never 0: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t float_order(float l) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);
  return l != l ? 0xFFFFFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t make_key(float l, uint32_t index) { return (uint64_t)float_order(l) << 32 | (uint32_t)~index; }
__device__ __forceinline__ int key_index(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ uint64_t wave_max_key(uint64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor(v, o);
    v = w > v ? w : v;
  }
  return v;
}

// The k-th largest of N keys per lane of a wave (0: none; 0 where there are fewer
// than k), bit by bit: the order first, then, only among keys of that order, the index.
template <int N>
__device__ uint64_t kth_key(const uint64_t (&key)[N], int k) {
  uint32_t hi = 0;
  int above = 0;  // keys of a larger order
  for (int b = 31; b >= 0; --b) {
    const uint32_t t = hi | 1u << b;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __builtin_popcountll(__ballot((uint32_t)(key[i] >> 32) >= t));
    if (n >= k) hi = t;
  }
  if (hi == 0) return 0;
  int same = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    above += __builtin_popcountll(__ballot((uint32_t)(key[i] >> 32) > hi));
    same += __builtin_popcountll(__ballot((uint32_t)(key[i] >> 32) == hi));
  }
  uint32_t lo = 0;
  if (above + same > k) {
    for (int b = 31; b >= 0; --b) {
      const uint32_t t = lo | 1u << b;
      int n = above;
#pragma unroll
      for (int i = 0; i < N; ++i) n += __builtin_popcountll(__ballot((uint32_t)(key[i] >> 32) == hi && (uint32_t)key[i] >= t));
      if (n >= k) lo = t;
    }
  }
  return (uint64_t)hi << 32 | lo;
}

// Reduces a wave's list of n <= kList keys to its k largest; returns the smallest of them.
__device__ uint64_t shrink_list(uint64_t* list, int& n, int k, int lane) {
  uint64_t key[kList / 64];
#pragma unroll
  for (int i = 0; i < kList / 64; ++i) key[i] = i * 64 + lane < n ? list[i * 64 + lane] : 0;
  const uint64_t least = kth_key(key, k);
  int at = 0;
#pragma unroll
  for (int i = 0; i < kList / 64; ++i) {
    const bool keep = key[i] != 0 && key[i] >= least;
    const uint64_t hits = __ballot(keep);
    if (keep) list[at + __builtin_popcountll(hits & ((1ull << lane) - 1))] = key[i];
    at += __builtin_popcountll(hits);
  }
  n = at;
  return least;
}

struct Sums {
  float m, s, a;  // a in units of log2: sum p log2(p / e^0)
  __device__ __forceinline__ void join(const Sums& o) {
    const float n = fmaxf(m, o.m), off = n == -INFINITY ? 0.f : n;
    const float d0 = fmaxf((m - off) * kLog2e, -1e30f), d1 = fmaxf((o.m - off) * kLog2e, -1e30f);
    const float f0 = __builtin_amdgcn_exp2f(d0), f1 = __builtin_amdgcn_exp2f(d1);
    a = f0 * (a + d0 * s) + f1 * (o.a + d1 * o.s);
    s = f0 * s + f1 * o.s;
    m = n;
  }
};

struct LogprobKernelArgs {
  LogprobArgs l;
  int split;  // blocks per row
  int steps;  // steps per block
  uint32_t* counters;
  float* sums;     // (M, split, 4)
  uint64_t* keys;  // (M, split, top)
};

// Block: `steps` steps of one row; with several blocks per row the last to arrive
// joins them. Bound: HBM, each logit is read once (a row that is not finite again,
// per alternative).
template <LogitType TYPE>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobKernelArgs p) {
  constexpr int SIZE = kSize<TYPE>, VEC = 16 / SIZE, LOADS = kPer / VEC;
  __shared__ uint64_t list[kWaves][kList];
  __shared__ uint64_t best[kMaxTop];
  __shared__ float wsum[kWaves][3];
  __shared__ int count[kWaves];
  __shared__ int s_last;
  const LogprobArgs& a = p.l;
  const int m = blockIdx.x / p.split, part = blockIdx.x - m * p.split;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), top = a.top;
  const char* row = static_cast<const char*>(a.logits) + (long long)m * a.row_stride * SIZE;
  // Places count from the 16-byte line in which the row starts.
  const int pad = (int)((reinterpret_cast<uintptr_t>(row) & 15) / SIZE);
  const long long places = (long long)a.V + pad;
  const char* line = row - pad * SIZE;

  u32x4 raw[LOADS];
  auto load = [&](long long first) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const long long at = first + ((long long)i * kThreads + tid) * VEC;
      if (at >= pad && at + VEC <= places) {
        raw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(line + at * SIZE));
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if constexpr (SIZE == 4) {
            const bool in = at + x >= pad && at + x < places;
            raw[i][x] = in ? *reinterpret_cast<const uint32_t*>(line + (at + x) * 4) : 0xFF800000u;
          } else {
            uint32_t v = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bool in = at + 2 * x + h >= pad && at + 2 * x + h < places;
              v |= (in ? (uint32_t)*reinterpret_cast<const uint16_t*>(line + (at + 2 * x + h) * 2)
                       : TYPE == LogitType::kBf16 ? 0xFF80u : 0xFC00u) << (16 * h);
            }
            raw[i][x] = v;
          }
        }
      }
    }
  };

  Sums sum = {-INFINITY, 0, 0};
  uint64_t lane_best = 0, least = 0;  // the largest key of this lane; keys below `least` are out
  int listed = 0;
  const long long begin = (long long)part * p.steps * kStep, end = min(begin + (long long)p.steps * kStep, places);
  if (begin < end) load(begin);
  for (long long first = begin; first < end; first += kStep) {
    float l[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t v = raw[i / VEC][i % VEC / (4 / SIZE)];
      if constexpr (SIZE == 4) l[i] = __builtin_bit_cast(float, v);
      else l[i] = bits_to_float<TYPE == LogitType::kBf16>((uint16_t)(v >> (16 * (i & 1))));
    }
    if (first + kStep < end) load(first + kStep);
    float lm = l[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) lm = fmaxf(lm, l[i]);
    const float n = fmaxf(sum.m, lm), off = n == -INFINITY ? 0.f : n;
    if (n > sum.m) {
      const float d = fmaxf((sum.m - off) * kLog2e, -1e30f), f = __builtin_amdgcn_exp2f(d);
      sum.a = f * (sum.a + d * sum.s);
      sum.s *= f;
      sum.m = n;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float d = (l[i] - off) * kLog2e, e = __builtin_amdgcn_exp2f(d);
      sum.s += e;
      sum.a += e * fmaxf(d, -1e30f);  // 0 for a logit of -inf
    }
    if (top > 0) {
      // Index of place `first + ((i / VEC) * kThreads + tid) * VEC + i % VEC`.
      auto index = [&](int i) { return (int)(first - pad + ((long long)(i / VEC) * kThreads + tid) * VEC + i % VEC); };
      const uint32_t least_order = (uint32_t)(least >> 32), lm_order = float_order(lm);
      const uint64_t hot = __ballot(lm_order >= least_order);
      if (hot) {
        if (lm_order > (uint32_t)(lane_best >> 32)) {
#pragma unroll
          for (int i = kPer - 1; i >= 0; --i)
            if (l[i] == lm && (unsigned)index(i) < (unsigned)a.V) lane_best = make_key(lm, index(i));
        }
        if (least == 0 || __builtin_popcountll(hot) > 8) {
          const uint64_t one[1] = {lane_best};
          const uint64_t t = kth_key(one, top);
          least = t > least ? t : least;
        }
        if (listed > kList / 2) {
          const uint64_t t = shrink_list(list[wave], listed, top, lane);
          least = t > least ? t : least;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint64_t key = make_key(l[i], index(i));
          const bool in = key >= least && (unsigned)index(i) < (unsigned)a.V;
          const uint64_t hits = __ballot(in);
          if (hits) {
            if (in) list[wave][listed + __builtin_popcountll(hits & ((1ull << lane) - 1))] = key;
            listed += __builtin_popcountll(hits);
          }
        }
      }
    }
  }

  // The block's sums and alternatives.
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum.join(Sums{__shfl_xor(sum.m, o), __shfl_xor(sum.s, o), __shfl_xor(sum.a, o)});
  if (listed > kList / kWaves / 2) shrink_list(list[wave], listed, top, lane);
  if (lane == 0) {
    wsum[wave][0] = sum.m;
    wsum[wave][1] = sum.s;
    wsum[wave][2] = sum.a;
    count[wave] = listed;
  }
  if (tid < top) best[tid] = 0;
  __syncthreads();
  sum = Sums{wsum[0][0], wsum[0][1], wsum[0][2]};
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum.join(Sums{wsum[w][0], wsum[w][1], wsum[w][2]});
  // A key's place is the number of larger ones.
  auto rank_lists = [&]() {
    for (int w = 0; w < kWaves; ++w)
      for (int i = tid; i < count[w]; i += kThreads) {
        const uint64_t key = list[w][i];
        int rank = 0;
        for (int x = 0; x < kWaves; ++x)
          for (int y = 0; y < count[x]; ++y) rank += list[x][y] > key;
        if (rank < top) best[rank] = key;
      }
  };
  if (top > 0) {
    rank_lists();
    __syncthreads();
  }
  if (p.split > 1) {
    const size_t at = (size_t)m * p.split + part;
    if (tid < top) handoff_store(&p.keys[at * top + tid], best[tid]);
    if (tid == 0) {
      handoff_store(p.sums + at * 4, sum.m, sum.s);
      handoff_store(p.sums + at * 4 + 2, sum.a);
    }
    if (!handoff_last(&p.counters[m], (uint32_t)p.split, &s_last)) return;
    const float* w = p.sums + (size_t)m * p.split * 4;
    sum = Sums{-INFINITY, 0, 0};
    if (lane < p.split) {
      const FloatPair ms = handoff_load_pair(w + lane * 4);
      sum = Sums{ms.a, ms.b, handoff_load(w + lane * 4 + 2)};
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum.join(Sums{__shfl_xor(sum.m, o), __shfl_xor(sum.s, o), __shfl_xor(sum.a, o)});
    if (top > 0) {
      // No key below the largest of the parts' last ones is among the row's.
      const uint64_t* keys = p.keys + (size_t)m * p.split * top;
      const uint64_t from = wave_max_key(lane < p.split ? handoff_load(&keys[(size_t)lane * top + top - 1]) : 0);
      if (tid < kWaves) count[tid] = 0;
      if (tid < top) best[tid] = 0;
      __syncthreads();
      for (int i = tid; i < p.split * top; i += kThreads) {
        const uint64_t key = handoff_load(&keys[i]);
        if (key >= from && key != 0) list[0][atomicAdd(&count[0], 1)] = key;  // any order: places go by keys
      }
      __syncthreads();
      rank_lists();
      __syncthreads();
    }
  }

  const float ln_s = logf(sum.s), lse = sum.m + ln_s;
  if (tid == 0) {
    a.entropy[m] = ln_s - kLn2 * sum.a / sum.s;
    if (a.targets) {
      const int64_t t = a.targets[m];
      a.logprob[m] = t < 0 ? 0.f : t >= a.V ? NAN : load_logit<TYPE>(row, t) - lse;
    }
  }
  if (top > 0 && !(sum.s == sum.s && sum.s > 0)) {
    // A row with a NaN or an infinity, or of nothing but -inf: one key after another.
    uint64_t below = ~0ull;
    for (int j = 0; j < top; ++j) {
      uint64_t k = 0;
      for (int i = tid; i < a.V; i += kThreads) {
        const uint64_t x = make_key(load_logit<TYPE>(row, i), i);
        if (x < below && x > k) k = x;
      }
      k = wave_max_key(k);
      __syncthreads();
      if (lane == 0) list[wave][0] = k;
      __syncthreads();
      for (int w = 0; w < kWaves; ++w) k = list[w][0] > k ? list[w][0] : k;
      below = k;
      if (tid == 0) best[j] = k;
    }
    __syncthreads();
  }
  if (tid < top) {
    const int id = key_index(best[tid]);
    a.top_ids[(size_t)m * top + tid] = id;
    a.top_logprobs[(size_t)m * top + tid] = load_logit<TYPE>(row, id) - lse;
  }
}

struct LogprobPlan {
  int split, steps;
};
LogprobPlan logprob_plan(int M, int V, int top, DeviceTopo topo) {
  // Blocks enough for four per CU, a step each at least; the joining block's list holds all parts' keys.
  const long long places = (long long)V + 7, most = (places + kStep - 1) / kStep;
  long long split = 4ll * topo.cus / M;
  if (split > kMaxSplit) split = kMaxSplit;
  if (top > 0 && split > kList / top) split = kList / top;
  if (split > most) split = most;
  if (split < 1 || M > kGemvMaxStrips) split = 1;
  const long long steps = (most + split - 1) / split;
  return {(int)((most + steps - 1) / steps), (int)steps};
}

}  // namespace

size_t logprobs_workspace(int M, int V, int top) {
  const LogprobPlan p = logprob_plan(M, V, top, device_topology());
  return p.split > 1 ? kWorkspaceHeader + (size_t)M * p.split * (16 + 8 * (size_t)top) : 0;
}

hipError_t launch_logprobs(const LogprobArgs& a, LogitType type, hipStream_t stream) {
  const LogprobPlan plan = logprob_plan(a.M, a.V, a.top, device_topology());
  LogprobKernelArgs p = {a, plan.split, plan.steps, reinterpret_cast<uint32_t*>(a.workspace), nullptr, nullptr};
  if (plan.split > 1) {
    p.sums = reinterpret_cast<float*>(a.workspace + kWorkspaceHeader);
    p.keys = reinterpret_cast<uint64_t*>(p.sums + (size_t)a.M * plan.split * 4);
  }
  const dim3 grid((unsigned)(a.M * plan.split));
  if (type == LogitType::kFp32) logprobs_kernel<LogitType::kFp32><<<grid, kThreads, 0, stream>>>(p);
  else if (type == LogitType::kBf16) logprobs_kernel<LogitType::kBf16><<<grid, kThreads, 0, stream>>>(p);
  else logprobs_kernel<LogitType::kFp16><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace qmm
