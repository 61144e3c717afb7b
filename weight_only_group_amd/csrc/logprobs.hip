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
#include <algorithm>

#include "handoff.h"
#include "layer.h"

namespace qmm {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Exponents are cut here, where the power is 0 and times any sum of up to 2^30 finite.
constexpr float kFar = -1e4f;
constexpr int kThreads = 256, kWaves = kThreads / 64;
// Bytes of logits per thread and step: 64, or 16 where the blocks of the wider step
// would leave CUs idle (one row of 32000 fp16: 10.6 us in 16 blocks, 11.6 us in 4).
constexpr int kWide = 64, kNarrow = 16;
constexpr int kList = 1024;    // keys a wave's list holds
constexpr int kMaxSplit = 64;
constexpr int kMaxKeys = 512;  // keys of a block's waves before their last selection

constexpr int logit_size(LogitType t) { return t == LogitType::kFp32 ? 4 : 2; }
// Leading bits of a logit's order that differ between values of the type; the
// others are 1 below zero (the order is the complement there) and 0 above.
constexpr int order_bits(LogitType t) { return t == LogitType::kFp32 ? 32 : t == LogitType::kBf16 ? 16 : 19; }

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
__device__ __forceinline__ float order_float(uint32_t order) {  // of an order that is no NaN's; -inf for 0
  const uint32_t b = order & 0x80000000u ? order & 0x7FFFFFFFu : ~order;
  return order == 0 ? -INFINITY : __builtin_bit_cast(float, b);
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

// The k-th largest of a wave's keys (0: none; 0 where there are fewer than k), bit by
// bit: the order first, then, only among keys of that order, the index. `count(f)`
// says for how many keys f holds.
template <int BITS, typename COUNT>
__device__ __forceinline__ uint64_t kth_key(COUNT count, int k) {
  uint32_t hi = 0;
#pragma unroll 1
  for (int b = 31; b >= 32 - BITS; --b) {
    const uint32_t t = hi | 1u << b;
    if (count([=](uint64_t x) { return (uint32_t)(x >> 32) >= t; }) >= k) hi = t;
  }
  if (hi == 0) return 0;
  if (BITS < 32 && !(hi & 0x80000000u)) hi |= (1u << (32 - BITS) % 32) - 1;
  const int above = count([=](uint64_t x) { return (uint32_t)(x >> 32) > hi; });
  uint32_t lo = 0;
  if (count([=](uint64_t x) { return (uint32_t)(x >> 32) >= hi; }) > k) {
#pragma unroll 1
    for (int b = 31; b >= 0; --b) {
      const uint32_t t = lo | 1u << b;
      if (above + count([=](uint64_t x) { return (uint32_t)(x >> 32) == hi && (uint32_t)x >= t; }) >= k) lo = t;
    }
  }
  return (uint64_t)hi << 32 | lo;
}

// Reduces a wave's list of n keys, k <= n <= kList, to its k largest; returns the
// smallest of them. Rare (rows that rise along the vocabulary): the list is read
// from LDS again and again rather than kept in registers.
template <int BITS>
__device__ __forceinline__ uint64_t shrink_list(uint64_t* list, int n, int k, int lane) {
  const uint64_t least = kth_key<BITS>(
      [=](auto f) {
        int c = 0;
        for (int i = 0; i < n; i += 64) c += __builtin_popcountll(__ballot(i + lane < n && f(list[i + lane])));
        return c;
      },
      k);
  int at = 0;
#pragma unroll 1
  for (int i = 0; i < n; i += 64) {
    const uint64_t key = i + lane < n ? list[i + lane] : 0;
    const uint64_t hits = __ballot(key >= least);
    if (key >= least) list[at + __builtin_popcountll(hits & ((1ull << lane) - 1))] = key;
    at += __builtin_popcountll(hits);
  }
  return least;
}

struct Sums {
  float m, s, a;  // a in units of log2: sum p log2(p / e^0)
  __device__ __forceinline__ void join(const Sums& o) {
    const float n = fmaxf(m, o.m), off = n == -INFINITY ? 0.f : n;
    const float d0 = fmaxf((m - off) * kLog2e, kFar), d1 = fmaxf((o.m - off) * kLog2e, kFar);
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
// joins them. Bound: HBM for many rows, each logit is read once (a row that is not finite
// again, per alternative): 4096 rows of 50257 fp32 in 200 us, 4.1 TB/s. The selection of
// alternatives and the hand-over for few: 96 rows of 128257 bf16 with 20 alternatives
// 23.8 us, one row of 32000 fp16 with 5 10.6 us.
template <LogitType TYPE, int BYTES>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(LogprobKernelArgs p) {
  constexpr int SIZE = logit_size(TYPE), VEC = 16 / SIZE, PER = BYTES / SIZE, STEP = kThreads * PER, BITS = order_bits(TYPE);
  constexpr int LOADS = PER / VEC;
  __shared__ __attribute__((aligned(16))) uint64_t list[kWaves][kList];
  __shared__ uint64_t best[kMaxTop], first_least, wave_least[kWaves];
  __shared__ float wsum[kWaves][3];
  __shared__ int s_count, s_last;
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
  uint64_t lane_best = 0;      // the largest key of this lane
  uint64_t least = 0;          // keys below it are out
  float least_logit = -INFINITY;
  int listed = 0;
  const long long begin = (long long)part * p.steps * STEP, end = min(begin + (long long)p.steps * STEP, places);
  if (begin < end) load(begin);
  for (long long first = begin; first < end; first += STEP) {
    float l[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t v = raw[i / VEC][i % VEC / (4 / SIZE)];
      if constexpr (SIZE == 4) l[i] = __builtin_bit_cast(float, v);
      else l[i] = bits_to_float<TYPE == LogitType::kBf16>((uint16_t)(v >> (16 * (i & 1))));
    }
    if (first + STEP < end) load(first + STEP);
    float lm = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) lm = fmaxf(lm, l[i]);
    const float n = fmaxf(sum.m, lm), off = n == -INFINITY ? 0.f : n;
    if (n > sum.m) {
      const float d = fmaxf((sum.m - off) * kLog2e, kFar), f = __builtin_amdgcn_exp2f(d);
      sum.a = f * (sum.a + d * sum.s);
      sum.s *= f;
      sum.m = n;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float d = (l[i] - off) * kLog2e, e = __builtin_amdgcn_exp2f(d);
      sum.s += e;
      sum.a += e * fmaxf(d, kFar);  // 0 for a logit of -inf
    }
    if (top == 0) continue;
    const uint64_t hot = __ballot(lm >= least_logit);
    if (hot != 0 || first == begin) {
      // Index of a thread's i-th logit of the step.
      const int base = (int)(first - pad) + tid * VEC;
      auto index = [&](int i) { return base + (i / VEC) * (kThreads * VEC) + i % VEC; };
      if (float_order(lm) > (uint32_t)(lane_best >> 32)) {
        int at = PER;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) at = l[i] == lm ? i : at;
        // (places outside the row hold -inf: with a maximum of -inf the first one inside counts)
        while (at < PER && (unsigned)index(at) >= (unsigned)a.V) ++at;
        if (at < PER) lane_best = make_key(lm, index(at));
      }
      if (first == begin) {
        // The bound that holds at first: the top-th of the threads' largest keys, found by one wave.
        list[0][tid] = lane_best;
        __syncthreads();
        if (wave == 0) {
          uint64_t key[kWaves];
#pragma unroll
          for (int w = 0; w < kWaves; ++w) key[w] = list[0][w * 64 + lane];
          least = kth_key<BITS>(
              [&](auto f) {
                int c = 0;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) c += __builtin_popcountll(__ballot(f(key[w])));
                return c;
              },
              top);
          if (lane == 0) first_least = least;
        }
        __syncthreads();
        least = first_least;
      } else if (least == 0 || __builtin_popcountll(hot) > 8) {
        const uint64_t t = kth_key<BITS>([&](auto f) { return (int)__builtin_popcountll(__ballot(f(lane_best))); }, top);
        least = t > least ? t : least;
      }
      least_logit = order_float((uint32_t)(least >> 32));
#pragma unroll
      for (int g = 0; g < PER; g += (PER < 8 ? PER : 8)) {
        if (listed > kList - 8 * 64) {
          const uint64_t t = shrink_list<BITS>(list[wave], listed, top, lane);
          listed = top;
          least = t > least ? t : least;
          least_logit = order_float((uint32_t)(least >> 32));
        }
#pragma unroll
        for (int i = g; i < g + (PER < 8 ? PER : 8); ++i) {
          if (!__any(l[i] >= least_logit)) continue;
          const uint64_t key = make_key(l[i], index(i));
          const bool in = key >= least && (unsigned)index(i) < (unsigned)a.V;
          const uint64_t hits = __ballot(in);
          if (in) list[wave][listed + __builtin_popcountll(hits & ((1ull << lane) - 1))] = key;
          listed += __builtin_popcountll(hits);
        }
      }
    }
  }

  // The block's sums and alternatives.
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum.join(Sums{__shfl_xor(sum.m, o), __shfl_xor(sum.s, o), __shfl_xor(sum.a, o)});
  if (listed > kMaxKeys / kWaves) {
    const uint64_t t = shrink_list<BITS>(list[wave], listed, top, lane);
    listed = top;
    least = t > least ? t : least;
  }
  if (lane == 0) {
    wsum[wave][0] = sum.m;
    wsum[wave][1] = sum.s;
    wsum[wave][2] = sum.a;
    wave_least[wave] = least;
  }
  if (tid < top) best[tid] = 0;
  if (tid == 0) s_count = 0;
  // Of the waves' keys those that reach the largest bound; a key's place is the number of larger ones.
  uint64_t mine[kMaxKeys / kWaves / 64];
#pragma unroll
  for (int i = 0; i < kMaxKeys / kWaves / 64; ++i) mine[i] = i * 64 + lane < listed ? list[wave][i * 64 + lane] : 0;
  __syncthreads();
  uint64_t* keys = &list[0][0];
  auto gather = [&](uint64_t key, uint64_t from) {
    if (key >= from && key != 0) keys[atomicAdd(&s_count, 1)] = key;  // in any order: places go by keys
  };
  auto rank_keys = [&]() {
    const int n = s_count;
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = keys[i];
      int rank = 0;
#pragma unroll 8
      for (int y = 0; y < n; ++y) rank += keys[y] > key;
      if (rank < top) best[rank] = key;
    }
  };
  sum = Sums{wsum[0][0], wsum[0][1], wsum[0][2]};
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum.join(Sums{wsum[w][0], wsum[w][1], wsum[w][2]});
  if (top > 0) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) least = wave_least[w] > least ? wave_least[w] : least;
#pragma unroll
    for (int i = 0; i < kMaxKeys / kWaves / 64; ++i) gather(mine[i], least);
    __syncthreads();
    rank_keys();
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
      const uint64_t* parts = p.keys + (size_t)m * p.split * top;
      const uint64_t from = wave_max_key(lane < p.split ? handoff_load(&parts[(size_t)lane * top + top - 1]) : 0);
      if (tid == 0) s_count = 0;
      if (tid < top) best[tid] = 0;
      __syncthreads();
      for (int i = tid; i < p.split * top; i += kThreads) gather(handoff_load(&parts[i]), from);
      __syncthreads();
      rank_keys();
      __syncthreads();
    }
  }

  // l - lse as (l - m) - ln S: m + ln S would be rounded to m's size, 5e-4 for logits of 1e4.
  const float ln_s = logf(sum.s);
  auto log_prob = [&](long long i) { return (load_logit<TYPE>(row, i) - sum.m) - ln_s; };
  if (tid == 0) {
    a.entropy[m] = ln_s - kLn2 * sum.a / sum.s;
    if (a.targets) {
      const int64_t t = a.targets[m];
      a.logprob[m] = t < 0 ? 0.f : t >= a.V ? NAN : log_prob(t);
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
    a.top_logprobs[(size_t)m * top + tid] = log_prob(id);
  }
}

struct LogprobPlan {
  int split, steps;
  bool narrow;
};
LogprobPlan logprob_plan(int M, int V, int top, LogitType type, DeviceTopo topo) {
  // Blocks enough for four per CU, a step each at least; the joining block's lists hold all parts' keys.
  const long long places = (long long)V + 16 / logit_size(type) - 1;
  const bool narrow = (long long)M * places * logit_size(type) < (long long)topo.cus * kThreads * kWide;
  const int step = kThreads * (narrow ? kNarrow : kWide) / logit_size(type);
  const long long most = (places + step - 1) / step;
  long long split = 4ll * topo.cus / M;
  if (split > kMaxSplit) split = kMaxSplit;
  if (top > 0 && split > kWaves * kList / top) split = kWaves * kList / top;
  if (split > most) split = most;
  if (split < 1 || M > kGemvMaxStrips) split = 1;
  const long long steps = (most + split - 1) / split;
  return {(int)((most + steps - 1) / steps), (int)steps, narrow};
}

}  // namespace

size_t logprobs_workspace(int M, int V, int top) {
  size_t need = 0;
  for (LogitType type : {LogitType::kFp16, LogitType::kBf16, LogitType::kFp32}) {
    const LogprobPlan p = logprob_plan(M, V, top, type, device_topology());
    if (p.split > 1) need = std::max(need, kWorkspaceHeader + (size_t)M * p.split * (16 + 8 * (size_t)top));
  }
  return need;
}

hipError_t launch_logprobs(const LogprobArgs& a, LogitType type, hipStream_t stream) {
  const LogprobPlan plan = logprob_plan(a.M, a.V, a.top, type, device_topology());
  LogprobKernelArgs p = {a, plan.split, plan.steps, reinterpret_cast<uint32_t*>(a.workspace), nullptr, nullptr};
  if (plan.split > 1) {
    p.sums = reinterpret_cast<float*>(a.workspace + kWorkspaceHeader);
    p.keys = reinterpret_cast<uint64_t*>(p.sums + (size_t)a.M * plan.split * 4);
  }
  // A launch's threads are counted in 32 bits: more rows than this (never split) go in several.
  constexpr int kMostRows = 1 << 22;
  const auto run = [&](auto kernel) {
    for (int m = 0; m < a.M; m += cmin(a.M - m, kMostRows)) {
      p.l.logits = static_cast<const char*>(a.logits) + (long long)m * a.row_stride * logit_size(type);
      p.l.targets = a.targets ? a.targets + m : nullptr;
      p.l.logprob = a.targets ? a.logprob + m : nullptr;
      p.l.entropy = a.entropy + m;
      p.l.top_logprobs = a.top ? a.top_logprobs + (size_t)m * a.top : nullptr;
      p.l.top_ids = a.top ? a.top_ids + (size_t)m * a.top : nullptr;
      kernel<<<dim3((unsigned)(cmin(a.M - m, kMostRows) * plan.split)), kThreads, 0, stream>>>(p);
    }
  };
  if (type == LogitType::kFp32) run(plan.narrow ? logprobs_kernel<LogitType::kFp32, kNarrow> : logprobs_kernel<LogitType::kFp32, kWide>);
  else if (type == LogitType::kBf16) run(plan.narrow ? logprobs_kernel<LogitType::kBf16, kNarrow> : logprobs_kernel<LogitType::kBf16, kWide>);
  else run(plan.narrow ? logprobs_kernel<LogitType::kFp16, kNarrow> : logprobs_kernel<LogitType::kFp16, kWide>);
  return hipGetLastError();
}

}  // namespace qmm
