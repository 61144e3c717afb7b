// Copying pages of caches, and packing the pages in use into the lowest ones.
//
// Packing: with n pages in use, those in use at or past n and the free ones below n
// are equally many; the i-th of the former goes to the i-th of the latter. Sources
// and destinations are apart, so that the copies need no order.
#include <algorithm>

#include "cache.h"
#include "fixed_div.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = kThreads * 64;  // bytes a block copies at a time
constexpr int kPools = 64;             // caches of a launch

struct CopyArgs {
  char* cache[kPools];
  int64_t bytes[kPools];  // of a page
  const int32_t *src, *dst;
  const int32_t* count;  // pairs, on the device; NULL: n
  int n, pages;
  // Compaction only: a table to rename.
  const int32_t *page_table, *kv_lens, *moved_to;
  int32_t* new_table;
  int B, table_stride, page_size;
};

// Pages of sequence b that are in use.
__device__ __forceinline__ int pages_of(const int32_t* kv_lens, int b, int page_size, int table_stride) {
  const int len = kv_lens[b];
  return len > 0 ? min((len - 1) / page_size + 1, table_stride) : 0;
}

// Block: pieces of pages of cache blockIdx.y. Bound: HBM.
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(CopyArgs a) {
  const int64_t bytes = a.bytes[blockIdx.y];
  char* cache = a.cache[blockIdx.y];
  const int n = a.count ? *a.count : a.n;
  const int pieces = (int)((bytes + kPiece - 1) / kPiece);
  for (long long unit = blockIdx.x; unit < (long long)n * pieces; unit += gridDim.x) {
    const int i = (int)(unit / pieces);
    const int from = a.src[i], to = a.dst[i];
    if (from < 0 || from >= a.pages || to < 0 || to >= a.pages) continue;
    const int64_t first = (unit - (long long)i * pieces) * kPiece + threadIdx.x * 16;
    const char* s = cache + (int64_t)from * bytes;
    char* d = cache + (int64_t)to * bytes;
    u32x4 v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t at = first + x * kThreads * 16;
      if (at < bytes) v[x] = *reinterpret_cast<const u32x4*>(s + at);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t at = first + x * kThreads * 16;
      if (at < bytes) *reinterpret_cast<u32x4*>(d + at) = v[x];
    }
  }
  if (a.new_table && blockIdx.y == 0) {
    const long long entries = (long long)a.B * a.table_stride;
    for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < entries; e += (long long)gridDim.x * kThreads) {
      const int b = (int)(e / a.table_stride), i = (int)(e - (long long)b * a.table_stride);
      const int page = a.page_table[e];
      const bool in_use = i < pages_of(a.kv_lens, b, a.page_size, a.table_stride) && page >= 0 && page < a.pages;
      a.new_table[e] = in_use ? a.moved_to[page] : page;
    }
  }
}

constexpr int kPlanThreads = 1024;
struct PlanArgs {
  CompactArgs c;
  int32_t *src, *dst, *count;
};

// One block: marks the pages in use in LDS, numbers them, and lists the moves.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PlanArgs p) {
  constexpr int kSpan = 256;  // pages per entry of `before`
  __shared__ uint32_t mark[kMostPages / 32];
  __shared__ int before[kMostPages / kSpan + 1];  // pages in use below kSpan i
  __shared__ int wave_sum[kPlanThreads / 64];
  const CompactArgs& c = p.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int spans = (c.pages + kSpan - 1) / kSpan;
  for (int i = tid; i < spans * (kSpan / 32); i += kPlanThreads) mark[i] = 0;
  __syncthreads();
  const long long entries = (long long)c.B * c.table_stride;
  for (long long e = tid; e < entries; e += kPlanThreads) {
    const int b = (int)(e / c.table_stride), i = (int)(e - (long long)b * c.table_stride);
    const int page = c.page_table[e];
    if (i < pages_of(c.kv_lens, b, c.page_size, c.table_stride) && page >= 0 && page < c.pages) atomicOr(&mark[page / 32], 1u << page % 32);
  }
  __syncthreads();
  // Running counts, 1024 spans at a time.
  int base = 0;
  for (int s0 = 0; s0 < spans; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int n = 0;
    if (s < spans)
#pragma unroll
      for (int w = 0; w < kSpan / 32; ++w) n += __builtin_popcount(mark[s * (kSpan / 32) + w]);
    int sum = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(sum, o);
      sum += lane >= o ? up : 0;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    int total = 0, ahead = 0;
    for (int w = 0; w < kPlanThreads / 64; ++w) {
      ahead += w < wave ? wave_sum[w] : 0;
      total += wave_sum[w];
    }
    if (s < spans) before[s] = base + ahead + sum - n;
    base += total;
    __syncthreads();
  }
  const int live = base;
  auto in_use_below = [&](int page) {  // page <= pages
    int n = page / kSpan < spans ? before[page / kSpan] : live;
    for (int w = page / kSpan * (kSpan / 32); w < page / 32; ++w) n += __builtin_popcount(mark[w]);
    return page % 32 ? n + __builtin_popcount(mark[page / 32] & ((1u << page % 32) - 1)) : n;
  };
  const int kept = in_use_below(live);
  if (tid == 0) {
    *c.live = live;
    *p.count = live - kept;
  }
  for (int page = tid; page < c.pages; page += kPlanThreads) {
    const bool used = mark[page / 32] >> page % 32 & 1;
    const int rank = in_use_below(page);
    if (page < live) {
      c.moved_to[page] = used ? page : -1;
      if (!used) p.dst[page - rank] = page;
    } else {
      if (used) p.src[rank - kept] = page;
      else c.moved_to[page] = -1;
    }
  }
  __syncthreads();
  for (int i = tid; i < live - kept; i += kPlanThreads) c.moved_to[p.src[i]] = p.dst[i];
}

template <typename RUN>
hipError_t each_launch(const PagePools& pools, CopyArgs& a, RUN run) {
  for (int first = 0; first < pools.n; first += kPools) {
    const int n = std::min(kPools, pools.n - first);
    int64_t most = 0;
    for (int i = 0; i < n; ++i) {
      a.cache[i] = static_cast<char*>(pools.caches[first + i]);
      a.bytes[i] = pools.page_bytes[first + i];
      most = std::max(most, a.bytes[i]);
    }
    run(n, (most + kPiece - 1) / kPiece);
    a.new_table = nullptr;  // renamed once
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_copy_pages(const PagePools& pools, int pages, const int32_t* src, const int32_t* dst, int n,
                             hipStream_t stream) {
  CopyArgs a = {};
  a.src = src;
  a.dst = dst;
  a.n = n;
  a.pages = pages;
  return each_launch(pools, a, [&](int caches, int64_t pieces) {
    const int64_t blocks = std::min<int64_t>(n * pieces, 1 << 16);
    copy_pages_kernel<<<dim3((unsigned)blocks, (unsigned)caches), kThreads, 0, stream>>>(a);
  });
}

// The moves (at most half of the pages, each place once), then their count.
size_t compact_workspace(int pages) { return kWorkspaceHeader + ((size_t)pages + 4) * 4; }

hipError_t launch_compact(const PagePools& pools, const CompactArgs& c, hipStream_t stream) {
  const int half = c.pages / 2;
  int32_t* lists = reinterpret_cast<int32_t*>(c.workspace + kWorkspaceHeader);
  const PlanArgs plan = {c, lists, lists + half, lists + 2 * half};
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(plan);
  CopyArgs a = {};
  a.src = plan.src;
  a.dst = plan.dst;
  a.count = plan.count;
  a.pages = c.pages;
  a.page_table = c.page_table;
  a.kv_lens = c.kv_lens;
  a.moved_to = c.moved_to;
  a.new_table = c.new_table;
  a.B = c.B;
  a.table_stride = c.table_stride;
  a.page_size = c.page_size;
  const int64_t most = std::min<int64_t>(half, (int64_t)c.B * c.table_stride);
  const int cus = device_topology().cus;
  const auto run = [&](int caches, int64_t pieces) {
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(most * pieces, 16ll * cus / std::min(caches, 16)));
    copy_pages_kernel<<<dim3((unsigned)blocks, (unsigned)std::max(caches, 1)), kThreads, 0, stream>>>(a);
  };
  if (pools.n == 0) {  // the table alone: a cache of no bytes
    run(0, 1);
    return hipGetLastError();
  }
  return each_launch(pools, a, run);
}

}  // namespace qmm
