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

// The entries of a page table whose page is in use.
struct UsedEntries {
  const int32_t* kv_lens;
  FixedDiv by_stride, by_page;
  int table_stride;
  __device__ __forceinline__ bool in_use(int entry) const {
    const int b = by_stride(entry), len = kv_lens[b];
    return len > 0 && entry - b * table_stride <= by_page(len - 1);
  }
};

struct CopyArgs {
  char* cache[kPools];
  int64_t bytes[kPools];  // of a page
  const int32_t *src, *dst;
  const int32_t* count;  // pairs, on the device; NULL: n
  int n, pages;
  // Compaction only: a table to rename.
  const int32_t *page_table, *moved_to;
  int32_t* new_table;
  int entries;
  UsedEntries table;
};

// Block: pieces of pages of cache blockIdx.y. Bound: memory; 1531 pages of 4 caches (32 KB a page, 401 MB read and written)
// take 60 us, 6.7 TB/s (part of it from the last-level cache; a copy of 8 GB reaches 4.3 TB/s, of 512 MB 5.3).
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
    for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < a.entries; e += (long long)gridDim.x * kThreads) {
      const int page = a.page_table[e];
      a.new_table[e] = a.table.in_use((int)e) && page >= 0 && page < a.pages ? a.moved_to[page] : page;
    }
  }
}

constexpr int kPlanThreads = 1024;
struct PlanArgs {
  CompactArgs c;
  UsedEntries table;
  int32_t *src, *dst, *count;
};

// One block: marks the pages in use in LDS, numbers them, and lists the moves. Bound by the latency of its few rounds
// through memory: 6000 pages, a table of 9000 entries 7.8 us (10.3 where each thread counts the marks below its page by
// itself); 64 pages 3.3 us.
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
  // Four entries of a thread at a time, asked for at once with their sequences' lengths.
  constexpr int kEntries = 4;
  const int entries = c.B * c.table_stride;
  for (int first = tid; first < entries; first += kEntries * kPlanThreads) {
    int page[kEntries];
    bool in_use[kEntries];
#pragma unroll
    for (int x = 0; x < kEntries; ++x) {
      const int e = (int)min((unsigned)first + x * kPlanThreads, (unsigned)entries - 1);
      page[x] = c.page_table[e];
      in_use[x] = p.table.in_use(e);
    }
#pragma unroll
    for (int x = 0; x < kEntries; ++x)  // (the last entry more than once, where they are past the end)
      if (in_use[x] && page[x] >= 0 && page[x] < c.pages) atomicOr(&mark[page[x] / 32], 1u << page[x] % 32);
    if (first > INT32_MAX - kEntries * kPlanThreads) break;
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
  auto marks_of = [&](int page) { return (uint64_t)mark[page / 32 + 1] << 32 | mark[page / 32]; };  // of 64 pages from page on
  int kept = live;  // of the pages in use, those below live
  if (live < spans * kSpan) {
    kept = before[live / kSpan];
    for (int page = live / kSpan * kSpan; page < live; page += 64)
      kept += __builtin_popcountll(marks_of(page) & (live - page < 64 ? (1ull << (live - page)) - 1 : ~0ull));
  }
  if (tid == 0) {
    *c.live = live;
    *p.count = live - kept;
  }
  // A wave takes a span, 64 pages at a time.
  for (int s = wave; s < spans; s += kPlanThreads / 64) {
    int below = before[s];
#pragma unroll
    for (int q = 0; q < kSpan / 64; ++q) {
      const uint64_t marks = marks_of(s * kSpan + 64 * q);
      const int page = s * kSpan + 64 * q + lane;
      const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(marks >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)marks, below));
      const bool used = marks >> lane & 1;
      below += __builtin_popcountll(marks);
      if (page >= c.pages) continue;
      if (page < live) {
        c.moved_to[page] = used ? page : -1;
        if (!used) p.dst[page - rank] = page;
      } else {
        if (used) p.src[rank - kept] = page;
        else c.moved_to[page] = -1;
      }
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
  const UsedEntries table = {c.kv_lens, fixed_div(c.table_stride), fixed_div(c.page_size), c.table_stride};
  const PlanArgs plan = {c, table, lists, lists + half, lists + 2 * half};
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(plan);
  CopyArgs a = {};
  a.src = plan.src;
  a.dst = plan.dst;
  a.count = plan.count;
  a.pages = c.pages;
  a.page_table = c.page_table;
  a.moved_to = c.moved_to;
  a.new_table = c.new_table;
  a.entries = c.B * c.table_stride;
  a.table = table;
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
