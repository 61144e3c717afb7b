// Internal declarations of the 4-bit cache and of the care of pages
// (include/qmm_cache.h): the validated arguments of each call and its launch.
#pragma once

#include "layer.h"

namespace qmm {

// ---- the 4-bit cache --------------------------------------------------------------
constexpr int kBlockTokens = 8;  // tokens of a head that lie interleaved
// Bytes of a block: codes, then a scale and a middle (fp16) per token and group.
__host__ __device__ constexpr int kv4_block_bytes(int D, int groups) { return 4 * D + 32 * groups; }

constexpr int kKv4Largest = 16384;
// A group of a larger scale (or of an infinite one) stands for NaN: 24 s, which the attention decodes with, is no fp16
// number beyond it.
constexpr int kKv4LargestScale = 2728;
// In AppendArgs and AttentionArgs the caches' pointers stand for bytes.
hipError_t launch_kv4_append(const AppendArgs& a, int group_size, bool bf16, bool adjacent, hipStream_t stream);

struct Kv4GatherArgs {
  const uint8_t *k_cache, *v_cache;
  const int64_t* slots;
  uint16_t *k, *v;
  int T, Hkv, D, group_size, pages, page_size;
};
hipError_t launch_kv4_gather(const Kv4GatherArgs& a, bool bf16, hipStream_t stream);

// Which kernel takes a call, and its grid.
enum Kv4Kernel { kKv4Tile, kKv4Pair, kKv4Parts, kKv4Blocks };
struct Kv4Launch {
  Kv4Kernel kernel;
  int rows;                 // of a block
  long long blocks;         // of the grid
  int resident, parts;      // kKv4Parts: blocks that run at a time, blocks beyond one a tile
  int threads;              // of a block
};
Kv4Launch kv4_attention_launch(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv, bool biased);
size_t kv4_attention_workspace(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv);
hipError_t launch_kv4_attention(const AttentionArgs& a, int group_size, bool bf16, hipStream_t stream);

// ---- the care of pages ----------------------------------------------------------------
constexpr int kMostCaches = 4096, kMostPages = 1 << 20;
struct PagePools {
  void* const* caches;
  const int64_t* page_bytes;
  int n;
};
hipError_t launch_copy_pages(const PagePools& pools, int pages, const int32_t* src, const int32_t* dst, int n,
                             hipStream_t stream);
struct CompactArgs {
  const int32_t *page_table, *kv_lens;
  int32_t *new_table, *moved_to, *live;
  int pages, table_stride, B, page_size;
  char* workspace;
};
size_t compact_workspace(int pages);
hipError_t launch_compact(const PagePools& pools, const CompactArgs& a, hipStream_t stream);

}  // namespace qmm
