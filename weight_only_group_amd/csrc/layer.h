// Internal declarations of the layer operators (include/qmm_layer.h): the
// validated arguments of each call and its launch.
#pragma once

#include "common.h"

namespace qmm {

// The workspace starts with the decode product's header of arrival counters
// (kept at zero between calls); every operator's data lies behind it.
constexpr size_t kWorkspaceHeader = size_t(kGemvMaxStrips) * 4;

// ---- mixture of experts ---------------------------------------------------------
constexpr int kMoeTokens = 64, kMoeExperts = 1024, kMoeTopK = 16;  // most of a call
constexpr int kMoeAssignments = kMoeTokens * kMoeTopK;
struct RouteArgs {
  const uint16_t* x;
  const uint16_t* router;
  int T, H, E, top_k;
  int renormalize;
  int32_t* ids;
  float* weights;
  float* logits;
  uint32_t* counters;
};
size_t moe_route_workspace(int T, int H, int E);
hipError_t launch_moe_route(const RouteArgs& a, bool bf16, hipStream_t stream);

// One packed weight of E experts.
struct ExpertPlanes {
  const uint32_t* qw;
  const uint32_t* qlo;
  const uint16_t* zeros;
  const uint16_t* scales;
};
struct MoeArgs {
  const uint16_t* x;
  const int32_t* ids;
  const float* weights;
  ExpertPlanes gate_up, down;
  uint16_t* y;
  char* workspace;
  int T, H, I, E, top_k;
  int gs_h, gs_i;  // rows per group of gate_up and down
};
size_t moe_workspace(int T, int H, int I, int E, int top_k);
hipError_t launch_moe(const MoeArgs& a, int bits, bool bf16, bool strips, hipStream_t stream);

// ---- append to the paged cache ----------------------------------------------------
struct AppendArgs {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  int T, Hq, Hkv, D, R, P;
  const float *cos, *sin;
  const int32_t* positions;
  const int64_t* slots;
  uint16_t *q_out, *k_cache, *v_cache;
  int pages, page_size;
};
hipError_t launch_kv_append(const AppendArgs& a, bool bf16, bool adjacent, hipStream_t stream);

// ---- attention to the paged cache ---------------------------------------------------
struct AttentionArgs {
  const uint16_t* q;
  long long q_stride;
  const uint16_t *k_cache, *v_cache;
  const int32_t *page_table, *kv_lens, *q_starts, *first, *end;
  const float* slopes;
  uint16_t* out;
  char* workspace;
  int T, Hq, Hkv, D, pages, page_size, table_stride, B, max_q, max_kv;
  float scale, softcap;
};
long long attention_blocks(int B, int Hq, int Hkv, int max_q, int max_kv);  // of the grid
size_t attention_workspace(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv);
hipError_t launch_attention(const AttentionArgs& a, bool bf16, hipStream_t stream);

// ---- log probabilities ----------------------------------------------------------------
constexpr int kMaxTop = 32;
enum class LogitType { kFp16, kBf16, kFp32 };
struct LogprobArgs {
  const void* logits;
  long long row_stride;
  int M, V, top;
  const int64_t* targets;
  float *logprob, *entropy, *top_logprobs;
  int32_t* top_ids;
  char* workspace;
};
size_t logprobs_workspace(int M, int V, int top);
hipError_t launch_logprobs(const LogprobArgs& a, LogitType type, hipStream_t stream);

}  // namespace qmm
