// C ABI of the layer operators: argument validation and dispatch. Every check
// runs on the host before anything is enqueued.
#include <math.h>

#include "../../include/qmm_layer.h"
#include "layer.h"
#include "status.h"

namespace {

using qmm::aligned;
using qmm::aligned16;
using qmm::fail;
using qmm::from_hip;
using qmm::ok;

qmm_status check_flags(unsigned flags, unsigned known) {
  if (flags & ~known) return fail(QMM_ERR_FLAGS, "flags=0x%x: bits other than 0x%x", flags, known);
  return QMM_OK;
}

qmm_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return QMM_OK;
  if (!workspace || bytes < need)
    return fail(QMM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? bytes : size_t(0));
  if (!aligned16(workspace)) return fail(QMM_ERR_ALIGN, "workspace must be 16-byte aligned");
  return QMM_OK;
}

// ---- mixture of experts ---------------------------------------------------------

static_assert(QMM_MOE_MAX_TOKENS == qmm::kMoeTokens && QMM_MOE_MAX_EXPERTS == qmm::kMoeExperts && QMM_MOE_MAX_TOP_K == qmm::kMoeTopK &&
              QMM_LOGPROBS_MAX_TOP == qmm::kMaxTop, "limits of the kernels");

qmm_status check_route_shape(int T, int H, int E) {
  if (T < 0 || T > QMM_MOE_MAX_TOKENS) return fail(QMM_ERR_SHAPE, "T=%d must be in [0, %d]", T, QMM_MOE_MAX_TOKENS);
  if (H < 32 || H % 32 || H > (1 << 20)) return fail(QMM_ERR_SHAPE, "H=%d must be a multiple of 32 in [32, 2^20]", H);
  if (E < 1 || E > QMM_MOE_MAX_EXPERTS) return fail(QMM_ERR_SHAPE, "E=%d must be in [1, %d]", E, QMM_MOE_MAX_EXPERTS);
  return QMM_OK;
}

bool moe_shape_ok(int T, int H, int I, int E, int top_k) {
  return T >= 0 && T <= QMM_MOE_MAX_TOKENS && H >= 32 && H % 32 == 0 && H <= (1 << 20) && I >= 32 && I % 32 == 0 &&
         I <= (1 << 20) && E >= 1 && E <= QMM_MOE_MAX_EXPERTS && top_k >= 1 && top_k <= QMM_MOE_MAX_TOP_K;
}

qmm_status check_experts(const qmm_experts* w, const char* what, int bits) {
  if (!w || !w->qweight || !w->zeros || !w->scales) return fail(QMM_ERR_NULL, "%s: a required pointer is NULL", what);
  if (bits == 3 && !w->qweight_lo) return fail(QMM_ERR_NULL, "%s: qweight_lo (1-bit plane) is NULL for 3-bit codes", what);
  if (!aligned16(w->qweight) || !aligned16(w->zeros) || !aligned16(w->scales) || (bits == 3 && !aligned16(w->qweight_lo)))
    return fail(QMM_ERR_ALIGN, "%s: planes, zeros and scales must be 16-byte aligned", what);
  return QMM_OK;
}

qmm::ExpertPlanes planes(const qmm_experts* w) {
  return {reinterpret_cast<const uint32_t*>(w->qweight), reinterpret_cast<const uint32_t*>(w->qweight_lo), w->zeros,
          w->scales};
}

// ---- attention ------------------------------------------------------------------

bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

qmm_status check_heads(int Hq, int Hkv, int D) {
  if (!head_dim_ok(D)) return fail(QMM_ERR_SHAPE, "D=%d is not one of 64, 128, 256", D);
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq > 4096)
    return fail(QMM_ERR_SHAPE, "Hq=%d (at most 4096) must be a positive multiple of Hkv=%d", Hq, Hkv);
  return QMM_OK;
}

// The kernels number a cache's rows (a token of a head) with 32 bits.
qmm_status check_cache(const void* k_cache, const void* v_cache, int pages, int Hkv, int page_size) {
  if (pages < 1 || page_size < 1 || (long long)pages * page_size >= (1ll << 31) || (long long)pages * page_size * Hkv >= (1ll << 31))
    return fail(QMM_ERR_SHAPE, "pages=%d and page_size=%d must be >= 1, pages * Hkv * page_size below 2^31", pages, page_size);
  if (!k_cache || !v_cache) return fail(QMM_ERR_NULL, "k_cache or v_cache is NULL");
  if (!aligned16(k_cache) || !aligned16(v_cache)) return fail(QMM_ERR_ALIGN, "k_cache and v_cache must be 16-byte aligned");
  return QMM_OK;
}

bool stride_ok(long long stride, long long least) { return stride >= least && stride % 8 == 0 && stride < (1ll << 40); }

bool attention_counts_ok(int B, int T, int Hq, int max_q, int max_kv) {
  return B >= 0 && T >= 0 && (long long)T * Hq < (1ll << 31) && max_q >= 0 && max_kv >= 0 && B <= 65535 &&
         (long long)max_q * Hq < (1ll << 31);
}

}  // namespace

extern "C" {

size_t qmm_moe_route_workspace_bytes(int T, int H, int E) {
  if (T < 1 || T > QMM_MOE_MAX_TOKENS || H < 32 || H % 32 || H > (1 << 20) || E < 1 || E > QMM_MOE_MAX_EXPERTS) return 0;
  return qmm::moe_route_workspace(T, H, E);
}

qmm_status qmm_moe_route(const uint16_t* x, int T, int H, const uint16_t* router, int E, int top_k, unsigned flags,
                         int32_t* ids, float* weights, float* logits, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  qmm_status st = check_flags(flags, QMM_BF16 | QMM_RENORMALIZE);
  if (st == QMM_OK) st = check_route_shape(T, H, E);
  if (st != QMM_OK) return st;
  if (top_k < 1 || top_k > E || top_k > QMM_MOE_MAX_TOP_K)
    return fail(QMM_ERR_SHAPE, "top_k=%d must be in [1, min(E=%d, %d)]", top_k, E, QMM_MOE_MAX_TOP_K);
  if (T == 0) return ok();
  if (!x || !router || !ids || !weights || !logits) return fail(QMM_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(x) || !aligned16(router)) return fail(QMM_ERR_ALIGN, "x and router must be 16-byte aligned");
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(logits, 4))
    return fail(QMM_ERR_ALIGN, "ids, weights and logits must be 4-byte aligned");
  st = check_workspace(workspace, workspace_bytes, qmm::moe_route_workspace(T, H, E));
  if (st != QMM_OK) return st;
  const qmm::RouteArgs a = {x, router, T, H, E, top_k, (flags & QMM_RENORMALIZE) != 0, ids, weights, logits,
                            static_cast<uint32_t*>(workspace)};
  return from_hip(qmm::launch_moe_route(a, (flags & QMM_BF16) != 0, stream), "qmm_moe_route launch");
}

size_t qmm_moe_workspace_bytes(int T, int H, int I, int E, int top_k) {
  return T > 0 && moe_shape_ok(T, H, I, E, top_k) ? qmm::moe_workspace(T, H, I, E, top_k) : 0;
}

qmm_status qmm_moe(const uint16_t* x, int T, int H, int I, int E, int top_k, const int32_t* ids, const float* weights,
                   const qmm_experts* gate_up, const qmm_experts* down, int bits, int group_size, unsigned flags,
                   uint16_t* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  qmm_status st = check_flags(flags, QMM_BF16 | QMM_STRIPS);
  if (st != QMM_OK) return st;
  if (!qmm::bits_ok(bits)) return fail(QMM_ERR_BITS, "bits=%d is not one of 1, 2, 3, 4, 8", bits);
  if (!moe_shape_ok(T, H, I, E, top_k))
    return fail(QMM_ERR_SHAPE, "T=%d must be in [0, %d], H=%d and I=%d multiples of 32 in [32, 2^20], E=%d in [1, %d], "
                "top_k=%d in [1, %d]", T, QMM_MOE_MAX_TOKENS, H, I, E, QMM_MOE_MAX_EXPERTS, top_k, QMM_MOE_MAX_TOP_K);
  if (group_size != -1 && (group_size <= 0 || group_size % 32 || H % group_size || I % group_size))
    return fail(QMM_ERR_GROUP, "group_size=%d must be -1 or a positive multiple of 32 dividing H=%d and I=%d", group_size,
                H, I);
  // The kernels address one expert's plane and scales with 32-bit byte offsets.
  if ((unsigned long long)H * 2 * I * (bits == 3 ? 2 : bits) / 8 >= (1ull << 32))
    return fail(QMM_ERR_SHAPE, "one expert's plane of H=%d by 2I=%d must be smaller than 4 GiB", H, 2 * I);
  if ((unsigned long long)T * top_k * I * 4 >= (1ull << 32))
    return fail(QMM_ERR_SHAPE, "T=%d, top_k=%d and I=%d: the intermediate must be smaller than 4 GiB", T, top_k, I);
  if (T == 0) return ok();
  if (!x || !ids || !weights || !y) return fail(QMM_ERR_NULL, "a required pointer is NULL");
  st = check_experts(gate_up, "gate_up", bits);
  if (st == QMM_OK) st = check_experts(down, "down", bits);
  if (st != QMM_OK) return st;
  if (!aligned16(x) || !aligned16(y)) return fail(QMM_ERR_ALIGN, "x and y must be 16-byte aligned");
  if (!aligned(ids, 4) || !aligned(weights, 4)) return fail(QMM_ERR_ALIGN, "ids and weights must be 4-byte aligned");
  st = check_workspace(workspace, workspace_bytes, qmm::moe_workspace(T, H, I, E, top_k));
  if (st != QMM_OK) return st;
  const qmm::MoeArgs a = {x, ids, weights, planes(gate_up), planes(down), y, static_cast<char*>(workspace), T, H, I, E,
                          top_k, qmm::group_rows(H, group_size), qmm::group_rows(I, group_size)};
  return from_hip(qmm::launch_moe(a, bits, (flags & QMM_BF16) != 0, (flags & QMM_STRIPS) != 0, stream), "qmm_moe launch");
}

qmm_status qmm_kv_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                         int64_t v_stride, int T, int Hq, int Hkv, int D, const float* cos, const float* sin, int R,
                         int P, const int32_t* positions, const int64_t* slots, uint16_t* q_out, uint16_t* k_cache,
                         uint16_t* v_cache, int pages, int page_size, unsigned flags, hipStream_t stream) {
  qmm_status st = check_flags(flags, QMM_BF16 | QMM_ADJACENT);
  if (st == QMM_OK) st = check_heads(Hq, Hkv, D);
  if (st != QMM_OK) return st;
  if (T < 0 || (long long)T * Hq * D >= (1ll << 31)) return fail(QMM_ERR_SHAPE, "T=%d: T * Hq * D must be below 2^31", T);
  if (R < 0 || R > D || R % 16) return fail(QMM_ERR_SHAPE, "R=%d must be a multiple of 16 in [0, D=%d]", R, D);
  if (R > 0 && P < 1) return fail(QMM_ERR_SHAPE, "P=%d must be >= 1", P);
  if (!stride_ok(q_stride, (long long)Hq * D) || !stride_ok(k_stride, (long long)Hkv * D) ||
      !stride_ok(v_stride, (long long)Hkv * D))
    return fail(QMM_ERR_SHAPE, "token strides must be multiples of 8 and at least a token's size");
  if (T == 0) return ok();
  st = check_cache(k_cache, v_cache, pages, Hkv, page_size);
  if (st != QMM_OK) return st;
  if (!q || !k || !v || !slots || !q_out || (R > 0 && (!cos || !sin || !positions)))
    return fail(QMM_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out))
    return fail(QMM_ERR_ALIGN, "q, k, v and q_out must be 16-byte aligned");
  if (R > 0 && (!aligned16(cos) || !aligned16(sin) || !aligned(positions, 4)))
    return fail(QMM_ERR_ALIGN, "cos and sin must be 16-byte, positions 4-byte aligned");
  if (!aligned(slots, 8)) return fail(QMM_ERR_ALIGN, "slots must be 8-byte aligned");
  const qmm::AppendArgs a = {q, k, v, q_stride, k_stride, v_stride, T, Hq, Hkv, D, R, P, cos, sin, positions, slots,
                             q_out, k_cache, v_cache, pages, page_size};
  return from_hip(qmm::launch_kv_append(a, (flags & QMM_BF16) != 0, (flags & QMM_ADJACENT) != 0, stream),
                  "qmm_kv_append launch");
}

size_t qmm_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv) {
  if (!head_dim_ok(D) || Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq > 4096 || !attention_counts_ok(B, T, Hq, max_q, max_kv) ||
      B < 1 || T < 1 || max_q < 1)
    return 0;
  return qmm::attention_workspace(B, T, Hq, Hkv, D, max_q, max_kv);
}

qmm_status qmm_attention(const uint16_t* q, int64_t q_stride, int T, int Hq, int Hkv, int D, const uint16_t* k_cache,
                         const uint16_t* v_cache, int pages, int page_size, const int32_t* page_table, int table_stride,
                         const int32_t* kv_lens, const int32_t* q_starts, int B, int max_q, int max_kv,
                         const int32_t* first, const int32_t* end, float scale, float softcap, const float* slopes,
                         unsigned flags, uint16_t* out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  qmm_status st = check_flags(flags, QMM_BF16);
  if (st == QMM_OK) st = check_heads(Hq, Hkv, D);
  if (st != QMM_OK) return st;
  if (!attention_counts_ok(B, T, Hq, max_q, max_kv))
    return fail(QMM_ERR_SHAPE, "B=%d (at most 65535), T=%d, max_q=%d and max_kv=%d must be >= 0, T * Hq and max_q * Hq below 2^31", B, T,
                max_q, max_kv);
  if (!stride_ok(q_stride, (long long)Hq * D))
    return fail(QMM_ERR_SHAPE, "q_stride=%lld must be a multiple of 8, at least Hq * D", (long long)q_stride);
  if (!isfinite(scale) || !isfinite(softcap) || softcap < 0)
    return fail(QMM_ERR_SHAPE, "scale=%g and softcap=%g must be finite, softcap not negative", scale, softcap);
  if (T == 0 || B == 0 || max_q == 0) return ok();
  st = check_cache(k_cache, v_cache, pages, Hkv, page_size);
  if (st != QMM_OK) return st;
  if (table_stride < 1 || (long long)table_stride * page_size >= (1ll << 31) || max_kv > (long long)table_stride * page_size)
    return fail(QMM_ERR_SHAPE, "max_kv=%d must not exceed table_stride=%d * page_size=%d (below 2^31)", max_kv,
                table_stride, page_size);
  // A launch's threads (256 a block) are counted in 32 bits.
  if (qmm::attention_blocks(B, Hq, Hkv, max_q, max_kv) >= (1ll << 24))
    return fail(QMM_ERR_SHAPE, "B=%d, Hkv=%d and max_q=%d: 2^24 blocks and more; pass the long sequences in a call of their own", B,
                Hkv, max_q);
  if (!q || !page_table || !kv_lens || !q_starts || !out) return fail(QMM_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(q) || !aligned16(out)) return fail(QMM_ERR_ALIGN, "q and out must be 16-byte aligned");
  if (!aligned(page_table, 4) || !aligned(kv_lens, 4) || !aligned(q_starts, 4) || !aligned(first, 4) || !aligned(end, 4) ||
      !aligned(slopes, 4))
    return fail(QMM_ERR_ALIGN, "page_table, kv_lens, q_starts, first, end and slopes must be 4-byte aligned");
  st = check_workspace(workspace, workspace_bytes, qmm::attention_workspace(B, T, Hq, Hkv, D, max_q, max_kv));
  if (st != QMM_OK) return st;
  const qmm::AttentionArgs a = {q, q_stride, k_cache, v_cache, page_table, kv_lens, q_starts, first, end, slopes, out,
                                static_cast<char*>(workspace), T, Hq, Hkv, D, pages, page_size, table_stride, B, max_q,
                                max_kv, scale, softcap};
  return from_hip(qmm::launch_attention(a, (flags & QMM_BF16) != 0, stream), "qmm_attention launch");
}

size_t qmm_logprobs_workspace_bytes(int M, int V, int top) {
  return M > 0 && V > 0 && top >= 0 && top <= QMM_LOGPROBS_MAX_TOP ? qmm::logprobs_workspace(M, V, top) : 0;
}

qmm_status qmm_logprobs(const void* logits, int64_t row_stride, int M, int V, const int64_t* targets, int top,
                        unsigned flags, float* logprob, float* entropy, float* top_logprobs, int32_t* top_ids,
                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
  qmm_status st = check_flags(flags, QMM_BF16 | QMM_FP32);
  if (st != QMM_OK) return st;
  if ((flags & QMM_BF16) && (flags & QMM_FP32)) return fail(QMM_ERR_FLAGS, "QMM_BF16 and QMM_FP32 exclude each other");
  if (M < 0 || V < 1 || V > (1 << 30)) return fail(QMM_ERR_SHAPE, "M=%d must be >= 0 and V=%d in [1, 2^30]", M, V);
  if (top < 0 || top > QMM_LOGPROBS_MAX_TOP || top > V)
    return fail(QMM_ERR_SHAPE, "top=%d must be in [0, min(V=%d, %d)]", top, V, QMM_LOGPROBS_MAX_TOP);
  if (row_stride < V || row_stride >= (1ll << 40))
    return fail(QMM_ERR_SHAPE, "row_stride=%lld must be at least V=%d", (long long)row_stride, V);
  if (M == 0) return ok();
  if (!logits || !entropy || (targets == nullptr) != (logprob == nullptr) || (top > 0 && (!top_logprobs || !top_ids)))
    return fail(QMM_ERR_NULL, "a required pointer is NULL (targets and logprob come together)");
  const bool fp32 = (flags & QMM_FP32) != 0;
  if (!aligned(logits, fp32 ? 4 : 2) || !aligned(targets, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
      !aligned(top_logprobs, 4) || !aligned(top_ids, 4))
    return fail(QMM_ERR_ALIGN, "an array is not aligned to its elements");
  st = check_workspace(workspace, workspace_bytes, qmm::logprobs_workspace(M, V, top));
  if (st != QMM_OK) return st;
  const qmm::LogprobArgs a = {logits, row_stride, M, V, top, targets, logprob, entropy, top_logprobs, top_ids,
                              static_cast<char*>(workspace)};
  const qmm::LogitType type = fp32 ? qmm::LogitType::kFp32
                              : (flags & QMM_BF16) ? qmm::LogitType::kBf16 : qmm::LogitType::kFp16;
  return from_hip(qmm::launch_logprobs(a, type, stream), "qmm_logprobs launch");
}

}  // extern "C"
