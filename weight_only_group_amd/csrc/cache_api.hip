// C ABI of the 4-bit cache and of the care of pages: argument validation and dispatch.
// Every check runs on the host before anything is enqueued.
#include "../../include/qmm_cache.h"
#include "cache.h"
#include "checks.h"

namespace {

using qmm::aligned;
using qmm::aligned16;
using qmm::check_append_arrays;
using qmm::check_append_shape;
using qmm::check_attention_arrays;
using qmm::check_attention_shape;
using qmm::check_cache;
using qmm::check_flags;
using qmm::check_workspace;
using qmm::fail;
using qmm::from_hip;
using qmm::ok;

bool kv4_sizes_ok(int D, int group_size) {
  return qmm::head_dim_ok(D) && (group_size == 32 || group_size == 64 || group_size == 128) && group_size <= D;
}

qmm_status check_kv4(int page_size, int D, int group_size) {
  if (!qmm::head_dim_ok(D)) return fail(QMM_ERR_SHAPE, "D=%d is not one of 64, 128, 256", D);
  if (!kv4_sizes_ok(D, group_size)) return fail(QMM_ERR_GROUP, "group_size=%d must be 32, 64 or 128 and at most D=%d", group_size, D);
  if (page_size < 1 || page_size % qmm::kBlockTokens)
    return fail(QMM_ERR_SHAPE, "page_size=%d must be a positive multiple of %d", page_size, qmm::kBlockTokens);
  return QMM_OK;
}

// A launch's blocks, counted as of 256 threads each.
long long blocks_of_256(const qmm::Kv4Launch& p) { return p.blocks * (p.threads / 256); }

qmm_status check_pools(void* const* caches, const int64_t* page_bytes, int n_caches, int pages) {
  if (n_caches < 0 || n_caches > qmm::kMostCaches) return fail(QMM_ERR_SHAPE, "n_caches=%d must be in [0, %d]", n_caches, qmm::kMostCaches);
  if (pages < 1) return fail(QMM_ERR_SHAPE, "pages=%d must be >= 1", pages);
  if (n_caches > 0 && (!caches || !page_bytes)) return fail(QMM_ERR_NULL, "caches or page_bytes is NULL");
  for (int i = 0; i < n_caches; ++i) {
    if (page_bytes[i] < 16 || page_bytes[i] % 16 || page_bytes[i] >= (1ll << 31))
      return fail(QMM_ERR_SHAPE, "page_bytes[%d]=%lld must be a positive multiple of 16 below 2^31", i, (long long)page_bytes[i]);
    if (!caches[i]) return fail(QMM_ERR_NULL, "caches[%d] is NULL", i);
    if (!aligned16(caches[i])) return fail(QMM_ERR_ALIGN, "caches[%d] must be 16-byte aligned", i);
  }
  return QMM_OK;
}

}  // namespace

static_assert(QMM_KV4_LARGEST == qmm::kKv4Largest && QMM_KV4_LARGEST_SCALE == qmm::kKv4LargestScale, "the limits of the kernels");

extern "C" {

size_t qmm_kv4_page_bytes(int page_size, int D, int group_size) {
  if (!kv4_sizes_ok(D, group_size) || page_size < 1 || page_size % qmm::kBlockTokens) return 0;
  return (size_t)(page_size / qmm::kBlockTokens) * qmm::kv4_block_bytes(D, D / group_size);
}

qmm_status qmm_kv4_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                          int64_t v_stride, int T, int Hq, int Hkv, int D, int group_size, const float* cos,
                          const float* sin, int R, int P, const int32_t* positions, const int64_t* slots,
                          uint16_t* q_out, uint8_t* k_cache, uint8_t* v_cache, int pages, int page_size, unsigned flags,
                          hipStream_t stream) {
  qmm_status st = check_flags(flags, QMM_BF16 | QMM_ADJACENT);
  if (st == QMM_OK) st = check_kv4(page_size, D, group_size);
  if (st != QMM_OK) return st;
  const qmm::AppendArgs a = {q, k, v, q_stride, k_stride, v_stride, T, Hq, Hkv, D, R, P, cos, sin, positions, slots,
                             q_out, reinterpret_cast<uint16_t*>(k_cache), reinterpret_cast<uint16_t*>(v_cache), pages, page_size};
  st = check_append_shape(a);
  if (st != QMM_OK) return st;
  if (T == 0) return ok();
  st = check_append_arrays(a);
  if (st != QMM_OK) return st;
  return from_hip(qmm::launch_kv4_append(a, group_size, (flags & QMM_BF16) != 0, (flags & QMM_ADJACENT) != 0, stream),
                  "qmm_kv4_append launch");
}

qmm_status qmm_kv4_gather(const uint8_t* k_cache, const uint8_t* v_cache, int pages, int Hkv, int page_size, int D,
                          int group_size, const int64_t* slots, int T, unsigned flags, uint16_t* k, uint16_t* v,
                          hipStream_t stream) {
  qmm_status st = check_flags(flags, QMM_BF16);
  if (st == QMM_OK) st = check_kv4(page_size, D, group_size);
  if (st != QMM_OK) return st;
  if (Hkv < 1 || Hkv > 4096) return fail(QMM_ERR_SHAPE, "Hkv=%d must be in [1, 4096]", Hkv);
  if (T < 0 || (long long)T * Hkv * D >= (1ll << 31)) return fail(QMM_ERR_SHAPE, "T=%d: T * Hkv * D must be in [0, 2^31)", T);
  if (T == 0) return ok();
  st = check_cache(k_cache, v_cache, pages, Hkv, page_size);
  if (st != QMM_OK) return st;
  if (!slots || !k || !v) return fail(QMM_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(k) || !aligned16(v)) return fail(QMM_ERR_ALIGN, "k and v must be 16-byte aligned");
  if (!aligned(slots, 8)) return fail(QMM_ERR_ALIGN, "slots must be 8-byte aligned");
  const qmm::Kv4GatherArgs a = {k_cache, v_cache, slots, k, v, T, Hkv, D, group_size, pages, page_size};
  return from_hip(qmm::launch_kv4_gather(a, (flags & QMM_BF16) != 0, stream), "qmm_kv4_gather launch");
}

size_t qmm_kv4_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv) {
  if (!qmm::attention_size_ok(B, T, Hq, Hkv, D, max_q, max_kv)) return 0;
  return qmm::kv4_attention_workspace(B, T, Hq, Hkv, D, max_q, max_kv);
}

qmm_status qmm_kv4_attention(const uint16_t* q, int64_t q_stride, int T, int Hq, int Hkv, int D, int group_size,
                             const uint8_t* k_cache, const uint8_t* v_cache, int pages, int page_size,
                             const int32_t* page_table, int table_stride, const int32_t* kv_lens,
                             const int32_t* q_starts, int B, int max_q, int max_kv, const int32_t* first,
                             const int32_t* end, float scale, float softcap, const float* slopes, unsigned flags,
                             uint16_t* out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  qmm_status st = check_flags(flags, QMM_BF16);
  if (st == QMM_OK) st = check_kv4(page_size, D, group_size);
  if (st != QMM_OK) return st;
  const qmm::AttentionArgs a = {q, q_stride, reinterpret_cast<const uint16_t*>(k_cache), reinterpret_cast<const uint16_t*>(v_cache),
                                page_table, kv_lens, q_starts, first, end, slopes, out, static_cast<char*>(workspace), T, Hq, Hkv, D,
                                pages, page_size, table_stride, B, max_q, max_kv, scale, softcap};
  st = check_attention_shape(a);
  if (st != QMM_OK) return st;
  if (T == 0 || B == 0 || max_q == 0) return ok();
  st = check_attention_arrays(a, blocks_of_256(qmm::kv4_attention_launch(B, T, Hq, Hkv, D, max_q, max_kv, slopes != nullptr)));
  if (st == QMM_OK)
    st = check_workspace(workspace, workspace_bytes, qmm::kv4_attention_workspace(B, T, Hq, Hkv, D, max_q, max_kv));
  if (st != QMM_OK) return st;
  return from_hip(qmm::launch_kv4_attention(a, group_size, (flags & QMM_BF16) != 0, stream), "qmm_kv4_attention launch");
}

qmm_status qmm_kv4_attention_plan_info(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv, int biased, int32_t* info,
                                       int n) {
  if (!qmm::attention_size_ok(B, T, Hq, Hkv, D, max_q, max_kv))
    return fail(QMM_ERR_SHAPE, "B=%d, T=%d, Hq=%d, Hkv=%d, D=%d, max_q=%d, max_kv=%d: no sizes of a launch", B, T, Hq, Hkv, D, max_q, max_kv);
  if (n > 0 && !info) return fail(QMM_ERR_NULL, "info is NULL");
  const qmm::Kv4Launch p = qmm::kv4_attention_launch(B, T, Hq, Hkv, D, max_q, max_kv, biased != 0);
  const qmm_status st = qmm::check_attention_blocks(B, Hkv, max_q, blocks_of_256(p));
  if (st != QMM_OK) return st;
  const int32_t v[6] = {p.kernel, p.rows, (int32_t)p.blocks, p.resident, p.parts,
                        qmm::device_topology().cus};
  for (int i = 0; i < n && i < 6; ++i) info[i] = v[i];
  return ok();
}

qmm_status qmm_kv_copy_pages(void* const* caches, const int64_t* page_bytes, int n_caches, int pages,
                             const int32_t* src, const int32_t* dst, int n, hipStream_t stream) {
  const qmm_status st = check_pools(caches, page_bytes, n_caches, pages);
  if (st != QMM_OK) return st;
  if (n < 0) return fail(QMM_ERR_SHAPE, "n=%d must be >= 0", n);
  if (n == 0 || n_caches == 0) return ok();
  if (!src || !dst) return fail(QMM_ERR_NULL, "src or dst is NULL");
  if (!aligned(src, 4) || !aligned(dst, 4)) return fail(QMM_ERR_ALIGN, "src and dst must be 4-byte aligned");
  return from_hip(qmm::launch_copy_pages({caches, page_bytes, n_caches}, pages, src, dst, n, stream), "qmm_kv_copy_pages launch");
}

size_t qmm_kv_compact_workspace_bytes(int pages) {
  return pages >= 1 && pages <= qmm::kMostPages ? qmm::compact_workspace(pages) : 0;
}

qmm_status qmm_kv_compact(void* const* caches, const int64_t* page_bytes, int n_caches, int pages,
                          const int32_t* page_table, int table_stride, const int32_t* kv_lens, int B, int page_size,
                          int32_t* new_table, int32_t* moved_to, int32_t* live, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  qmm_status st = check_pools(caches, page_bytes, n_caches, pages);
  if (st != QMM_OK) return st;
  if (pages > qmm::kMostPages) return fail(QMM_ERR_SHAPE, "pages=%d: at most %d", pages, qmm::kMostPages);
  if (B < 0 || table_stride < 1 || (long long)B * table_stride >= (1ll << 31))
    return fail(QMM_ERR_SHAPE, "B=%d must be >= 0 and table_stride=%d >= 1, B * table_stride below 2^31", B, table_stride);
  if (page_size < 1) return fail(QMM_ERR_SHAPE, "page_size=%d must be >= 1", page_size);
  if (!moved_to || !live || (B > 0 && (!page_table || !kv_lens || !new_table))) return fail(QMM_ERR_NULL, "a required pointer is NULL");
  if (!aligned(page_table, 4) || !aligned(kv_lens, 4) || !aligned(new_table, 4) || !aligned(moved_to, 4) || !aligned(live, 4))
    return fail(QMM_ERR_ALIGN, "page_table, kv_lens, new_table, moved_to and live must be 4-byte aligned");
  st = check_workspace(workspace, workspace_bytes, qmm::compact_workspace(pages));
  if (st != QMM_OK) return st;
  const qmm::CompactArgs a = {page_table, kv_lens, new_table, moved_to, live, pages, table_stride, B, page_size,
                              static_cast<char*>(workspace)};
  return from_hip(qmm::launch_compact({caches, page_bytes, n_caches}, a, stream), "qmm_kv_compact launch");
}

}  // extern "C"
