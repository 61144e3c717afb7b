// Argument checks that the C ABI's calls on layers and caches share.
#pragma once

#include <math.h>

#include "../../include/qmm_layer.h"
#include "layer.h"
#include "status.h"

namespace qmm {
namespace {

inline qmm_status check_flags(unsigned flags, unsigned known) {
  if (flags & ~known) return fail(QMM_ERR_FLAGS, "flags=0x%x: bits other than 0x%x", flags, known);
  return QMM_OK;
}

inline qmm_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return QMM_OK;
  if (!workspace || bytes < need)
    return fail(QMM_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? bytes : size_t(0));
  if (!aligned16(workspace)) return fail(QMM_ERR_ALIGN, "workspace must be 16-byte aligned");
  return QMM_OK;
}

inline bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

inline qmm_status check_heads(int Hq, int Hkv, int D) {
  if (!head_dim_ok(D)) return fail(QMM_ERR_SHAPE, "D=%d is not one of 64, 128, 256", D);
  if (Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq > 4096)
    return fail(QMM_ERR_SHAPE, "Hq=%d (at most 4096) must be a positive multiple of Hkv=%d", Hq, Hkv);
  return QMM_OK;
}

inline bool stride_ok(long long stride, long long least) { return stride >= least && stride % 8 == 0 && stride < (1ll << 40); }

inline bool attention_counts_ok(int B, int T, int Hq, int max_q, int max_kv) {
  return B >= 0 && T >= 0 && (long long)T * Hq < (1ll << 31) && max_q >= 0 && max_kv >= 0 && B <= 65535 &&
         (long long)max_q * Hq < (1ll << 31);
}

inline bool attention_size_ok(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv) {
  return head_dim_ok(D) && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hq <= 4096 && attention_counts_ok(B, T, Hq, max_q, max_kv) &&
         B >= 1 && T >= 1 && max_q >= 1;
}

// The kernels number a cache's rows (a token of a head) with 32 bits.
inline qmm_status check_cache(const void* k_cache, const void* v_cache, int pages, int Hkv, int page_size) {
  if (pages < 1 || page_size < 1 || (long long)pages * page_size >= (1ll << 31) || (long long)pages * page_size * Hkv >= (1ll << 31))
    return fail(QMM_ERR_SHAPE, "pages=%d and page_size=%d must be >= 1, pages * Hkv * page_size below 2^31", pages, page_size);
  if (!k_cache || !v_cache) return fail(QMM_ERR_NULL, "k_cache or v_cache is NULL");
  if (!aligned16(k_cache) || !aligned16(v_cache)) return fail(QMM_ERR_ALIGN, "k_cache and v_cache must be 16-byte aligned");
  return QMM_OK;
}

// ---- the append to a paged cache: sizes, then (with tokens) arrays ----------------------

inline qmm_status check_append_shape(const AppendArgs& a) {
  const qmm_status st = check_heads(a.Hq, a.Hkv, a.D);
  if (st != QMM_OK) return st;
  if (a.T < 0 || (long long)a.T * a.Hq * a.D >= (1ll << 31)) return fail(QMM_ERR_SHAPE, "T=%d: T * Hq * D must be below 2^31", a.T);
  if (a.R < 0 || a.R > a.D || a.R % 16) return fail(QMM_ERR_SHAPE, "R=%d must be a multiple of 16 in [0, D=%d]", a.R, a.D);
  if (a.R > 0 && a.P < 1) return fail(QMM_ERR_SHAPE, "P=%d must be >= 1", a.P);
  if (!stride_ok(a.q_stride, (long long)a.Hq * a.D) || !stride_ok(a.k_stride, (long long)a.Hkv * a.D) ||
      !stride_ok(a.v_stride, (long long)a.Hkv * a.D))
    return fail(QMM_ERR_SHAPE, "token strides must be multiples of 8 and at least a token's size");
  return QMM_OK;
}

inline qmm_status check_append_arrays(const AppendArgs& a) {
  const qmm_status st = check_cache(a.k_cache, a.v_cache, a.pages, a.Hkv, a.page_size);
  if (st != QMM_OK) return st;
  if (!a.q || !a.k || !a.v || !a.slots || !a.q_out || (a.R > 0 && (!a.cos || !a.sin || !a.positions)))
    return fail(QMM_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.q_out))
    return fail(QMM_ERR_ALIGN, "q, k, v and q_out must be 16-byte aligned");
  if (a.R > 0 && (!aligned16(a.cos) || !aligned16(a.sin) || !aligned(a.positions, 4)))
    return fail(QMM_ERR_ALIGN, "cos and sin must be 16-byte, positions 4-byte aligned");
  if (!aligned(a.slots, 8)) return fail(QMM_ERR_ALIGN, "slots must be 8-byte aligned");
  return QMM_OK;
}

// ---- the attention to a paged cache: sizes, then (with work) arrays ----------------------

inline qmm_status check_attention_shape(const AttentionArgs& a) {
  const qmm_status st = check_heads(a.Hq, a.Hkv, a.D);
  if (st != QMM_OK) return st;
  if (!attention_counts_ok(a.B, a.T, a.Hq, a.max_q, a.max_kv))
    return fail(QMM_ERR_SHAPE, "B=%d (at most 65535), T=%d, max_q=%d and max_kv=%d must be >= 0, T * Hq and max_q * Hq below 2^31", a.B,
                a.T, a.max_q, a.max_kv);
  if (!stride_ok(a.q_stride, (long long)a.Hq * a.D))
    return fail(QMM_ERR_SHAPE, "q_stride=%lld must be a multiple of 8, at least Hq * D", a.q_stride);
  if (!isfinite(a.scale) || !isfinite(a.softcap) || a.softcap < 0)
    return fail(QMM_ERR_SHAPE, "scale=%g and softcap=%g must be finite, softcap not negative", a.scale, a.softcap);
  return QMM_OK;
}

// A launch's threads (256 a block) are counted in 32 bits.
inline qmm_status check_attention_blocks(int B, int Hkv, int max_q, long long blocks) {
  if (blocks >= (1ll << 24))
    return fail(QMM_ERR_SHAPE, "B=%d, Hkv=%d and max_q=%d: 2^24 blocks and more; pass the long sequences in a call of their own", B, Hkv, max_q);
  return QMM_OK;
}

inline qmm_status check_attention_arrays(const AttentionArgs& a, long long blocks) {
  const qmm_status st = check_cache(a.k_cache, a.v_cache, a.pages, a.Hkv, a.page_size);
  if (st != QMM_OK) return st;
  if (a.table_stride < 1 || (long long)a.table_stride * a.page_size >= (1ll << 31) || a.max_kv > (long long)a.table_stride * a.page_size)
    return fail(QMM_ERR_SHAPE, "max_kv=%d must not exceed table_stride=%d * page_size=%d (below 2^31)", a.max_kv, a.table_stride,
                a.page_size);
  const qmm_status grid = check_attention_blocks(a.B, a.Hkv, a.max_q, blocks);
  if (grid != QMM_OK) return grid;
  if (!a.q || !a.page_table || !a.kv_lens || !a.q_starts || !a.out) return fail(QMM_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(a.q) || !aligned16(a.out)) return fail(QMM_ERR_ALIGN, "q and out must be 16-byte aligned");
  if (!aligned(a.page_table, 4) || !aligned(a.kv_lens, 4) || !aligned(a.q_starts, 4) || !aligned(a.first, 4) || !aligned(a.end, 4) ||
      !aligned(a.slopes, 4))
    return fail(QMM_ERR_ALIGN, "page_table, kv_lens, q_starts, first, end and slopes must be 4-byte aligned");
  return QMM_OK;
}

}  // namespace
}  // namespace qmm
