/*
 * qmm_cache.h -- C ABI of a paged key/value cache held in 4 bits and of the care
 * of a cache's pages, for AMD Instinct MI355X (gfx950): the append that
 * quantises keys and values, reading tokens back, the attention to such a
 * cache, copying pages, and packing the pages in use.
 *
 * The conventions are those of qmm_layer.h, whose qmm_kv_append and
 * qmm_attention do the same on a cache of 16-bit values: device pointers,
 * arguments checked on the host before anything is enqueued, values that only
 * the device sees stated at each call, the same workspaces.
 *
 * The 4-bit cache: k_cache and v_cache are (pages, Hkv, qmm_kv4_page_bytes())
 * bytes. Slot s is token s % page_size of page s / page_size. The D channels
 * of a token's head fall into groups of group_size; a group has a scale s and
 * a middle m, both fp16 (s with at most 8 significant bits, so that s times a
 * code's distance from 8 is exact in fp16), and code c of it stands for
 *   m + s (c - 8)
 * A group whose s or m is not finite, or whose s is beyond +-QMM_KV4_LARGEST_SCALE
 * (24 s is then no fp16 number; qmm_kv4_append gives 2192 at most), stands for NaN. The
 * format is the same for fp16 and bf16 queries. A head's tokens of a page lie in blocks of eight
 * tokens, one behind another, each of 4 D + 32 D / group_size bytes:
 *   keys:   codes (8 tokens, D / 8 words), then fp16 (8 tokens, [s, m], groups);
 *           word (D / 32) g + i of a token (little-endian, 0 <= g < 4) has channels
 *           32 i + 8 g + e, 0 <= e < 8: even e in nibble e / 2, odd e in nibble 4 + e / 2
 *   values: codes (D / 4, 8 tokens, 16-bit words), channel 4 n + r in nibble r of word
 *           n, then fp16 (groups, [s, m], 8 tokens)
 * Requirements of every call on it: D 64, 128 or 256; group_size 32, 64 or
 * 128, dividing D; page_size a positive multiple of 8; pages * Hkv * page_size
 * < 2^31; k_cache and v_cache 16-byte aligned.
 */
#ifndef QMM_CACHE_H
#define QMM_CACHE_H

#include "qmm_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QMM_KV4_LARGEST 16384      /* keys and values are cut to +-16384 */
#define QMM_KV4_LARGEST_SCALE 2728 /* of a group that stands for numbers */

/* Bytes of one head of a page: page_size (D / 2 + 4 D / group_size); 0 for arguments that no call takes. */
size_t qmm_kv4_page_bytes(int page_size, int D, int group_size);

/*
 * qmm_kv4_append -- qmm_kv_append to a 4-bit cache: rotates queries and keys of T
 * new tokens and quantises keys and values into their slots. A key is rotated
 * and rounded once to fp32. Of a group's values x, cut to +-QMM_KV4_LARGEST (lo and hi
 * the least and largest), in fp32 arithmetic:
 *   s = fp16(bf16((hi - lo) / 15)),  m = fp16(lo + 8 s),
 *   c = 8 + rint((x - m) / s), cut to [0, 15];  8 where s is 0
 * (all roundings to nearest even). A group with a NaN gets NaN for s and m.
 * Arguments, requirements and flags are qmm_kv_append's (and those above); the
 * eight tokens of a block may come in any calls and any order.
 */
qmm_status qmm_kv4_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                          int64_t v_stride, int T, int Hq, int Hkv, int D, int group_size, const float* cos,
                          const float* sin, int R, int P, const int32_t* positions, const int64_t* slots,
                          uint16_t* q_out, uint8_t* k_cache, uint8_t* v_cache, int pages, int page_size, unsigned flags,
                          hipStream_t stream);

/*
 * qmm_kv4_gather -- tokens of a 4-bit cache as 16-bit values: k[t], v[t] (T, Hkv, D)
 * dense, fp16 or (QMM_BF16) bf16, are those of slots[t] (int64), each m + s (c - 8)
 * in fp32 rounded once to the type. Slots may repeat; one outside the cache gives 0.
 * Requirements: T * Hkv * D < 2^31; k and v 16-byte aligned, slots 8-byte.
 */
qmm_status qmm_kv4_gather(const uint8_t* k_cache, const uint8_t* v_cache, int pages, int Hkv, int page_size, int D,
                          int group_size, const int64_t* slots, int T, unsigned flags, uint16_t* k, uint16_t* v,
                          hipStream_t stream);

/*
 * qmm_kv4_attention -- qmm_attention to a 4-bit cache: the same formulas, masks,
 * arguments and requirements (and those above), with keys and values as the
 * cache's codes stand for, exactly (a scale of more than 8 significant bits, which no call
 * writes, may put s (c - 8) off by s / 64), and sums in fp32. Of a query head's
 * channels those smaller than 2^-14 of its largest one (bf16: 2^-17) are rounded to
 * steps of 2^-24 of the power of two below that. The weights exp(s) are rounded to
 * fp16 (for bf16 data too; weights below 2^-32 of a row's largest count as 0), the same
 * rounded weights make the denominator. A query with a value that is not finite
 * gives NaN where it sees a key.
 */
size_t qmm_kv4_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv);
qmm_status qmm_kv4_attention(const uint16_t* q, int64_t q_stride, int T, int Hq, int Hkv, int D, int group_size,
                             const uint8_t* k_cache, const uint8_t* v_cache, int pages, int page_size,
                             const int32_t* page_table, int table_stride, const int32_t* kv_lens,
                             const int32_t* q_starts, int B, int max_q, int max_kv, const int32_t* first,
                             const int32_t* end, float scale, float softcap, const float* slopes, unsigned flags,
                             uint16_t* out, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * qmm_kv4_attention_plan_info -- the launch qmm_kv4_attention makes for these sizes on the
 * current device, with (biased) or without slopes, for tests and measurement. Host only:
 * no work is enqueued. Writes min(n, 6) ints:
 *   info[0] kernel: 0 = a tile of 16 rows a block, 1 = two tiles a block, 2 = tiles in
 *           parts of their keys, which blocks share, 3 = blocks of many rows
 *   info[1] rows of a block     info[2] blocks of the grid
 *   info[3] kernel 2: blocks that run at a time, for which the parts are cut, else 0
 *   info[4] kernel 2: blocks that the parts may come to beyond one a tile, else 0
 *   info[5] compute units of the device
 * Returns QMM_ERR_NULL for a NULL info with n > 0, QMM_ERR_SHAPE for sizes that
 * qmm_kv4_attention would reject or for which it launches nothing, else QMM_OK.
 */
qmm_status qmm_kv4_attention_plan_info(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv, int biased, int32_t* info,
                                       int n);

/*
 * The care of pages, for caches of any kind: n_caches arrays (one layer's k_cache,
 * another's v_cache, ...), each of `pages` pages, cache i of page_bytes[i] bytes a
 * page (all heads). `caches` and `page_bytes` are host arrays of n_caches, read
 * before the call returns.
 * Requirements: 0 <= n_caches <= 4096; pages >= 1; caches 16-byte aligned, page_bytes positive
 * multiples of 16 below 2^31; caches must not overlap.
 *
 * qmm_kv_copy_pages -- page dst[i] of every cache becomes page src[i], i < n: pages
 * of a forked sequence that is to write on, a prefix for another owner. src and dst (n,) int32. A pair with an
 * index outside [0, pages) is left out. A page may be copied many times; no
 * page may be in dst twice, nor in dst and (of another pair) in src.
 */
qmm_status qmm_kv_copy_pages(void* const* caches, const int64_t* page_bytes, int n_caches, int pages,
                             const int32_t* src, const int32_t* dst, int n, hipStream_t stream);

/*
 * qmm_kv_compact -- packs the pages in use into the lowest ones. In use are the
 * pages page_table[b, i] with i < ceil(kv_lens[b] / page_size) (and i <
 * table_stride), those of several sequences once; `live` of them. Pages in use
 * below `live` stay; the others, in rising order, go to the free ones below
 * `live`, in rising order. After it the pages from `live` on are free.
 *   page_table (B, table_stride) int32, kv_lens (B,) int32
 *   new_table  (B, table_stride): page_table with the places in use renamed, the others as they were
 *   moved_to   (pages,) int32: where each page is now, -1 for a free one
 *   live       (1,) int32
 * new_table may be page_table. An entry in use outside [0, pages) is no page and left as it is.
 * Requirements: pages <= 2^20, B * table_stride < 2^31, page_size >= 1; int32 arrays 4-byte aligned.
 */
size_t qmm_kv_compact_workspace_bytes(int pages);
qmm_status qmm_kv_compact(void* const* caches, const int64_t* page_bytes, int n_caches, int pages,
                          const int32_t* page_table, int table_stride, const int32_t* kv_lens, int B, int page_size,
                          int32_t* new_table, int32_t* moved_to, int32_t* live, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_CACHE_H */
