/*
 * qmm_layer.h -- C ABI of the operators between the quantised products of a
 * decoder layer (qmm.h), for AMD Instinct MI355X (gfx950): a mixture-of-experts
 * layer with quantised experts, the append of keys and values to a paged cache
 * with the position rotation on the way, the attention that reads that cache,
 * and log probabilities of tokens.
 *
 * The conventions are those of qmm.h: device pointers, row-major arrays, fp16
 * (or, with QMM_BF16, bf16) data as uint16_t bit patterns, the caller owns
 * every buffer, arguments are checked on the host before anything is enqueued,
 * QMM_OK means the work was enqueued on `stream`, qmm_last_error() holds the
 * message of a refusal. Sizes that count tokens, sequences or rows may be zero:
 * the call then does nothing and returns QMM_OK.
 *
 * Values that only the device sees (expert ids, positions, slots, page ids,
 * lengths) are not refused; what a value outside its range does is stated at
 * each call, and none reads or writes outside the arrays given.
 *
 * Workspaces are as qmm_gemv's: a caller-owned buffer, 16-byte aligned, at
 * least as large as the call's ..._workspace_bytes() says, zero-filled once when
 * it is allocated. It starts with the same 128 KiB header of arrival counters,
 * which every call leaves at zero, so that one buffer serves calls of every
 * kind (qmm_gemv's too), as long as calls that share it do not overlap in time.
 */
#ifndef QMM_LAYER_H
#define QMM_LAYER_H

#include "qmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags, next to QMM_BF16 and QMM_STRIPS; each call names those it takes and
 * refuses others with QMM_ERR_FLAGS. */
#define QMM_RENORMALIZE 4u /* qmm_moe_route: the chosen experts' weights sum to one */
#define QMM_ADJACENT 8u    /* qmm_kv_append: rotated pairs are neighbours (2i, 2i + 1), else (i, i + R / 2) */
#define QMM_FP32 16u       /* qmm_logprobs: logits are fp32 */

#define QMM_MOE_MAX_TOKENS 64
#define QMM_MOE_MAX_EXPERTS 1024
#define QMM_MOE_MAX_TOP_K 16
#define QMM_LOGPROBS_MAX_TOP 32

/*
 * qmm_moe_route -- which experts each token goes to, and with what weight:
 *   logits[t, e] = sum_h x[t, h] router[e, h]                (fp32)
 *   ids[t, :]    = the top_k experts of the largest logits, largest first
 *                  (equal logits: the lower expert first)
 *   weights[t, j] = exp(logits[t, ids[t, j]]) / sum exp(logits[t, e])  over all
 *                  e, or over the chosen ones with QMM_RENORMALIZE
 *   x       (T, H), router (E, H); fp16, or bf16 with QMM_BF16
 *   ids     (T, top_k) int32; weights (T, top_k) fp32; logits (T, E) fp32
 * Requirements: 0 <= T <= 64, H % 32 == 0, 1 <= E <= 1024, 1 <= top_k <=
 * min(16, E); x and router 16-byte aligned, the rest 4-byte aligned. Flags:
 * QMM_BF16, QMM_RENORMALIZE. A NaN logit counts as the largest of all, and the
 * token's weights are NaN.
 */
size_t qmm_moe_route_workspace_bytes(int T, int H, int E);
qmm_status qmm_moe_route(const uint16_t* x, int T, int H, const uint16_t* router, int E, int top_k, unsigned flags,
                         int32_t* ids, float* weights, float* logits, void* workspace, size_t workspace_bytes,
                         hipStream_t stream);

/* The packed weights of E experts, one behind another: each expert's K x N
 * weight as qmm_pack (or, with QMM_STRIPS, qmm_to_strips) lays it out. */
typedef struct qmm_experts {
  const int32_t* qweight;    /* (E, plane) words                            */
  const int32_t* qweight_lo; /* (E, plane) words of the 1-bit plane, 3 bits */
  const uint16_t* zeros;     /* (E, G, N)                                   */
  const uint16_t* scales;    /* (E, G, N)                                   */
} qmm_experts;

/*
 * qmm_moe -- the experts' part of a mixture-of-experts layer, for a few tokens:
 *   (g, u) = x[t] @ dequantize(gate_up[e])      e = ids[t, j]; g the first I columns, u the others
 *   h      = g / (1 + exp(-g)) * u
 *   y[t]   = sum_j weights[t, j] * (h @ dequantize(down[e]))
 *   x       (T, H);  ids (T, top_k) int32, weights (T, top_k) fp32, as qmm_moe_route gives them
 *   gate_up E weights of H x 2I, down E weights of I x H, both of `bits` and `group_size`
 *   y       (T, H); sums in fp32, rounded once to nearest even
 * An expert's weight is read once for all its tokens. h is kept to 16
 * significant bits (two bf16 parts) between the products.
 * The order of every sum is fixed by ids: equal inputs give equal bits.
 * Requirements: 0 <= T <= 64, H % 32 == 0, I % 32 == 0, group_size -1 or a
 * positive multiple of 32 dividing H and I, 1 <= top_k <= 16, 1 <= E <= 1024;
 * x, planes, zeros, scales, y and workspace 16-byte aligned; one expert's plane
 * smaller than 4 GiB. Flags: QMM_BF16, QMM_STRIPS. An id outside [0, E) adds
 * nothing to its token; an expert must not come twice for one token.
 */
size_t qmm_moe_workspace_bytes(int T, int H, int I, int E, int top_k);
qmm_status qmm_moe(const uint16_t* x, int T, int H, int I, int E, int top_k, const int32_t* ids, const float* weights,
                   const qmm_experts* gate_up, const qmm_experts* down, int bits, int group_size, unsigned flags,
                   uint16_t* y, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Paged cache: keys and values of Hkv heads in pages of page_size tokens,
 * k_cache and v_cache (pages, Hkv, page_size, D): a head's tokens of one page
 * lie one behind another. Slot s is token s % page_size of page s / page_size.
 * pages * Hkv * page_size < 2^31.
 *
 * qmm_kv_append -- rotates the queries and the keys of T new tokens and puts
 * keys and values into the cache:
 *   q_out[t] = rot(q[t]);  k_cache[slots[t]] = rot(k[t]);  v_cache[slots[t]] = v[t]
 * rot turns the first R of a head's D values by the angles of row positions[t]
 * of cos and sin: the pair (a, b) becomes (a c - b s, b c + a s). In fp32,
 * rounded once.
 *   q (T, Hq, D), k, v (T, Hkv, D): heads dense, q_stride, k_stride, v_stride
 *           elements from token to token (views of one product's rows)
 *   cos, sin (P, R / 2) fp32;  positions (T,) int32;  slots (T,) int64
 *   q_out   (T, Hq, D) dense
 * Requirements: D 64, 128 or 256; 0 <= R <= D, R % 16 == 0 (R 0: no rotation,
 * cos, sin and positions unused); strides multiples of 8, at least a token's
 * size; T * Hq * D < 2^31; q, k, v, q_out and caches 16-byte aligned, cos, sin
 * 16-byte, positions 4-byte, slots 8-byte. Flags: QMM_BF16, QMM_ADJACENT.
 * A token whose slot is outside the cache (a negative one, say) is not stored;
 * its query is still rotated. Positions are cut to [0, P). No two tokens of a
 * call may have the same slot.
 */
qmm_status qmm_kv_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                         int64_t v_stride, int T, int Hq, int Hkv, int D, const float* cos, const float* sin, int R,
                         int P, const int32_t* positions, const int64_t* slots, uint16_t* q_out, uint16_t* k_cache,
                         uint16_t* v_cache, int pages, int page_size, unsigned flags, hipStream_t stream);

/*
 * qmm_attention -- attention of new tokens to their sequences' cached keys.
 * Sequence b has the query rows [q_starts[b], q_starts[b + 1]) and kv_lens[b]
 * cached tokens, the new ones the last of them: its query i is at position
 * p = kv_lens[b] - (number of its queries) + i. A query sees the keys j with
 * max(0, first[t]) <= j < min(end[t], kv_lens[b]); without `first` from 0,
 * without `end` up to and with its own position (causal).
 *   s_j = scale * q . k_j;  softcap > 0: s_j = softcap * tanh(s_j / softcap);
 *   s_j -= slopes[h] * |p - j|  (with slopes)
 *   out = sum_j exp(s_j) v_j / sum_j exp(s_j);  0 where a query sees no key
 * Keys that a query does not see have no part in its result, whatever they
 * hold. `first` and `end` make sliding windows (first = p + 1 - window),
 * documents (first = the document's start) and two-way prefixes (end =
 * max(p + 1, prefix length)).
 *   q (T, Hq, D), heads dense, q_stride elements from token to token; out (T, Hq, D) dense
 *   k_cache, v_cache as above; page_table (B, table_stride) int32: page of tokens
 *           [i page_size, (i + 1) page_size) of sequence b at [b, i]
 *   kv_lens (B,), q_starts (B + 1,), first, end (T,) int32; slopes (Hq,) fp32
 *   max_q, max_kv: bounds of the sequences' queries and keys. Of a sequence with more, the further
 *           queries are left out and the further keys not seen; positions go by all of them
 * A token that is left out, or of no sequence (before the first, behind the last: q_starts must
 * not fall), gets 0. With B or max_q 0 nothing is written.
 * Query head h reads key head h / (Hq / Hkv). Scores, softmax and sums are fp32
 * (with a softcap of up to 64 a score may be off by softcap * 2^-22, with a larger
 * one by a few roundings of its own size);
 * the weights exp(s) are rounded to the data type for the product with v, and
 * the same rounded weights make the denominator.
 * Requirements: D 64, 128 or 256; Hq % Hkv == 0; page_size >= 1; q_stride % 8
 * == 0 and >= Hq * D; scale and softcap finite, softcap >= 0; q, out, caches
 * and workspace 16-byte aligned, the int32 and fp32 arrays 4-byte;
 * max_kv <= table_stride * page_size < 2^31, T * Hq and max_q * Hq < 2^31, B <=
 * 65535, pages * Hkv * page_size < 2^31, and B * Hkv * (max_q * Hq / Hkv / 16 + 1)
 * below 2^24 (with more than 64 query rows per key head an eighth of it). Flags: QMM_BF16.
 * Page ids are cut to [0, pages). Equal inputs give equal bits.
 */
size_t qmm_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv);
qmm_status qmm_attention(const uint16_t* q, int64_t q_stride, int T, int Hq, int Hkv, int D, const uint16_t* k_cache,
                         const uint16_t* v_cache, int pages, int page_size, const int32_t* page_table, int table_stride,
                         const int32_t* kv_lens, const int32_t* q_starts, int B, int max_q, int max_kv,
                         const int32_t* first, const int32_t* end, float scale, float softcap, const float* slopes,
                         unsigned flags, uint16_t* out, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * qmm_logprobs -- log probabilities of given tokens under rows of logits:
 *   lse = log(sum_v exp(l_v));  logprob[m] = l[m, targets[m]] - lse
 *   entropy[m] = -sum_v p_v log(p_v),  p_v = exp(l_v - lse)   (a p of 0 adds 0)
 *   top_ids[m, :], top_logprobs[m, :]: the `top` largest logits, largest first
 *           (equal ones: the lower index first), and l - lse of each
 *   logits  (M, V), row_stride elements from row to row: fp16, bf16 (QMM_BF16) or fp32 (QMM_FP32)
 *   targets (M,) int64, or NULL with logprob NULL; the results fp32, top_ids int32
 * A negative target marks a row without one: its logprob is 0. One of V or more
 * gives NaN. Logits of -inf are tokens of probability 0; a row of nothing else,
 * or with a NaN or +inf, gives NaN for logprob (where it has a target), entropy
 * and top_logprobs; in top_ids a NaN counts as larger than all.
 * Requirements: M >= 0, V >= 1, row_stride >= V, 0 <= top <= min(32, V); logits
 * aligned to their type, targets 8-byte, the rest 4-byte, workspace 16-byte.
 * Flags: QMM_BF16 or QMM_FP32.
 */
size_t qmm_logprobs_workspace_bytes(int M, int V, int top);
qmm_status qmm_logprobs(const void* logits, int64_t row_stride, int M, int V, const int64_t* targets, int top,
                        unsigned flags, float* logprob, float* entropy, float* top_logprobs, int32_t* top_ids,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_LAYER_H */
