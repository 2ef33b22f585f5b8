/*
 * libq4dec, serving operators: the position rotation with the append to a
 * paged key/value cache, the attention that reads that cache, and the
 * sampling of a token from a row of logits. They sit between the projections
 * and heads of q4dec.h in a decoder's step: q4_gemv / q4_gemv_multi /
 * q4_gemm_s64 (QKV) -> kv_append_rope -> paged_attention -> q4_gemv (O) ...
 * q4_gemv (head logits) -> sample_logits.
 *
 * The attention family is the one the model cards describe ("Gemma 4 E2B
 * (text decoder) - Core AI" and "Gemma 4 E4B", signature features: head
 * widths 256 and 512, a 512-token sliding window, QK-norm, scale-free V norm,
 * attention scale 1.0, two rotation bases, shared key/value heads). The cards
 * keep a contiguous cache per layer; the pages here are this library's own.
 *
 * The conventions of q4dec.h hold for every call: device memory owned by the
 * caller, no allocation, no copy and no synchronisation, validation on the
 * host before anything is enqueued, a negative status with
 * q4dec_last_error(), work enqueued on `stream` of the current device.
 * Values that only the device knows (slots, page numbers, lengths) are
 * checked by the kernels: a bad one is skipped, nothing outside the given
 * buffers is read or written, and the optional device int32 `err_flag` is
 * set to 1 (never cleared).
 *
 * Paged cache: keys and values each are [n_pages, n_kv, page_size, head_dim],
 * contiguous, 16-byte aligned; page_size is a power of two in [16, 4096].
 * Slot s of the cache is row s % page_size of page s / page_size. Elements
 * are bf16, or e4m3 (OCP fp8: 4 exponent bits, bias 7, largest 448, no
 * infinity) with one fp32 scale per key/value head: value = element * scale.
 */
#ifndef Q4DEC_SERVE_H
#define Q4DEC_SERVE_H

#include "q4dec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of a cache. */
#define Q4DEC_KV_BF16 0
#define Q4DEC_KV_E4M3 1

/* kv_append_rope: one layer's new query, key and value rows, from the fp32
 * projections to what the attention reads. For token t and each head, in
 * fp32:
 *   x <- x * (mean(x^2) + eps)^(-1/2) * norm   (q with q_norm, k with k_norm,
 *        v without a weight; each only if asked for)
 *   q, k: for j < n_freqs the pair (x[j], x[j + rot_dim / 2]) is turned by
 *        the angle positions[t] * freqs[j]; all other elements stay
 * and then q is rounded to bf16 into q_out, k and v are rounded to nearest
 * even into the cache at slots[t] (e4m3: x / scale, clamped to +-448; NaN
 * stays NaN). The angle is formed and reduced in fp64, so far positions lose
 * nothing; sin and cos are fp32.
 *   q, k, v   fp32 [n_tok, n_q or n_kv heads, head_dim]; a token's row starts
 *             every q_stride / k_stride / v_stride elements (a multiple of 4;
 *             the three may be parts of one fused row). n_q = 0 (q NULL)
 *             only appends; n_kv = 0 (k, v, caches and slots NULL) only
 *             rotates q, as layers that share another layer's cache need.
 *   head_dim  64, 128, 256 or 512; n_q and n_kv at most 4096.
 *   rot_dim   even, in [2, head_dim]; n_freqs in [0, rot_dim / 2].
 *   q_norm, k_norm  fp32 [head_dim] or NULL (no norm); v_norm 0 or 1.
 *   freqs     fp64 [n_freqs], radians per position (NULL if n_freqs is 0).
 *   positions int32 [n_tok]; any value.
 *   slots     int32 [n_tok]; a negative slot marks a padded token whose key
 *             and value are not stored, a slot beyond the cache is not stored
 *             either and sets err_flag. Two tokens of one call must not share
 *             a slot: which of them each element of it then holds is not
 *             defined.
 *   k_scale, v_scale  fp32 [n_kv], for e4m3 only (NULL: 1.0).
 *   q_out     bf16 [n_tok, n_q, head_dim].
 * q, k, v, norms, caches and q_out 16-byte aligned; freqs 8, the rest 4.
 * q_out must not overlap the inputs. n_tok = 0 does nothing; n_tok < 2^24.
 * Errors: NULL pointer, a size out of range, misalignment; UNSUPPORTED for
 *         another head_dim. */
int kv_append_rope(const float* q, int64_t q_stride, const float* k,
                   int64_t k_stride, const float* v, int64_t v_stride,
                   int64_t n_tok, int64_t n_q, int64_t n_kv, int64_t head_dim,
                   const float* q_norm, const float* k_norm, int32_t v_norm,
                   float eps, const double* freqs, int64_t n_freqs,
                   int64_t rot_dim, const int32_t* positions,
                   const int32_t* slots, int32_t kv_type, const float* k_scale,
                   const float* v_scale, void* k_cache, void* v_cache,
                   int64_t n_pages, int64_t page_size, uint16_t* q_out,
                   int32_t* err_flag, void* stream);

/* Workspace bytes paged_attention needs for these bounds (0 for invalid
 * ones). It depends on the current device's number of compute units. */
size_t paged_attention_workspace_bytes(int64_t n_seq, int64_t n_q,
                                       int64_t n_kv, int64_t head_dim,
                                       int64_t max_q_len, int64_t max_kv_len,
                                       int64_t window);

/* paged_attention: causal attention of the new tokens of n_seq sequences
 * over their cached keys and values. Sequence b has the query rows
 * q_starts[b] .. q_starts[b + 1] - 1 and kv_lens[b] cached tokens, its new
 * ones included: its i-th query row stands at position
 *   p = kv_lens[b] - q_len + i
 * and sees the positions j <= p, with window > 0 only those with
 * j > p - window. Position j lies in row j % page_size of page
 * page_table[b * table_stride + j / page_size]. Query head h reads key/value
 * head h / (n_q / n_kv). For each row and head
 *   out = sum_j softmax_j(scale * q . k_j) v_j,
 * zero for a row that sees nothing (p < 0). One token per sequence is the
 * decode step, a few the check of drafted tokens, many a prefill chunk.
 * Scores, softmax statistics and output sums are fp32; for the matrix cores
 * the probabilities are rounded to bf16 (where max_q_len * n_q / n_kv <= 32
 * to two bf16 parts, about 16 bits), the output once to bf16.
 *   q, out     bf16 [n_tok, n_q, head_dim], 16-byte aligned, no overlap. Rows
 *              before q_starts[0] and from q_starts[n_seq] on are left as
 *              they are.
 *   head_dim   64, 128, 256 or 512; n_q a multiple of n_kv, at most 4096, at
 *              most 64 query heads per key/value head.
 *   k_cache, v_cache  as written by kv_append_rope; only pages that hold a
 *              position some row sees are read, so entries of the table for
 *              others may hold anything. A page number outside
 *              [0, n_pages) sets err_flag and its positions are not seen.
 *   k_scale, v_scale  fp32 [n_kv], for e4m3 only (NULL: 1.0).
 *   page_table int32 [n_seq, table_stride].
 *   q_starts   int32 [n_seq + 1], not decreasing, within [0, n_tok];
 *   kv_lens    int32 [n_seq], within [0, max_kv_len]. A sequence with other
 *              values, or with more than max_q_len rows, sets err_flag and
 *              its rows are left as they are.
 *   max_q_len, max_kv_len  bounds on the lengths (the launch is sized by
 *              them: tight ones are faster); max_kv_len <= table_stride *
 *              page_size and 2^30, max_q_len * n_q < 2^30.
 *   window     0: none; scale: any finite number.
 *   ws         device workspace, ws_bytes >= paged_attention_workspace_bytes
 *              of the same bounds, 256-byte aligned, caller-owned, no initial
 *              contents needed (NULL if 0 bytes are needed). Calls that share
 *              one ws must not overlap in time.
 * Deterministic: the same call gives the same bits. Where a sequence's keys
 * are cut into partial sums goes by the bounds and by the lengths of the whole
 * batch, so its last bits may differ in other company. A key or value that a
 * row does not see does not touch it. A NaN or infinity in a key that it sees
 * makes it what the formula makes it. In a value that it sees a NaN makes its
 * column of the row NaN, an infinity that infinity however small its
 * probability, and infinities of both signs NaN.
 * Errors: NULL pointer, a size out of range, workspace too small,
 *         misalignment; UNSUPPORTED for another head_dim, more query heads per
 *         key/value head, or bounds that allow 2^31 or more pieces of work
 *         (n_seq * n_kv * rows / 16 or 128 * keys / 64 or 32). */
int paged_attention(const uint16_t* q, int64_t n_tok, int64_t n_q,
                    int64_t n_kv, int64_t head_dim, const void* k_cache,
                    const void* v_cache, int32_t kv_type, int64_t n_pages,
                    int64_t page_size, const float* k_scale,
                    const float* v_scale, const int32_t* page_table,
                    int64_t table_stride, const int32_t* q_starts,
                    const int32_t* kv_lens, int64_t n_seq, int64_t max_q_len,
                    int64_t max_kv_len, float scale, int64_t window, void* ws,
                    size_t ws_bytes, uint16_t* out, int32_t* err_flag,
                    void* stream);

/* Workspace bytes sample_logits needs (0 for invalid shapes). */
size_t sample_logits_workspace_bytes(int64_t n_rows, int64_t vocab);

/* sample_logits: one token per row of logits, beside the heads' greedy
 * argmax. For row r, with its own temperature T, top_k, top_p, min_p and a
 * number u in [0, 1):
 *   l_i = cap * tanh(z_i / cap) / T      (no cap: z_i / T)
 *   w_i = exp(l_i - max_i l_i)
 * The tokens are ranked by z, the lower index first among equals. Of them
 * stay, in this order: the first top_k; of those the ones whose better-ranked
 * weights sum to less than top_p of the whole; of those the ones with
 * w_i >= min_p. The first-ranked token always stays. The token drawn is the
 * lowest index i with sum of the w_j that stay, j <= i, > u * their whole sum;
 * its share of that sum is prob_out. Logits that are NaN or -infinity are
 * never drawn; if a row has no other, idx_out = -1 and prob_out = NaN. T <= 0
 * (or NaN) is greedy: the first-ranked token, probability 1.
 * Weights are formed in fp64 and summed as 42-bit fixed-point fractions of
 * the largest one, so sums do not depend on their order and the result is
 * deterministic; a token lighter than 2^-43 of the heaviest is never drawn.
 * Tokens that must not be drawn are best masked by -infinity: under a small
 * top_k finite masks cost a row milliseconds.
 *   logits   fp32 [n_rows, vocab], row r at r * row_stride elements
 *            (q4_gemv, q4_gemv_multi and q4_gemm_s64 write such rows);
 *            4-byte aligned.
 *   cap      30.0 for Gemma 4; none if <= 0, NaN or infinite.
 *   temperature, top_k (int32), top_p, min_p  [n_rows] or NULL (1.0, off,
 *            off, off). top_k <= 0 or >= vocab, top_p >= 1 (or NaN) and
 *            min_p <= 0 (or NaN) switch a filter off.
 *   u        fp32 [n_rows]; values outside [0, 1) are clamped into it, NaN
 *            counts as 0.
 *   ws       device workspace, ws_bytes >= sample_logits_workspace_bytes,
 *            256-byte aligned, caller-owned, no initial contents needed;
 *            calls that share one ws must not overlap in time.
 *   idx_out  int32 [n_rows]; prob_out fp32 [n_rows] (NULL allowed).
 * n_rows = 0 does nothing.
 * Errors: NULL pointer, vocab not in [1, 2^20], n_rows not in [0, 65535],
 *         row_stride < vocab, workspace too small, misalignment. */
int sample_logits(const float* logits, int64_t n_rows, int64_t vocab,
                  int64_t row_stride, float cap, const float* temperature,
                  const int32_t* top_k, const float* top_p, const float* min_p,
                  const float* u, void* ws, size_t ws_bytes, int32_t* idx_out,
                  float* prob_out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* Q4DEC_SERVE_H */
