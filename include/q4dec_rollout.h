/*
 * libq4dec, operators of rollouts: several continuations of one text, and
 * speculative steps. They stand beside the serving operators of
 * q4dec_serve.h: paged_attention_shared in the place of paged_attention where
 * sequences begin alike, verify_drafts in the place of sample_logits where a
 * step has checked drafted tokens:
 * kv_append_rope -> paged_attention_shared -> ... q4_gemv_multi /
 * q4_gemm_s64 (head logits of every row) -> verify_drafts.
 *
 * The verify pass over drafted tokens is the one of the mixed-bit page
 * ("Gemma-4 E2B mobile mixed-bit QAT weights", its MTP sections P5c and P5d:
 * a few draft rows against weights read once), which keeps greedy matches. To
 * keep drafts by their probabilities is the published rejection rule of
 * speculative sampling; the page has neither it nor pages that sequences share.
 *
 * The conventions of q4dec.h and q4dec_serve.h hold: device memory owned by
 * the caller, no allocation, no copy and no synchronisation, validation on the
 * host before anything is enqueued, a negative status with q4dec_last_error(),
 * work enqueued on `stream` of the current device. Values that only the device
 * knows are checked by the kernels: nothing outside the given buffers is read
 * or written, and a bad one sets the optional device int32 `err_flag` to 1
 * (never cleared).
 */
#ifndef Q4DEC_ROLLOUT_H
#define Q4DEC_ROLLOUT_H

#include "q4dec_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes paged_attention_shared needs (0 for invalid shapes, and
 * where none is needed). */
size_t paged_attention_shared_workspace_bytes(int64_t n_tok, int64_t n_seq,
                                              int64_t n_groups, int64_t n_q,
                                              int64_t n_kv, int64_t head_dim,
                                              int64_t max_q_len,
                                              int64_t max_kv_len,
                                              int64_t max_shared_len);

/* paged_attention_shared: what paged_attention (without a window) computes,
 * for sequences that begin with the same positions. Of a group of sequences
 * the keys and values that all share are read once, by the rows of all of
 * them together. The arguments are paged_attention's, with a table that names
 * every sequence's pages as there, and:
 *   group_starts  int32 [n_groups + 1]: group g is the sequences
 *              group_starts[g] .. group_starts[g + 1] - 1; not decreasing,
 *              within [0, n_seq]. Sequences outside every group, and groups
 *              of one, share nothing.
 *   shared_lens  int32 [n_groups]: the first so many positions are the same
 *              for all sequences of the group: their keys and values are read
 *              from the pages that the table names for the group's first sequence
 *              (also where that one has no rows in the call). Any number, also
 *              one that ends inside a page (each sequence may then hold a copy
 *              of that page), within [0, max_shared_len]. A sequence whose
 *              rows do not all see them (kv_lens - q_len + 1 < shared_lens) is
 *              attended alone.
 *   max_shared_len  bound on shared_lens, at most max_kv_len.
 * A group whose values are out of their ranges shares nothing and sets
 * err_flag (a call that does not share looks at none of them); where
 * group_starts or q_starts decrease anywhere, no group shares. What is not
 * valid of a sequence is treated as by paged_attention; rows that two sequences
 * name (q_starts that decrease) hold what either makes of them.
 * A call shares where its longest sequence has at most 128 rows (max_q_len *
 * n_q / n_kv: decode and drafted tokens) and the bounds say that enough bytes
 * of the cache are read less; elsewhere, as for prefill chunks (also beside
 * decodes), whose products and not whose reads take the time, it is
 * paged_attention.
 * Scores, softmax statistics and sums are fp32; where a call shares, the
 * probabilities are rounded to two bf16 parts (about 16 bits), as
 * paged_attention's of few rows are, elsewhere as there; the output once to
 * bf16.
 * Deterministic, as paged_attention is; NaN and infinities count as there.
 *   ws         device workspace, ws_bytes >= paged_attention_shared_workspace_bytes
 *              of the same sizes and bounds, 256-byte aligned, caller-owned,
 *              no initial contents needed. Calls that share one ws must not
 *              overlap in time.
 * Errors: as paged_attention; n_groups not in [0, 65535], max_shared_len not
 *         in [0, max_kv_len]. */
int paged_attention_shared(const uint16_t* q, int64_t n_tok, int64_t n_q,
                           int64_t n_kv, int64_t head_dim, const void* k_cache,
                           const void* v_cache, int32_t kv_type,
                           int64_t n_pages, int64_t page_size,
                           const float* k_scale, const float* v_scale,
                           const int32_t* page_table, int64_t table_stride,
                           const int32_t* q_starts, const int32_t* kv_lens,
                           int64_t n_seq, const int32_t* group_starts,
                           const int32_t* shared_lens, int64_t n_groups,
                           int64_t max_q_len, int64_t max_kv_len,
                           int64_t max_shared_len, float scale, void* ws,
                           size_t ws_bytes, uint16_t* out, int32_t* err_flag,
                           void* stream);

/* Workspace bytes verify_drafts needs (0 for invalid shapes). */
size_t verify_drafts_workspace_bytes(int64_t n_rows, int64_t n_seq,
                                     int64_t vocab, int32_t has_draft_logits);

/* verify_drafts: which drafted tokens of each sequence stay, and the token
 * after them, such that what comes out is distributed as if each token had
 * been drawn from the target. Sequence b has the rows starts[b] ..
 * starts[b + 1] - 1 of the target's logits, one more than it has drafts (one
 * row: no draft, a plain draw). p_r is the distribution that sample_logits
 * draws from in row r, with the sequence's temperature, top_k, top_p and min_p
 * (the filters, ties, masks and greedy rows as there); q_r the one of the row
 * of draft_logits, under the same settings, or, without draft_logits, all on
 * the draft itself. From the first row on, draft x = drafts[r] stays if
 *   u[r] * q_r(x) < p_r(x).
 * At the first row where it does not, the next token is drawn from
 * max(0, p_r - q_r) (from p_r where that is zero everywhere); where all stay,
 * from the last row's p. The token drawn is the lowest index i with
 * sum_{j <= i} of these > u_draw[b] * their whole sum.
 *   tokens_out int32 [n_rows]: in the sequence's rows the drafts that stay, the
 *              new token, then -1.
 *   prob_out   fp32 [n_rows] (NULL allowed): p_r of each of these tokens, 0
 *              beside a -1.
 *   count_out  int32 [n_seq]: how many tokens there are, one more than drafts
 *              that stay (0 for a sequence without rows).
 * A row without a token that may be drawn gives -1 and probability NaN.
 * In calls with filters weights and their sums are as sample_logits has them
 * (fp64, 42-bit fixed-point fractions in integer sums). In calls without any
 * (top_k, top_p and min_p all NULL) a weight in a sum is off by up to 2^-33 of
 * itself, and the sums are fp64 over groups of a row, then as above; so are the
 * weights in max(0, p - q) of rows that no filter touches, summed in 60-bit
 * fractions. The result is deterministic.
 *   logits     fp32 [n_rows, vocab], row r at r * row_stride elements.
 *   draft_logits fp32, rows of the same numbers at draft_stride elements; the
 *              one in the place of a sequence's last row is not read. NULL:
 *              drafts without probabilities (from a table, or greedy).
 *   cap, draft_cap  softcaps of the two; none if <= 0, NaN or infinite.
 *   drafts     int32 [n_rows]; the one of a sequence's last row is not looked
 *              at. One outside [0, vocab) sets err_flag and does not stay.
 *   starts     int32 [n_seq + 1], not decreasing, within [0, n_rows]. A
 *              sequence with other values sets err_flag; its outputs, and rows
 *              of no sequence, are left as they are; rows that two sequences name
 *              (starts that decrease) hold what either makes of them.
 *   temperature, top_k (int32), top_p, min_p  [n_seq] or NULL.
 *   u          fp32 [n_rows], u_draw fp32 [n_seq], in [0, 1); others are
 *              clamped into it, NaN counts as 0.
 *   ws         device workspace, ws_bytes >= verify_drafts_workspace_bytes,
 *              256-byte aligned, caller-owned, no initial contents needed;
 *              calls that share one ws must not overlap in time.
 * n_rows = 0 or n_seq = 0 does nothing.
 * Errors: NULL pointer, vocab not in [1, 2^20], n_rows not in [0, 32767],
 *         n_seq not in [0, 32767], a stride < vocab, workspace too small,
 *         misalignment. */
int verify_drafts(const float* logits, int64_t n_rows, int64_t vocab,
                  int64_t row_stride, float cap, const float* draft_logits,
                  int64_t draft_stride, float draft_cap, const int32_t* drafts,
                  const int32_t* starts, int64_t n_seq,
                  const float* temperature, const int32_t* top_k,
                  const float* top_p, const float* min_p, const float* u,
                  const float* u_draw, void* ws, size_t ws_bytes,
                  int32_t* tokens_out, float* prob_out, int32_t* count_out,
                  int32_t* err_flag, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* Q4DEC_ROLLOUT_H */
