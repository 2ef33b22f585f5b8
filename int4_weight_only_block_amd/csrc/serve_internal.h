// What the serving operators share: their debug bits and the host checks of
// a paged key/value cache and of an attention call.
#pragma once

#include <math.h>

#include "q4dec_internal.h"
#include "q4dec_serve.h"

namespace q4dec {

// their bits among q4dec_internal.h's, and their units' readers
enum ServeDebugBit : int {
  kDbgAppendGrid = 19,  // kv_append_kernel: grid does not cover the heads
  kDbgAttnGrid = 20,    // attention kernels: more workgroups or rows than the workspace holds
  kDbgSampleGrid = 21,  // sample kernels: groups do not cover the vocabulary, or a step outside the histogram
  kDbgVerifyGrid = 22,  // verify kernels: groups do not cover the vocabulary
};
uint32_t debug_take_kv_append();
uint32_t debug_take_paged_attention();
uint32_t debug_take_sample_logits();
uint32_t debug_take_paged_attention_shared();
uint32_t debug_take_verify_drafts();

constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxGroup = 64;  // query heads per key/value head
constexpr int64_t kMinPage = 16, kMaxPage = 4096;

// The cache arguments of `name`; *page_shift = log2(page_size).
inline int check_cache(const char* name, const void* k_cache, const void* v_cache, int32_t kv_type, int64_t n_pages,
                       int64_t page_size, const float* k_scale, const float* v_scale, int* page_shift) {
  if (!k_cache) return fail(Q4DEC_ERR_NULL, "%s: k_cache is NULL", name);
  if (!v_cache) return fail(Q4DEC_ERR_NULL, "%s: v_cache is NULL", name);
  if (kv_type != Q4DEC_KV_BF16 && kv_type != Q4DEC_KV_E4M3)
    return fail(Q4DEC_ERR_SHAPE, "%s: kv_type must be Q4DEC_KV_BF16 or Q4DEC_KV_E4M3 (got %d)", name, int(kv_type));
  if (page_size < kMinPage || page_size > kMaxPage || (page_size & (page_size - 1)))
    return fail(Q4DEC_ERR_SHAPE, "%s: page_size must be a power of two in [16, 4096] (got %lld)", name,
                (long long)page_size);
  if (n_pages <= 0 || n_pages > ((int64_t(1) << 31) - 1) / page_size)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_pages must be positive, n_pages * page_size below 2^31 (got %lld)", name,
                (long long)n_pages);
  if (kv_type == Q4DEC_KV_BF16 && (k_scale || v_scale))
    return fail(Q4DEC_ERR_SHAPE, "%s: k_scale and v_scale belong to an e4m3 cache", name);
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16))
    return fail(Q4DEC_ERR_ALIGN, "%s: k_cache and v_cache must be 16-byte aligned", name);
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4))
    return fail(Q4DEC_ERR_ALIGN, "%s: k_scale and v_scale must be 4-byte aligned", name);
  int s = 0;
  while ((int64_t(1) << s) < page_size) ++s;
  *page_shift = s;
  return Q4DEC_OK;
}

// The arguments of attention call `name`; those of a call without sequences or
// tokens, which does nothing, only as far as that is known.
inline int check_attention(const char* name, const uint16_t* q, int64_t n_tok, int64_t n_q, int64_t n_kv, int64_t head_dim,
                           const void* k_cache, const void* v_cache, int32_t kv_type, int64_t n_pages, int64_t page_size,
                           const float* k_scale, const float* v_scale, const int32_t* page_table, int64_t table_stride,
                           const int32_t* q_starts, const int32_t* kv_lens, int64_t n_seq, int64_t max_q_len,
                           int64_t max_kv_len, float scale, const uint16_t* out, int* page_shift) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 512)
    return fail(Q4DEC_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128, 256 or 512 (got %lld)", name,
                (long long)head_dim);
  if (n_kv <= 0 || n_q <= 0 || n_q > kMaxHeads || n_q % n_kv)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_q must be a positive multiple of n_kv, at most 4096 (got %lld, %lld)", name,
                (long long)n_q, (long long)n_kv);
  if (n_q / n_kv > kMaxGroup)
    return fail(Q4DEC_ERR_UNSUPPORTED, "%s: more than %d query heads per key/value head (n_q %lld, n_kv %lld)", name,
                int(kMaxGroup), (long long)n_q, (long long)n_kv);
  if (n_tok < 0 || n_tok >= (int64_t(1) << 31) / n_q)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_tok must be in [0, 2^31 / n_q) (got %lld)", name, (long long)n_tok);
  if (n_seq < 0 || n_seq > 65535)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_seq must be in [0, 65535] (got %lld)", name, (long long)n_seq);
  if (n_seq == 0 || n_tok == 0) return Q4DEC_OK;
  if (max_q_len <= 0 || max_q_len >= (int64_t(1) << 30) / n_q)
    return fail(Q4DEC_ERR_SHAPE, "%s: max_q_len must be in [1, 2^30 / n_q) (got %lld)", name, (long long)max_q_len);
  if (!isfinite(scale)) return fail(Q4DEC_ERR_SHAPE, "%s: scale must be finite", name);
  if (!q) return fail(Q4DEC_ERR_NULL, "%s: q is NULL", name);
  if (!out) return fail(Q4DEC_ERR_NULL, "%s: out is NULL", name);
  if (!page_table) return fail(Q4DEC_ERR_NULL, "%s: page_table is NULL", name);
  if (!q_starts) return fail(Q4DEC_ERR_NULL, "%s: q_starts is NULL", name);
  if (!kv_lens) return fail(Q4DEC_ERR_NULL, "%s: kv_lens is NULL", name);
  const int rc = check_cache(name, k_cache, v_cache, kv_type, n_pages, page_size, k_scale, v_scale, page_shift);
  if (rc != Q4DEC_OK) return rc;
  if (table_stride <= 0 || table_stride >= (int64_t(1) << 31))
    return fail(Q4DEC_ERR_SHAPE, "%s: table_stride must be in [1, 2^31) (got %lld)", name, (long long)table_stride);
  if (max_kv_len < 0 || max_kv_len > (int64_t(1) << 30) || (max_kv_len + page_size - 1) / page_size > table_stride)
    return fail(Q4DEC_ERR_SHAPE, "%s: max_kv_len must be in [0, table_stride * page_size], at most 2^30 (got %lld)", name,
                (long long)max_kv_len);
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(Q4DEC_ERR_ALIGN, "%s: q and out must be 16-byte aligned", name);
  if (!aligned(page_table, 4) || !aligned(q_starts, 4) || !aligned(kv_lens, 4))
    return fail(Q4DEC_ERR_ALIGN, "%s: page_table, q_starts and kv_lens must be 4-byte aligned", name);
  return Q4DEC_OK;
}

}  // namespace q4dec
