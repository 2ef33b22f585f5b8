// What the serving operators share: their debug bits and the host checks of
// a paged key/value cache.
#pragma once

#include "q4dec_internal.h"
#include "q4dec_serve.h"

namespace q4dec {

// their bits among q4dec_internal.h's, and their units' readers
enum ServeDebugBit : int {
  kDbgAppendGrid = 19,  // kv_append_kernel: grid does not cover the heads
  kDbgAttnGrid = 20,    // attention kernels: more workgroups or rows than the workspace holds
  kDbgSampleGrid = 21,  // sample kernels: groups do not cover the vocabulary, or a step outside the histogram
};
uint32_t debug_take_kv_append();
uint32_t debug_take_paged_attention();
uint32_t debug_take_sample_logits();

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

}  // namespace q4dec
