// paged_attention: softmax(scale q k^T) v of the new tokens of several
// sequences over their paged keys and values (causal, optional window,
// grouped heads). The simple form: one workgroup per query row and head, its
// waves taking the keys in turn with a running maximum and sum each.
#include <math.h>

#include "q4dec_internal.h"
#include "q4dec_serve.h"
#include "serve_internal.h"

namespace q4dec {
Q4DEC_DEBUG_READER(paged_attention)

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;

struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* q_starts;
  const int32_t* kv_lens;
  int32_t* err;
  int64_t table_stride;
  int n_tok, n_q, n_kv, group, n_pages, page_shift;
  int max_q, max_kv;
  int64_t window;
  float scale;
};

// Bounds of sequence b; false if they are not valid.
__device__ __forceinline__ bool sequence_of(const AttnArgs& a, int b, int& start, int& q_len, int& kv_len) {
  start = a.q_starts[b];
  q_len = a.q_starts[b + 1] - start;
  kv_len = a.kv_lens[b];
  const bool ok = start >= 0 && q_len >= 0 && start <= a.n_tok && q_len <= a.n_tok - start && q_len <= a.max_q &&
                  kv_len >= 0 && kv_len <= a.max_kv;
  return ok;
}

template <int E, bool E4M3>
__device__ __forceinline__ void load_elements(const uint8_t* base, size_t off, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if constexpr (E4M3)
      x[i] = __builtin_amdgcn_cvt_f32_fp8(int(base[off + i]), 0);
    else
      x[i] = bf16_to_f32(reinterpret_cast<const uint16_t*>(base)[off + i]);
  }
}

template <int D, bool E4M3>
__global__ __launch_bounds__(kAttnThreads) void attn_row_kernel(AttnArgs a) {
  constexpr int E = D / 64;
  __shared__ float part[kAttnWaves][D + 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = blockIdx.x, hq = blockIdx.y, b = blockIdx.z;
  int start, q_len, kv_len;
  if (!sequence_of(a, b, start, q_len, kv_len)) {
    if (a.err && threadIdx.x == 0) *a.err = 1;
    return;
  }
  if (i >= q_len) return;
  const int h = hq / a.group;
  const size_t row = (size_t(start + i) * a.n_q + hq) * D + lane * E;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_to_f32(a.q[row + e]);
    o[e] = 0.0f;
  }
  const float ks = a.scale * (a.k_scale ? a.k_scale[h] : 1.0f);
  const int64_t p = int64_t(kv_len) - q_len + i;
  const int64_t first = a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = first + wave; j <= p; j += kAttnWaves) {
    const int page = a.page_table[b * a.table_stride + (j >> a.page_shift)];
    if (page < 0 || page >= a.n_pages) {
      if (a.err && lane == 0) *a.err = 1;
      continue;
    }
    const size_t off = ((size_t(page) * a.n_kv + h) << a.page_shift) * D +
                       size_t(j & ((int64_t(1) << a.page_shift) - 1)) * D + lane * E;
    float k[E], v[E];
    load_elements<E, E4M3>(a.k_cache, off, k);
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    s = group_sum<64>(s) * ks;
    load_elements<E, E4M3>(a.v_cache, off, v);
    const float mn = s > m ? s : m;  // a NaN score leaves the maximum and makes the sum NaN
    const float keep = m == -INFINITY ? 0.0f : expf(m - mn), w = s == -INFINITY ? 0.0f : expf(s - mn);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * v[e];
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[wave][lane * E + e] = o[e];
  if (lane == 0) {
    part[wave][D] = m;
    part[wave][D + 1] = l;
  }
  __syncthreads();
  if (wave != 0) return;
  float mx = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kAttnWaves; ++w) mx = fmaxf(mx, part[w][D]);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int w = 0; w < kAttnWaves; ++w) {
    const float mw = part[w][D];
    const float f = mw == -INFINITY ? (part[w][D + 1] == 0.0f ? 0.0f : 1.0f) : expf(mw - mx);
    sum += part[w][D + 1] * f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += part[w][lane * E + e] * f;
  }
  const float vs = a.v_scale ? a.v_scale[h] : 1.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[row + e] = f32_to_bf16_rne(sum == 0.0f ? 0.0f : o[e] / sum * vs);
}

}  // namespace q4dec

extern "C" size_t paged_attention_workspace_bytes(int64_t n_seq, int64_t n_q, int64_t n_kv, int64_t head_dim,
                                                  int64_t max_q_len, int64_t max_kv_len, int64_t window) {
  return 0;
}

extern "C" int paged_attention(const uint16_t* q, int64_t n_tok, int64_t n_q, int64_t n_kv, int64_t head_dim,
                               const void* k_cache, const void* v_cache, int32_t kv_type, int64_t n_pages,
                               int64_t page_size, const float* k_scale, const float* v_scale,
                               const int32_t* page_table, int64_t table_stride, const int32_t* q_starts,
                               const int32_t* kv_lens, int64_t n_seq, int64_t max_q_len, int64_t max_kv_len,
                               float scale, int64_t window, void* ws, size_t ws_bytes, uint16_t* out,
                               int32_t* err_flag, void* stream) {
  using namespace q4dec;
  const char* name = "paged_attention";
  if (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 512)
    return fail(Q4DEC_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128, 256 or 512 (got %lld)", name,
                (long long)head_dim);
  if (n_kv <= 0 || n_q <= 0 || n_q > 65535 || n_q % n_kv)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_q must be a positive multiple of n_kv, at most 65535 (got %lld, %lld)", name,
                (long long)n_q, (long long)n_kv);
  if (n_q / n_kv > kMaxGroup)
    return fail(Q4DEC_ERR_UNSUPPORTED, "%s: more than %d query heads per key/value head (n_q %lld, n_kv %lld)", name,
                int(kMaxGroup), (long long)n_q, (long long)n_kv);
  if (n_tok < 0 || n_tok >= (int64_t(1) << 31) / n_q)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_tok must be in [0, 2^31 / n_q) (got %lld)", name, (long long)n_tok);
  if (n_seq < 0 || n_seq > 65535)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_seq must be in [0, 65535] (got %lld)", name, (long long)n_seq);
  if (n_seq == 0 || n_tok == 0) return Q4DEC_OK;
  if (max_q_len <= 0 || max_q_len >= (int64_t(1) << 31))
    return fail(Q4DEC_ERR_SHAPE, "%s: max_q_len must be in [1, 2^31) (got %lld)", name, (long long)max_q_len);
  if (window < 0) return fail(Q4DEC_ERR_SHAPE, "%s: window must not be negative (got %lld)", name, (long long)window);
  if (!isfinite(scale)) return fail(Q4DEC_ERR_SHAPE, "%s: scale must be finite", name);
  if (!q) return fail(Q4DEC_ERR_NULL, "%s: q is NULL", name);
  if (!out) return fail(Q4DEC_ERR_NULL, "%s: out is NULL", name);
  if (!page_table) return fail(Q4DEC_ERR_NULL, "%s: page_table is NULL", name);
  if (!q_starts) return fail(Q4DEC_ERR_NULL, "%s: q_starts is NULL", name);
  if (!kv_lens) return fail(Q4DEC_ERR_NULL, "%s: kv_lens is NULL", name);
  int page_shift = 0;
  const int rc = check_cache(name, k_cache, v_cache, kv_type, n_pages, page_size, k_scale, v_scale, &page_shift);
  if (rc != Q4DEC_OK) return rc;
  if (table_stride <= 0 || table_stride >= (int64_t(1) << 31))
    return fail(Q4DEC_ERR_SHAPE, "%s: table_stride must be in [1, 2^31) (got %lld)", name, (long long)table_stride);
  if (max_kv_len < 0 || max_kv_len >= (int64_t(1) << 31) || (max_kv_len + page_size - 1) / page_size > table_stride)
    return fail(Q4DEC_ERR_SHAPE, "%s: max_kv_len must be in [0, table_stride * page_size] (got %lld)", name,
                (long long)max_kv_len);
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(Q4DEC_ERR_ALIGN, "%s: q and out must be 16-byte aligned", name);
  if (!aligned(page_table, 4) || !aligned(q_starts, 4) || !aligned(kv_lens, 4))
    return fail(Q4DEC_ERR_ALIGN, "%s: page_table, q_starts and kv_lens must be 4-byte aligned", name);
  const size_t need = paged_attention_workspace_bytes(n_seq, n_q, n_kv, head_dim, max_q_len, max_kv_len, window);
  if (need > 0 && !ws) return fail(Q4DEC_ERR_NULL, "%s: ws is NULL", name);
  if (ws_bytes < need)
    return fail(Q4DEC_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws_bytes, need);
  if (!aligned(ws, 256)) return fail(Q4DEC_ERR_ALIGN, "%s: ws must be 256-byte aligned", name);
  AttnArgs a;
  a.q = q, a.out = out;
  a.k_cache = static_cast<const uint8_t*>(k_cache), a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale, a.v_scale = v_scale;
  a.page_table = page_table, a.q_starts = q_starts, a.kv_lens = kv_lens, a.err = err_flag;
  a.table_stride = table_stride;
  a.n_tok = int(n_tok), a.n_q = int(n_q), a.n_kv = int(n_kv), a.group = int(n_q / n_kv);
  a.n_pages = int(n_pages), a.page_shift = page_shift;
  a.max_q = int(max_q_len < n_tok ? max_q_len : n_tok), a.max_kv = int(max_kv_len);
  a.window = window, a.scale = scale;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 grid(unsigned(a.max_q), unsigned(n_q), unsigned(n_seq));
  const bool f8 = kv_type == Q4DEC_KV_E4M3;
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kAttnThreads), 0, st, a); };
  switch (int(head_dim)) {
    case 64: f8 ? go(attn_row_kernel<64, true>) : go(attn_row_kernel<64, false>); break;
    case 128: f8 ? go(attn_row_kernel<128, true>) : go(attn_row_kernel<128, false>); break;
    case 256: f8 ? go(attn_row_kernel<256, true>) : go(attn_row_kernel<256, false>); break;
    default: f8 ? go(attn_row_kernel<512, true>) : go(attn_row_kernel<512, false>); break;
  }
  return launch_status(name);
}
