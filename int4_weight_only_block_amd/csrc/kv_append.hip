// kv_append_rope: per-head RMS norm, rotary positions, query rows to bf16 and
// key/value rows into a paged cache (bf16 or e4m3). The rotation, the norms
// and the head widths are those of the "Gemma 4 E2B (text decoder) - Core AI"
// and "Gemma 4 E4B" cards (signature features: QK-norm, scale-free V norm,
// two rotation bases, head widths 256 and 512).
//
// A head of a token is 16, 32 or 64 lanes of a wave, 4 or 8 elements a lane.
// The mean of squares is a cross-lane sum; the rotation's partner element
// (rot_dim / 2 away) is another lane's for most head widths, so the normed
// head goes through LDS once. The angle is position * frequency in fp64,
// reduced to a fraction of a turn before it is rounded to fp32: at position
// 131072 an fp32 product would be off by 2^-8 of a radian. The 4, 8
// or 16 heads of a workgroup share the angles.
//
// Bound by memory for many tokens: 2048 of 8 + 2 heads of 512 into an e4m3
// cache, 71 MB, take 16.1 us (4.4 TB/s; a large copy moves 5.1). One token
// (3.05 us) is the latency of a launch and one chain of loads.
#include "q4dec_internal.h"
#include "q4dec_serve.h"
#include "serve_internal.h"

namespace q4dec {
Q4DEC_DEBUG_READER(kv_append)

constexpr int kAppendThreads = 256;
constexpr int kAppendWaves = kAppendThreads / 64;
constexpr int kMaxFreqs = 256;

struct AppendArgs {
  const float* q;
  const float* k;
  const float* v;
  int64_t q_stride, k_stride, v_stride;
  int n_q, n_kv;
  const float* q_norm;
  const float* k_norm;
  int v_norm;
  float eps;
  const double* freqs;
  int n_freqs, half;  // half = rot_dim / 2
  const int32_t* positions;
  const int32_t* slots;
  const float* k_scale;
  const float* v_scale;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int64_t n_slots;
  int page_shift;
  uint16_t* q_out;
  int32_t* err;
};

// A lane's 4 or 8 consecutive elements, by 16-byte loads and one store.
template <int E>
__device__ __forceinline__ void load_row(const float* p, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + i);
    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
  }
}

template <int E>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&x)[E]) {
  static_assert(E == 4 || E == 8, "8 or 16 bytes");
  uint32_t w[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) w[i] = f32_to_bf16_rne(x[2 * i]) | uint32_t(f32_to_bf16_rne(x[2 * i + 1])) << 16;
  if constexpr (E == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  if constexpr (E == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Orders this wave's LDS stores before its loads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One rounding, to nearest even, of values clamped to the finite range (the
// conversion would make NaN of larger ones; the clamp keeps a NaN).
__device__ __forceinline__ float clamp_e4m3(float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; }

template <int E>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&x)[E], float scale) {
  float y[E];
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = clamp_e4m3(x[i] / scale);
  int w[E / 4];
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], w[i], true);
  }
  if constexpr (E == 4) *reinterpret_cast<int*>(p) = w[0];
  if constexpr (E == 8) *reinterpret_cast<int2*>(p) = make_int2(w[0], w[1]);
}

// Lanes of a head: 4 elements each, 8 of 512; the others of the wave take the
// next heads. (Spread over all 64, a head of 64 is 4 bytes a lane: 1998 tokens
// of 16 + 4 such heads 12.4 us instead of 7.4, of 12 + 4 heads of 128 11.9
// instead of 9.7.)
constexpr int lanes_of_head(int d) { return d >= 512 ? 64 : d / 4; }
constexpr int heads_of_group(int d) { return kAppendWaves * 64 / lanes_of_head(d); }

template <int D, bool E4M3>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs a) {
  constexpr int L = lanes_of_head(D), E = D / L, H = heads_of_group(D);
  const int heads = a.n_q + 2 * a.n_kv;
  Q4_DCHECK(int(gridDim.y) * H >= heads && a.n_freqs <= kMaxFreqs, kDbgAppendGrid);
  __shared__ float2 turn[kMaxFreqs];  // (cos, sin) of this token's angles
  __shared__ __align__(16) float row[H][D];
  const int t = blockIdx.x;
  const int lane = threadIdx.x % L;  // of the head
  const int mine = L == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / L) : int(threadIdx.x) / L;
  // the row is on its way while the angles are formed
  const int h = int(blockIdx.y) * H + mine;
  const bool is_q = h < a.n_q, is_v = h >= a.n_q + a.n_kv;
  const int hk = is_v ? h - a.n_q - a.n_kv : h - a.n_q;  // key/value head
  float x[E];
  int64_t slot = -1;
  if (h < heads) {
    const float* src = is_q   ? a.q + size_t(t) * a.q_stride + size_t(h) * D
                       : is_v ? a.v + size_t(t) * a.v_stride + size_t(hk) * D
                              : a.k + size_t(t) * a.k_stride + size_t(hk) * D;
    load_row<E>(src + lane * E, x);
    if (!is_q) slot = a.slots[t];
  }
  if (int(threadIdx.x) < a.n_freqs) {
    const double turns = double(a.positions[t]) * a.freqs[threadIdx.x] * 0.15915494309189535;  // 1 / (2 pi)
    float s, c;
    sincospif(float(2.0 * (turns - rint(turns))), &s, &c);
    turn[threadIdx.x] = make_float2(c, s);
  }
  __syncthreads();
  if (h >= heads) return;
  const float* norm = is_q ? a.q_norm : is_v ? nullptr : a.k_norm;
  if (is_v ? a.v_norm != 0 : norm != nullptr) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
    const float inv = 1.0f / sqrtf(group_sum<L>(ss) * (1.0f / D) + a.eps);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] *= inv;
    if (!is_v) {
      float w[E];
      load_row<E>(norm + lane * E, w);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] *= w[i];
    }
  }
  if (!is_v && a.n_freqs > 0) {
#pragma unroll
    for (int i = 0; i < E; ++i) row[mine][lane * E + i] = x[i];
    wave_sync();
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int j = lane * E + i;
      const bool upper = j >= a.half;
      const int f = upper ? j - a.half : j;
      if (f < a.n_freqs) {
        const float2 cs = turn[f];
        const float o = row[mine][upper ? f : j + a.half];
        x[i] = upper ? x[i] * cs.x + o * cs.y : x[i] * cs.x - o * cs.y;
      }
    }
  }
  if (is_q) {
    store_bf16<E>(a.q_out + (size_t(t) * a.n_q + h) * D + lane * E, x);
    return;
  }
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    if (a.err && lane == 0) *a.err = 1;
    return;
  }
  const int64_t page = slot >> a.page_shift, at = slot & ((int64_t(1) << a.page_shift) - 1);
  const size_t off = ((size_t(page) * a.n_kv + hk) << a.page_shift) * D + size_t(at) * D + lane * E;
  uint8_t* cache = is_v ? a.v_cache : a.k_cache;
  if constexpr (E4M3) {
    const float* sc = is_v ? a.v_scale : a.k_scale;
    store_e4m3<E>(cache + off, x, sc ? sc[hk] : 1.0f);
  } else {
    store_bf16<E>(reinterpret_cast<uint16_t*>(cache) + off, x);
  }
}

}  // namespace q4dec

extern "C" int kv_append_rope(const float* q, int64_t q_stride, const float* k, int64_t k_stride, const float* v,
                              int64_t v_stride, int64_t n_tok, int64_t n_q, int64_t n_kv, int64_t head_dim,
                              const float* q_norm, const float* k_norm, int32_t v_norm, float eps,
                              const double* freqs, int64_t n_freqs, int64_t rot_dim, const int32_t* positions,
                              const int32_t* slots, int32_t kv_type, const float* k_scale, const float* v_scale,
                              void* k_cache, void* v_cache, int64_t n_pages, int64_t page_size, uint16_t* q_out,
                              int32_t* err_flag, void* stream) {
  using namespace q4dec;
  const char* name = "kv_append_rope";
  if (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 512)
    return fail(Q4DEC_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128, 256 or 512 (got %lld)", name,
                (long long)head_dim);
  if (n_tok < 0 || n_tok >= (int64_t(1) << 24))  // (a workgroup each, 2^32 threads)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_tok must be in [0, 2^24) (got %lld)", name, (long long)n_tok);
  if (n_q < 0 || n_kv < 0 || n_q + n_kv == 0 || n_q > kMaxHeads || n_kv > kMaxHeads)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_q and n_kv must be in [0, 4096], not both 0 (got %lld, %lld)", name,
                (long long)n_q, (long long)n_kv);
  if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
    return fail(Q4DEC_ERR_SHAPE, "%s: rot_dim must be even and in [2, head_dim] (got %lld)", name,
                (long long)rot_dim);
  if (n_freqs < 0 || n_freqs > rot_dim / 2)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_freqs must be in [0, rot_dim / 2] (got %lld)", name, (long long)n_freqs);
  if (!(eps >= 0.0f)) return fail(Q4DEC_ERR_SHAPE, "%s: eps must not be negative or NaN", name);
  if (n_tok == 0) return Q4DEC_OK;  // (tensors without elements have no address)
  if (n_freqs > 0 && !freqs) return fail(Q4DEC_ERR_NULL, "%s: freqs is NULL", name);
  if (n_freqs > 0 && !positions) return fail(Q4DEC_ERR_NULL, "%s: positions is NULL", name);
  if (!aligned(freqs, 8)) return fail(Q4DEC_ERR_ALIGN, "%s: freqs must be 8-byte aligned", name);
  if (!aligned(positions, 4) || !aligned(slots, 4))
    return fail(Q4DEC_ERR_ALIGN, "%s: positions and slots must be 4-byte aligned", name);
  if (!aligned(q_norm, 16) || !aligned(k_norm, 16))
    return fail(Q4DEC_ERR_ALIGN, "%s: q_norm and k_norm must be 16-byte aligned", name);
  if (n_q > 0) {
    if (!q) return fail(Q4DEC_ERR_NULL, "%s: q is NULL", name);
    if (!q_out) return fail(Q4DEC_ERR_NULL, "%s: q_out is NULL", name);
    if (q_stride < n_q * head_dim || q_stride % 4)
      return fail(Q4DEC_ERR_SHAPE, "%s: q_stride must be a multiple of 4 and at least n_q * head_dim (got %lld)", name,
                  (long long)q_stride);
    if (!aligned(q, 16) || !aligned(q_out, 16))
      return fail(Q4DEC_ERR_ALIGN, "%s: q and q_out must be 16-byte aligned", name);
  }
  int page_shift = 0;
  if (n_kv > 0) {
    if (!k) return fail(Q4DEC_ERR_NULL, "%s: k is NULL", name);
    if (!v) return fail(Q4DEC_ERR_NULL, "%s: v is NULL", name);
    if (!slots) return fail(Q4DEC_ERR_NULL, "%s: slots is NULL", name);
    if (k_stride < n_kv * head_dim || k_stride % 4)
      return fail(Q4DEC_ERR_SHAPE, "%s: k_stride must be a multiple of 4 and at least n_kv * head_dim (got %lld)",
                  name, (long long)k_stride);
    if (v_stride < n_kv * head_dim || v_stride % 4)
      return fail(Q4DEC_ERR_SHAPE, "%s: v_stride must be a multiple of 4 and at least n_kv * head_dim (got %lld)",
                  name, (long long)v_stride);
    if (!aligned(k, 16) || !aligned(v, 16))
      return fail(Q4DEC_ERR_ALIGN, "%s: k and v must be 16-byte aligned", name);
    const int rc = check_cache(name, k_cache, v_cache, kv_type, n_pages, page_size, k_scale, v_scale, &page_shift);
    if (rc != Q4DEC_OK) return rc;
  }
  AppendArgs a;
  a.q = q, a.k = k, a.v = v;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.n_q = int(n_q), a.n_kv = int(n_kv);
  a.q_norm = q_norm, a.k_norm = k_norm, a.v_norm = v_norm, a.eps = eps;
  a.freqs = freqs, a.n_freqs = int(n_freqs), a.half = int(rot_dim / 2);
  a.positions = positions, a.slots = slots;
  a.k_scale = k_scale, a.v_scale = v_scale;
  a.k_cache = static_cast<uint8_t*>(k_cache), a.v_cache = static_cast<uint8_t*>(v_cache);
  a.n_slots = n_pages * page_size, a.page_shift = page_shift;
  a.q_out = q_out, a.err = err_flag;
  const int heads = a.n_q + 2 * a.n_kv;
  const dim3 grid(unsigned(n_tok), unsigned((heads + heads_of_group(int(head_dim)) - 1) / heads_of_group(int(head_dim))));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool f8 = n_kv > 0 && kv_type == Q4DEC_KV_E4M3;
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kAppendThreads), 0, st, a); };
  switch (int(head_dim)) {
    case 64: f8 ? go(kv_append_kernel<64, true>) : go(kv_append_kernel<64, false>); break;
    case 128: f8 ? go(kv_append_kernel<128, true>) : go(kv_append_kernel<128, false>); break;
    case 256: f8 ? go(kv_append_kernel<256, true>) : go(kv_append_kernel<256, false>); break;
    default: f8 ? go(kv_append_kernel<512, true>) : go(kv_append_kernel<512, false>); break;
  }
  return launch_status(name);
}
