// paged_attention_shared: the attention of paged_attention where the sequences
// of a group begin with the same positions. Softmax sums can be cut anywhere
// along the keys, so a row's sums are formed in two parts:
//  1. over the positions that a group shares, by all rows of the group
//     together: the keys and values are read once for 128 rows (or 16, where
//     the groups have few), not once for every sequence;
//  2. over the positions after them, sequence by sequence;
// and joined: m = max_i m_i, l = sum_i l_i 2^(m_i - m), o = sum_i o_i 2^(m_i - m)
// over all pieces of both parts, in their order.
// The parts are the kernels of paged_attention with other bounds
// (attention_kernels.h), so their cut into equal stretches from the lengths on
// the device holds here too.
#include "attention_kernels.h"
#include "q4dec_rollout.h"

namespace q4dec {
Q4DEC_DEBUG_READER(paged_attention_shared)

// Sums of a row and four of its columns over some of its pieces.
struct RowSums {
  float m, l;
  f32x4 x;
  bool blank;  // a piece whose scores are all -infinity (see kBlank)

  // Pieces from, from + STEP .. below n: get(i, ml, o). The lanes' n may differ;
  // a lane without pieces gets piece 0.
  template <int STEP, class GET>
  __device__ __forceinline__ void add(int from, int n, GET get) {
    constexpr int kSide = 8;  // loads in flight
#pragma unroll 1
    for (int at = from; __any(at < n); at += kSide * STEP) {
      float2 ml[kSide];
      f32x4 o[kSide];
#pragma unroll
      for (int j = 0; j < kSide; ++j) {
        const int i = at + j * STEP;
        get(i < n ? i : 0, ml[j], o[j]);
        const bool on = i < n;
        ml[j] = on ? ml[j] : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = on ? o[j][e] : 0.0f;
      }
      float mx = m;
#pragma unroll
      for (int j = 0; j < kSide; ++j) mx = fmaxf(mx, ml[j].x);
      const float base = mx == -INFINITY ? 0.0f : mx, f0 = __builtin_amdgcn_exp2f(m - base);
      l *= f0;
      x *= f0;
#pragma unroll
      for (int j = 0; j < kSide; ++j) {
        const float f = __builtin_amdgcn_exp2f(ml[j].x - base);
        blank |= (ml[j].x == -INFINITY) & (ml[j].y != 0.0f);
        l += ml[j].y * f;
        x += o[j] * f;
      }
      m = mx;
    }
  }
  // where x is NaN: again, with infinities that stay (see `scaled`)
  template <int STEP, class GET>
  __device__ __forceinline__ f32x4 again(int from, int n, GET get) const {
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
    for (int i = from; __any(i < n); i += STEP) {
      float2 ml;
      f32x4 o;
      get(i < n ? i : 0, ml, o);
      if (i < n) y += scaled(o, __builtin_amdgcn_exp2f(ml.x - base));
    }
    return y;
  }
  __device__ __forceinline__ void join(const RowSums& b) {
    const float mx = fmaxf(m, b.m), base = mx == -INFINITY ? 0.0f : mx;
    const float f = __builtin_amdgcn_exp2f(m - base), g = __builtin_amdgcn_exp2f(b.m - base);
    m = mx;
    l = l * f + b.l * g;
    x = scaled(x, f) + scaled(b.x, g);
    blank |= b.blank;
  }
};

// Four waves share the pieces of 32 rows of a head and 8 columns. One pass: the
// maximum is followed as it goes, since finding it first is a second chain of
// loads. Bound by reading the partial results (33 MB for 128 rows of two heads of
// 256 in 128 pieces each: 8.5 us); 2, 8 and 16 waves: 4, 0 and 15 us more. MANY:
// the shared part's results are attn_many_kernel's.
constexpr int kJoinWaves = 4;
template <int D, bool MANY>
__global__ __launch_bounds__(64 * kJoinWaves) void join_shared_kernel(AttnArgs a, Partials begin, Partials own) {
  __shared__ RowSums other[kJoinWaves - 1][64];
  const int lane = threadIdx.x & 63, taker = threadIdx.x >> 6, c = lane & 31, half = lane >> 5;
  const int block = blockIdx.x / (D / 8), piece = blockIdx.x % (D / 8), h = blockIdx.y, col = 8 * piece + 4 * half;
  const int64_t rows = int64_t(a.n_tok) * a.group, at = int64_t(block) * 32 + c, row = at < rows ? at : rows - 1;
  const int64_t of = row / a.group * a.n_q + h * a.group + row % a.group;  // its row of q and out
  const int2 mine = own.rows_of[of], common = begin.rows_of[of];
  const int n_own = mine.y >> 8, r_own = mine.y >> 1 & 127;
  // (of a row that shares nothing the second is whatever was there)
  int n_begin = (mine.y & 1) && n_own > 0 ? common.y >> 8 : 0;
  const int r_begin = common.y >> 1 & 127;
  if (n_begin < 0 || common.x < 0 || common.x > begin.slots - n_begin || r_begin >= begin.rows) n_begin = 0;

  auto get = [&](int i, float2& ml, f32x4& o) {  // the shared part's first
    const float2* from_ml;
    const f32x4* from;
    if (i < n_begin) {
      const size_t slot = size_t(common.x) + i;
      if constexpr (MANY) {
        const size_t b = block_at(begin, slot, r_begin >> 5);
        from_ml = begin.ml + b * 32 + (r_begin & 31);
        from = reinterpret_cast<const f32x4*>(begin.o) + (b * (D / 8) + piece) * 64 + half * 32 + (r_begin & 31);
      } else {
        from_ml = begin.ml + slot * kFewRows + r_begin;
        from = reinterpret_cast<const f32x4*>(begin.o + (slot * begin.rows + r_begin) * D + col);
      }
    } else {
      const size_t slot = size_t(mine.x) + (i - n_begin);
      from_ml = own.ml + slot * kFewRows + r_own;
      from = reinterpret_cast<const f32x4*>(own.o + (slot * own.rows + r_own) * D + col);
    }
    ml = *from_ml;
    o = *from;
  };
  const int n = n_begin + n_own;
  RowSums s = {-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}, false};
  s.add<kJoinWaves>(taker, n, get);
  if (__ballot(any_nan(s.x))) s.x = s.again<kJoinWaves>(taker, n, get);
  if (taker > 0) other[taker - 1][lane] = s;
  __syncthreads();
  if (taker > 0) return;
#pragma unroll
  for (int w = 1; w < kJoinWaves; ++w) s.join(other[w - 1][lane]);
  if (at >= rows || n_own == 0) return;
  if (s.m == -INFINITY && s.blank) s.l = NAN;
  const float inv = s.l == 0.0f ? 0.0f : (a.v_scale ? a.v_scale[h] : 1.0f) / s.l;
  *reinterpret_cast<uint2*>(a.out + size_t(of) * D + col) =
      make_uint2(pack_bf16(s.x[0] * inv, s.x[1] * inv), pack_bf16(s.x[2] * inv, s.x[3] * inv));
}

// How a call is cut. Depends on the bounds only.
struct SharedPlan {
  bool plain;  // paged_attention's own plan: sharing does not pay
  bool many;   // the shared part by attn_many_kernel
  int halves;  // of its keys
  int begin_wgs, least, own_wgs;
  int begin_slots, begin_rows, own_slots, own_rows;
  int64_t begin_blocks, own_blocks;  // bounds on the blocks, 2^31 if there may be more
  size_t begin_o, begin_ml, own_o, own_ml, rows, floors;
};
SharedPlan shared_plan_of(int64_t n_tok, int64_t n_seq, int64_t n_groups, int64_t n_q, int64_t n_kv, int64_t d, int64_t max_q,
                          int64_t max_kv, int64_t max_shared) {
  SharedPlan p = {};
  const int64_t group = n_q / n_kv, cus = device_cu_count(), resident = (d >= 512 ? 1 : 2) * cus, limit = int64_t(1) << 31;
  if (max_q > n_tok) max_q = n_tok;
  p.plain = n_groups == 0 || max_shared < 16 || n_groups >= n_seq || max_q * group > 128 || n_tok * group > (1 << 22);
  if (p.plain) return p;
  // the shared part: groups of at most n_tok rows in all
  p.many = n_tok * group > 2 * kFewRows * n_groups;
  const int64_t tile = p.many ? kManyRows : kFewRows, block = p.many ? (d <= 128 ? 64 : 32) : 64;
  const int64_t tiles = n_tok * group / tile + n_groups;  // (each group's last one may be short)
  const int64_t blocks = max_shared / block + 1;
  // Partial results are as many bytes as the keys: 128 rows of 256 are 131 KB, and
  // so are 128 such keys and values. Two groups of waves that share a unit's keys
  // halve them (32 sequences of 4 rows, 32768 positions: 56.6 us and 51.1), which
  // for narrower heads makes no difference and for 512-wide ones has no room.
  p.halves = d == 256 ? 2 : 1;
  p.least = p.many ? 4 : 1;  // (4, 8, 16: 512-wide heads 81.5, 81.3 and 84.3 us, 128-wide 48.5, 50.9 and 54.8)
  p.begin_blocks = tiles * n_kv > limit / blocks ? limit : tiles * n_kv * blocks;
  const int64_t most = (p.begin_blocks + p.least - 1) / p.least, places = p.many ? resident / p.halves : resident;
  p.begin_wgs = int(most < places ? most : places);
  p.begin_rows = int(n_tok * group < tile ? n_tok * group : tile);
  if (p.many) p.begin_rows = (p.begin_rows + 31) / 32 * 32;
  // each sequence's own part
  const int64_t of_one = n_seq * ((max_q * group + kFewRows - 1) / kFewRows), of_all = n_tok * group / kFewRows + n_seq;
  const int64_t units = n_kv * (of_one < of_all ? of_one : of_all), own_blocks = (max_kv + 15) / 64 + 1;
  p.own_blocks = units > limit / own_blocks ? limit : units * own_blocks;
  p.own_wgs = int(p.own_blocks < resident ? p.own_blocks : resident);
  p.own_rows = int(max_q * group < kFewRows ? max_q * group : kFewRows);
  if (p.begin_blocks >= limit || p.own_blocks >= limit) return p;
  p.begin_slots = int(p.begin_wgs + tiles * n_kv);
  p.own_slots = int(p.own_wgs + units);
  p.begin_o = align256(size_t(p.begin_slots) * p.begin_rows * d * sizeof(float));
  p.begin_ml = align256(size_t(p.begin_slots) * (p.many ? p.begin_rows : kFewRows) * sizeof(float2));
  p.own_o = align256(size_t(p.own_slots) * p.own_rows * d * sizeof(float));
  p.own_ml = align256(size_t(p.own_slots) * kFewRows * sizeof(float2));
  p.rows = align256(size_t(n_tok) * n_q * sizeof(int2));
  p.floors = align256(size_t(n_seq) * sizeof(int));
  return p;
}

}  // namespace q4dec

extern "C" size_t paged_attention_shared_workspace_bytes(int64_t n_tok, int64_t n_seq, int64_t n_groups, int64_t n_q,
                                                         int64_t n_kv, int64_t head_dim, int64_t max_q_len,
                                                         int64_t max_kv_len, int64_t max_shared_len) {
  using namespace q4dec;
  if (n_seq <= 0 || n_seq > 65535 || n_groups < 0 || n_groups > 65535 || n_kv <= 0 || n_q <= 0 || n_q > kMaxHeads ||
      n_q % n_kv || n_q / n_kv > kMaxGroup || (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 512) ||
      n_tok <= 0 || n_tok >= (int64_t(1) << 31) / n_q || max_q_len <= 0 || max_q_len >= (int64_t(1) << 30) / n_q ||
      max_kv_len < 0 || max_kv_len > (int64_t(1) << 30) || max_shared_len < 0 || max_shared_len > max_kv_len)
    return 0;
  const SharedPlan p = shared_plan_of(n_tok, n_seq, n_groups, n_q, n_kv, head_dim, max_q_len, max_kv_len, max_shared_len);
  if (p.plain) return paged_attention_workspace_bytes(n_seq, n_q, n_kv, head_dim, max_q_len, max_kv_len, 0);
  return p.begin_o + p.begin_ml + p.own_o + p.own_ml + 2 * p.rows + p.floors;
}

extern "C" int paged_attention_shared(const uint16_t* q, int64_t n_tok, int64_t n_q, int64_t n_kv, int64_t head_dim,
                                      const void* k_cache, const void* v_cache, int32_t kv_type, int64_t n_pages,
                                      int64_t page_size, const float* k_scale, const float* v_scale,
                                      const int32_t* page_table, int64_t table_stride, const int32_t* q_starts,
                                      const int32_t* kv_lens, int64_t n_seq, const int32_t* group_starts,
                                      const int32_t* shared_lens, int64_t n_groups, int64_t max_q_len, int64_t max_kv_len,
                                      int64_t max_shared_len, float scale, void* ws, size_t ws_bytes, uint16_t* out,
                                      int32_t* err_flag, void* stream) {
  using namespace q4dec;
  const char* name = "paged_attention_shared";
  int page_shift = 0;
  const int rc = check_attention(name, q, n_tok, n_q, n_kv, head_dim, k_cache, v_cache, kv_type, n_pages, page_size, k_scale,
                                 v_scale, page_table, table_stride, q_starts, kv_lens, n_seq, max_q_len, max_kv_len, scale,
                                 out, &page_shift);
  if (rc != Q4DEC_OK || n_seq == 0 || n_tok == 0) return rc;
  if (n_groups < 0 || n_groups > 65535)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_groups must be in [0, 65535] (got %lld)", name, (long long)n_groups);
  if (max_shared_len < 0 || max_shared_len > max_kv_len)
    return fail(Q4DEC_ERR_SHAPE, "%s: max_shared_len must be in [0, max_kv_len] (got %lld)", name, (long long)max_shared_len);
  if (n_groups > 0 && !group_starts) return fail(Q4DEC_ERR_NULL, "%s: group_starts is NULL", name);
  if (n_groups > 0 && !shared_lens) return fail(Q4DEC_ERR_NULL, "%s: shared_lens is NULL", name);
  if (!aligned(group_starts, 4) || !aligned(shared_lens, 4))
    return fail(Q4DEC_ERR_ALIGN, "%s: group_starts and shared_lens must be 4-byte aligned", name);
  const SharedPlan p = shared_plan_of(n_tok, n_seq, n_groups, n_q, n_kv, head_dim, max_q_len, max_kv_len, max_shared_len);
  if (p.begin_blocks >= (int64_t(1) << 31) || p.own_blocks >= (int64_t(1) << 31))
    return fail(Q4DEC_ERR_UNSUPPORTED, "%s: the bounds allow 2^31 pieces of work or more", name);
  const size_t need = paged_attention_shared_workspace_bytes(n_tok, n_seq, n_groups, n_q, n_kv, head_dim, max_q_len,
                                                             max_kv_len, max_shared_len);
  if (need > 0 && !ws) return fail(Q4DEC_ERR_NULL, "%s: ws is NULL", name);
  if (ws_bytes < need)
    return fail(Q4DEC_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws_bytes, need);
  if (!aligned(ws, 256)) return fail(Q4DEC_ERR_ALIGN, "%s: ws must be 256-byte aligned", name);
  if (p.plain)
    return paged_attention(q, n_tok, n_q, n_kv, head_dim, k_cache, v_cache, kv_type, n_pages, page_size, k_scale, v_scale,
                           page_table, table_stride, q_starts, kv_lens, n_seq, max_q_len, max_kv_len, scale, 0, ws, ws_bytes,
                           out, err_flag, stream);
  SharedArgs s;
  s.q = q, s.out = out;
  s.k_cache = static_cast<const uint8_t*>(k_cache), s.v_cache = static_cast<const uint8_t*>(v_cache);
  s.k_scale = k_scale, s.v_scale = v_scale;
  s.page_table = page_table, s.q_starts = q_starts, s.kv_lens = kv_lens, s.err = err_flag;
  s.table_stride = table_stride;
  s.n_seq = int(n_seq), s.n_tok = int(n_tok), s.n_q = int(n_q), s.n_kv = int(n_kv), s.group = int(n_q / n_kv);
  s.n_pages = int(n_pages), s.page_shift = page_shift;
  s.max_q = int(max_q_len < n_tok ? max_q_len : n_tok), s.max_kv = int(max_kv_len);
  s.window = 0, s.scale = scale;
  s.group_starts = group_starts, s.shared_lens = shared_lens;
  s.n_all = int(n_seq), s.n_groups = int(n_groups), s.max_shared = int(max_shared_len);
  s.floors = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + p.begin_o + p.begin_ml + p.own_o + p.own_ml + 2 * p.rows);
  BeginArgs ba;
  static_cast<SharedArgs&>(ba) = s;
  ba.n_seq = int(n_groups);
  OwnArgs oa;
  static_cast<SharedArgs&>(oa) = s;
  uint8_t* at = static_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    uint8_t* x = at;
    at += bytes;
    return x;
  };
  Partials begin = {}, own = {};
  begin.o = reinterpret_cast<float*>(take(p.begin_o)), begin.ml = reinterpret_cast<float2*>(take(p.begin_ml));
  own.o = reinterpret_cast<float*>(take(p.own_o)), own.ml = reinterpret_cast<float2*>(take(p.own_ml));
  begin.rows_of = reinterpret_cast<int2*>(take(p.rows)), own.rows_of = reinterpret_cast<int2*>(take(p.rows));
  begin.rows = p.begin_rows, own.rows = p.own_rows, begin.slots = p.begin_slots, own.slots = p.own_slots;
  begin.cleared = own.rows_of;  // (rows of q that belong to no sequence have no pieces)
  hipStream_t st = static_cast<hipStream_t>(stream);
  auto go = [&](auto dim, auto f8) {
    constexpr int D = decltype(dim)::value;
    constexpr bool F8 = decltype(f8)::value;
    constexpr int few_lds = kAttnWaves * (D + 4) * int(sizeof(float));
    constexpr int kHalves = D == 256 ? 2 : 1;
    if (p.many)
      hipLaunchKernelGGL((attn_many_kernel<D, F8, kHalves, BeginArgs>), dim3(p.begin_wgs),
                         dim3(ManyGeometry<D>::THREADS * kHalves), ManyGeometry<D>::kLds * kHalves, st, ba, begin, p.begin_wgs,
                         p.least);
    else
      hipLaunchKernelGGL((attn_few_kernel<D, F8, false, BeginArgs>), dim3(p.begin_wgs), dim3(kAttnThreads),
                         size_t(few_lds) * p.begin_rows, st, ba, begin, p.begin_wgs);
    hipLaunchKernelGGL((attn_few_kernel<D, F8, false, OwnArgs>), dim3(p.own_wgs), dim3(kAttnThreads),
                       size_t(few_lds) * p.own_rows, st, oa, own, p.own_wgs);
    const unsigned blocks = unsigned((n_tok * s.group + 31) / 32);
    const dim3 grid(blocks * (D / 8), unsigned(n_kv));
    if (p.many)
      hipLaunchKernelGGL((join_shared_kernel<D, true>), grid, dim3(64 * kJoinWaves), 0, st, oa, begin, own);
    else
      hipLaunchKernelGGL((join_shared_kernel<D, false>), grid, dim3(64 * kJoinWaves), 0, st, oa, begin, own);
  };
  auto by_type = [&](auto dim) {
    kv_type == Q4DEC_KV_E4M3 ? go(dim, std::true_type{}) : go(dim, std::false_type{});
  };
  switch (int(head_dim)) {
    case 64: by_type(std::integral_constant<int, 64>{}); break;
    case 128: by_type(std::integral_constant<int, 128>{}); break;
    case 256: by_type(std::integral_constant<int, 256>{}); break;
    default: by_type(std::integral_constant<int, 512>{}); break;
  }
  return launch_status(name);
}
