// paged_attention_shared: the attention of paged_attention where the sequences
// of a group begin with the same positions. Softmax sums can be cut anywhere
// along the keys, so a row's sums are formed in two parts:
//  - over the positions that a group shares, by all rows of the group
//    together: the keys and values are read once for 128 rows (or 16, where
//    the groups have few), not once for every sequence;
//  - over the positions after them, sequence by sequence;
// and joined: m = max_i m_i, l = sum_i l_i 2^(m_i - m), o = sum_i o_i 2^(m_i - m)
// over all pieces of both parts, in their order.
// The parts are the work of paged_attention with other bounds
// (attention_kernels.h), so their cut into equal stretches from the lengths on
// the device holds here too. Both are done by one launch, a workgroup of each
// on every compute unit: one's waits (and the second is mostly waiting) are the
// other's time.
// Measured: 32 sequences of 4 rows of 2 heads of 256, 32768 shared positions and
// up to 700 of their own 43 us (31 and 11 the join): 95 MB read at 3.1 TB/s beside
// 37 MB of partial results written, and the products with the second part of the
// probabilities (3 us); paged_attention takes 181 us. 16 sequences of 5 tokens over
// 9000 positions of 8 heads of 128 40 us and 105, 24 of 8 rows over 50001 positions
// of 512 87 us and 245.
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

// Both parts: the first `own_wgs` workgroups (a multiple of 8, one or more on each
// die) each sequence's own positions, the others the shared ones.
template <int D, bool F8, bool MANY>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_shared_kernel(BeginArgs ba, Partials begin, OwnArgs oa, Partials own,
                                                                      int begin_wgs, int own_wgs, int least) {
  if (int(blockIdx.x) < own_wgs)
    attn_few<D, F8, false>(oa, own, own_wgs, blockIdx.x, own_wgs);
  else if constexpr (MANY)
    attn_many<D, F8, 1>(ba, begin, begin_wgs, least, blockIdx.x - own_wgs, begin_wgs);
  else
    attn_few<D, F8, false>(ba, begin, begin_wgs, blockIdx.x - own_wgs, begin_wgs);
}
// 512-wide heads: attn_few takes every register of a SIMD for one wave, attn_many
// needs two; a launch each. (Each sequence's own positions by attn_many too, in
// one launch, a compute unit for one or the other: 24 sequences of 8 rows over
// 50001 shared positions 92 us and 83.5, when probabilities had one part.)
template <int D, bool F8, class ARGS>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_few_part_kernel(ARGS a, Partials part, int workgroups) {
  attn_few<D, F8, false>(a, part, workgroups, blockIdx.x, gridDim.x);
}
template <int D, bool F8>
__global__ __launch_bounds__(ManyGeometry<D>::THREADS, 2) void attn_many_part_kernel(BeginArgs a, Partials part, int workgroups,
                                                                                     int least) {
  attn_many<D, F8, 1>(a, part, workgroups, least, blockIdx.x, gridDim.x);
}

// WAVES waves share the pieces of 32 rows of a head and 8 columns: 4, or 16 where
// there are few rows (whose pieces are then many: 16 rows over 32000 positions
// 41.2 us and 32.5; where there are many 16 are slower, 36.8 and 50). One pass:
// the maximum is followed as it goes, since finding it first is a second chain
// of loads. Bound by reading the partial results: 37 MB in 10.9 us. MANY: the
// shared part's results are attn_many's.
template <int D, bool MANY, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void join_shared_kernel(AttnArgs a, Partials begin, Partials own) {
  __shared__ RowSums other[WAVES - 1][64];
  const int lane = threadIdx.x & 63, taker = threadIdx.x >> 6, c = lane & 31, half = lane >> 5;
  const int block = blockIdx.x / (D / 8), piece = blockIdx.x % (D / 8), h = blockIdx.y, col = 8 * piece + 4 * half;
  const int64_t rows = int64_t(a.n_tok) * a.group, at = int64_t(block) * 32 + c, row = at < rows ? at : rows - 1;
  const int token = int(row / a.group);
  const int64_t of = int64_t(token) * a.n_q + h * a.group + row % a.group;  // its row of q and out
  const int4 mine = own.rows_of[of], common = begin.rows_of[of];
  // Is it a row of a sequence? Then this call has written the first of these, and
  // where that says so the second; else they hold anything.
  int start = 0, q_len = 0, kv_len = 0, floor = 0;
  const bool in = mine.w >= 0 && mine.w < a.n_seq && sequence_of(a, mine.w, start, q_len, kv_len, floor) && token >= start &&
                  token - start < q_len;
  const int r_own = mine.z >> 1 & (kFewRows - 1), r_begin = common.z >> 1 & (kManyRows - 1);
  auto pieces_in = [](const Partials& p, const int4& x) { return x.x >= 0 && x.y > 0 && x.x <= p.slots - x.y ? x.y : 0; };
  const int n_own = in && r_own < own.rows ? pieces_in(own, mine) : 0;
  const int n_begin = n_own > 0 && (mine.z & 1) && r_begin < begin.rows ? pieces_in(begin, common) : 0;

  auto get = [&](int i, float2& ml, f32x4& o) {  // the shared part's first; of a row without pieces anything
    const float2* from_ml = own.ml;
    const f32x4* from = reinterpret_cast<const f32x4*>(own.o);
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
    } else if (i < n_begin + n_own) {
      const size_t slot = size_t(mine.x) + (i - n_begin);
      from_ml = own.ml + slot * kFewRows + r_own;
      from = reinterpret_cast<const f32x4*>(own.o + (slot * own.rows + r_own) * D + col);
    }
    ml = *from_ml;
    o = *from;
  };
  const int n = n_begin + n_own;
  RowSums s = {-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}, false};
  s.add<WAVES>(taker, n, get);
  if (__ballot(any_nan(s.x))) s.x = s.again<WAVES>(taker, n, get);
  if (taker > 0) other[taker - 1][lane] = s;
  __syncthreads();
  if (taker > 0) return;
#pragma unroll
  for (int w = 1; w < WAVES; ++w) s.join(other[w - 1][lane]);
  if (at >= rows || n_own == 0) return;
  if (s.m == -INFINITY && s.blank) s.l = NAN;
  const float inv = s.l == 0.0f ? 0.0f : (a.v_scale ? a.v_scale[h] : 1.0f) / s.l;
  *reinterpret_cast<uint2*>(a.out + size_t(of) * D + col) =
      make_uint2(pack_bf16(s.x[0] * inv, s.x[1] * inv), pack_bf16(s.x[2] * inv, s.x[3] * inv));
}

constexpr unsigned kFewJoins = 128;  // workgroups of 4 waves that leave a compute unit idle

// How a call is cut. Depends on the bounds and the bytes of a cached element only.
struct SharedPlan {
  bool plain;  // paged_attention's own plan: sharing does not pay
  bool many;   // the shared part by attn_many
  int begin_wgs, least, own_wgs, together;
  int begin_slots, begin_rows, own_slots, own_rows;
  int64_t begin_blocks, own_blocks;  // bounds on the blocks
  size_t begin_o, begin_ml, own_o, own_ml, rows;
};
SharedPlan shared_plan_of(int64_t n_tok, int64_t n_seq, int64_t n_groups, int64_t n_q, int64_t n_kv, int64_t d, int64_t max_q,
                          int64_t max_kv, int64_t max_shared, int64_t es) {
  SharedPlan p = {};
  const int64_t group = n_q / n_kv, cus = device_cu_count(), limit = int64_t(1) << 31;
  if (max_q > n_tok) max_q = n_tok;
  // What sharing saves reading, in bytes, has to make up for a second launch and
  // for partial results. (us alone / shared: 256-wide heads, 24 sequences over 849
  // positions (40 MB) 18.7 / 25.4, 6 over 7812 (40 MB) 23.3 / 26.6, 12 over 3551
  // (80 MB) 25.3 / 21.9, 4 over 32000 (196 MB) 45.7 / 31.2; in e4m3 12 over 3551
  // (40 MB) 25.7 / 26.2, 48 over 1662 (78 MB) 28.6 / 28.0. Of 64, 3 over 39062 (40 MB)
  // 22.1 / 19.5. 512-wide, with a third launch: 24 over 1273 (115 MB) 36.9 / 44.2, 4
  // over 34000 (208 MB) 59.2 / 66.7, 12 over 10653 (240 MB) 60.3 / 47.1; in e4m3 12 over
  // 10653 (120 MB) 47.6 / 53.1, 6 over 46875 (240 MB) 67.4 / 65.1.) The host knows
  // bounds only: every group counts as if it shared the most, sequences of none as
  // if they did. Rows for a whole tile of a sequence have nothing left to share.
  const double saved = 2.0 * double(n_seq - n_groups) * double(max_shared) * double(n_kv * d * es);
  p.plain = n_groups == 0 || max_shared < 16 || n_groups >= n_seq || max_q * group > 128 || n_tok * group > (1 << 22) ||
            saved < (d >= 512 ? 200e6 : 56e6);
  if (p.plain) return p;
  // the shared part: groups of at most n_tok rows in all
  p.many = n_tok * group > 2 * kFewRows * n_groups;
  const int64_t tile = p.many ? kManyRows : kFewRows, block = p.many ? (d <= 128 ? 64 : 32) : 64;
  const int64_t tiles = n_tok * group / tile + n_groups;  // (each group's last one may be short)
  const int64_t blocks = max_shared / block + 1;
  p.least = p.many ? 4 : 1;  // (4, 8, 16: 512-wide heads 86, 86 and 92 us, 128-wide 39.7, 39.1 and 48.7)
  p.begin_blocks = tiles * n_kv > limit / blocks ? limit : tiles * n_kv * blocks;
  // A workgroup of each part for every compute unit. More of the first would run
  // beside each other, but leave more partial results, which are as many bytes as
  // the keys (128 rows of 256 are 131 KB, and so are 128 such keys and values).
  const int64_t most = (p.begin_blocks + p.least - 1) / p.least;
  p.begin_wgs = int(most < cus ? most : cus);
  // Tiles of rows that read the same keys side by side: 24 sequences of 8 rows of
  // 512, two tiles, 87.5 us and 92.6. Not where it leaves compute units without work
  // (three tiles of 8 heads would have 240 of 256: 37.1 to 38.6 us and 37.3, when
  // probabilities had one part).
  const int64_t row_tiles = (n_tok * group + tile - 1) / tile;
  p.together = p.many && n_groups == 1 && p.begin_wgs % (row_tiles * n_kv) == 0 ? int(row_tiles) : 1;
  p.begin_rows = int(n_tok * group < tile ? n_tok * group : tile);
  if (p.many) p.begin_rows = (p.begin_rows + 31) / 32 * 32;
  // each sequence's own part
  const int64_t of_one = n_seq * ((max_q * group + kFewRows - 1) / kFewRows), of_all = n_tok * group / kFewRows + n_seq;
  const int64_t units = n_kv * (of_one < of_all ? of_one : of_all), own_blocks = (max_kv + 15) / 64 + 1;
  p.own_blocks = units > limit / own_blocks ? limit : units * own_blocks;
  p.own_wgs = int(p.own_blocks < cus ? (p.own_blocks + 7) / 8 * 8 : cus);
  p.own_rows = int(max_q * group < kFewRows ? max_q * group : kFewRows);
  // (32-bit sums of the blocks; paged_attention's units are larger, up to 128 rows of a sequence)
  if (p.begin_blocks >= limit || p.own_blocks >= limit) {
    p = {};
    p.plain = true;
    return p;
  }
  p.begin_slots = int(p.begin_wgs + tiles * n_kv);
  p.own_slots = int(p.own_wgs + units);
  p.begin_o = align256(size_t(p.begin_slots) * p.begin_rows * d * sizeof(float));
  p.begin_ml = align256(size_t(p.begin_slots) * (p.many ? p.begin_rows : kFewRows) * sizeof(float2));
  p.own_o = align256(size_t(p.own_slots) * p.own_rows * d * sizeof(float));
  p.own_ml = align256(size_t(p.own_slots) * kFewRows * sizeof(float2));
  p.rows = align256(size_t(n_tok) * n_q * sizeof(int4));
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
  size_t most = 0;  // (of a cache in either type)
  for (const int64_t es : {1, 2}) {
    const SharedPlan p = shared_plan_of(n_tok, n_seq, n_groups, n_q, n_kv, head_dim, max_q_len, max_kv_len, max_shared_len, es);
    const size_t bytes = p.plain ? paged_attention_workspace_bytes(n_seq, n_q, n_kv, head_dim, max_q_len, max_kv_len, 0)
                                 : p.begin_o + p.begin_ml + p.own_o + p.own_ml + 2 * p.rows;
    if (bytes > most) most = bytes;
  }
  return most;
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
  const SharedPlan p = shared_plan_of(n_tok, n_seq, n_groups, n_q, n_kv, head_dim, max_q_len, max_kv_len, max_shared_len,
                                      kv_type == Q4DEC_KV_E4M3 ? 1 : 2);
  const size_t need = paged_attention_shared_workspace_bytes(n_tok, n_seq, n_groups, n_q, n_kv, head_dim, max_q_len,
                                                             max_kv_len, max_shared_len);
  if (need > 0 && !ws) return fail(Q4DEC_ERR_NULL, "%s: ws is NULL", name);
  if (ws_bytes < need)
    return fail(Q4DEC_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws_bytes, need);
  if (!aligned(ws, 256)) return fail(Q4DEC_ERR_ALIGN, "%s: ws must be 256-byte aligned", name);
  if (p.plain) {
    const int done = paged_attention(q, n_tok, n_q, n_kv, head_dim, k_cache, v_cache, kv_type, n_pages, page_size, k_scale,
                                     v_scale, page_table, table_stride, q_starts, kv_lens, n_seq, max_q_len, max_kv_len, scale,
                                     0, ws, ws_bytes, out, err_flag, stream);
    if (done != Q4DEC_ERR_UNSUPPORTED) return done;
    return fail(done, "%s: the bounds allow 2^31 pieces of work or more", name);
  }
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
  BeginArgs ba;
  static_cast<SharedArgs&>(ba) = s;
  ba.n_seq = int(n_groups);
  ba.tiles = p.together;
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
  begin.rows_of = reinterpret_cast<int4*>(take(p.rows)), own.rows_of = reinterpret_cast<int4*>(take(p.rows));
  begin.rows = p.begin_rows, own.rows = p.own_rows, begin.slots = p.begin_slots, own.slots = p.own_slots;
  hipStream_t st = static_cast<hipStream_t>(stream);
  auto go = [&](auto dim, auto f8) {
    constexpr int D = decltype(dim)::value;
    constexpr bool F8 = decltype(f8)::value;
    auto few_lds = [](int rows) { return (size_t(kAttnWaves) * rows * (D + 4) + D / 32 * 64 * 4) * sizeof(float); };
    const size_t own_lds = few_lds(p.own_rows);
    if constexpr (D <= 256) {
      auto both = [&](auto many, size_t begin_lds) {
        hipLaunchKernelGGL((attn_shared_kernel<D, F8, decltype(many)::value>), dim3(p.own_wgs + p.begin_wgs), dim3(kAttnThreads),
                           own_lds > begin_lds ? own_lds : begin_lds, st, ba, begin, oa, own, p.begin_wgs, p.own_wgs, p.least);
      };
      p.many ? both(std::true_type{}, size_t(ManyGeometry<D>::kLds)) : both(std::false_type{}, few_lds(p.begin_rows));
    } else {
      if (p.many)
        hipLaunchKernelGGL((attn_many_part_kernel<D, F8>), dim3(p.begin_wgs), dim3(ManyGeometry<D>::THREADS),
                           ManyGeometry<D>::kLds, st, ba, begin, p.begin_wgs, p.least);
      else
        hipLaunchKernelGGL((attn_few_part_kernel<D, F8, BeginArgs>), dim3(p.begin_wgs), dim3(kAttnThreads),
                           few_lds(p.begin_rows), st, ba, begin, p.begin_wgs);
      hipLaunchKernelGGL((attn_few_part_kernel<D, F8, OwnArgs>), dim3(p.own_wgs), dim3(kAttnThreads), own_lds, st, oa, own,
                         p.own_wgs);
    }
    const unsigned blocks = unsigned((n_tok * s.group + 31) / 32);
    const dim3 grid(blocks * (D / 8), unsigned(n_kv));
    auto join = [&](auto many, auto waves) {
      constexpr int W = decltype(waves)::value;
      hipLaunchKernelGGL((join_shared_kernel<D, decltype(many)::value, W>), grid, dim3(64 * W), 0, st, oa, begin, own);
    };
    auto join_of = [&](auto many) {
      grid.x * grid.y < kFewJoins ? join(many, std::integral_constant<int, 16>{}) : join(many, std::integral_constant<int, 4>{});
    };
    p.many ? join_of(std::true_type{}) : join_of(std::false_type{});
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
