// paged_attention: the plan of a call, its checks and launches. The kernels are
// in attention_kernels.h.
#include "attention_kernels.h"

namespace q4dec {
Q4DEC_DEBUG_READER(paged_attention)

// How a call is cut into workgroups. Depends on the bounds only, so a
// captured call replays with other lengths.
struct AttnPlan {
  bool many;
  bool whole;      // a workgroup a unit
  int halves;      // groups of waves that share a unit's keys (many rows)
  int workgroups;
  int least;       // blocks of a stretch (many rows)
  int rows;        // of a partial result
  int64_t owners;  // entries of Partials::owned
  int tiles;       // as there
  bool join;
  int64_t pieces;  // bound on the blocks, 2^31 if there may be more
  size_t o_bytes, ml_bytes, owned_bytes;
};
AttnPlan plan_of(int64_t n_seq, int64_t n_q, int64_t n_kv, int64_t d, int64_t max_q, int64_t max_kv, int64_t window) {
  AttnPlan p = {};
  const int64_t group = n_q / n_kv, rows = max_q * group, cus = device_cu_count();
  p.many = rows > 2 * kFewRows;
  const int64_t tile = p.many ? kManyRows : kFewRows, tiles = (rows + tile - 1) / tile;
  // keys a unit's rows see at most, with the first group of 16 partly used
  const int64_t tokens = p.many ? (tile + group - 2) / group + 1 : max_q;
  int64_t keys = max_kv;
  if (window > 0 && window < keys - tokens - 15) keys = window + tokens + 15;  // (any window up to 2^63 - 1)
  const int64_t block = p.many ? (d <= 128 ? 64 : 32) : 64;  // (few rows: the smallest kind)
  const int64_t units = n_seq * n_kv * tiles, unit_blocks = (keys + 15) / block + 1, limit = int64_t(1) << 31;
  p.pieces = units > limit / unit_blocks ? limit : units * unit_blocks;
  // A stretch of few blocks is mostly its beginning and its partial result,
  // and a unit in many pieces keeps the join busy: at least 1/64 of a unit, 4
  // to 16 blocks. 64 tokens over 32768 keys (513 blocks a unit) take 60 us
  // with 16 blocks at least and 87 with 4 or 8, chunks under a window of 512
  // (19 blocks a unit) 80 us with 16 and 56 with 4.
  const int64_t share = keys / block / 64;
  p.least = p.many ? int(share < 4 ? 4 : share > 16 ? 16 : share) : 1;
  // as many as are resident at once (512-wide heads: one a compute unit),
  // and no more than there are stretches
  p.halves = 1;
  const int64_t resident = (d >= 512 ? 1 : 2) * cus, most = (p.pieces + p.least - 1) / p.least;
  p.workgroups = int(most < resident ? most : resident);
  p.join = p.workgroups > 1;
  // Short units go to a workgroup each, with no partial results and no join:
  // six chunks of 512 under a window of 512 (19 blocks a unit) take 36 us so
  // and 58 in equal stretches, two prompts of 2048 over 8 heads of 128 (33
  // blocks, twice the units that are resident) 81 and 163. Long units of
  // uneven lengths would keep few busy (five chunks up to 12288 keys: 2050 us
  // and 1040), and few units leave most of the chip idle (16 units of 34
  // blocks: 44 us and 31). Units that have a compute unit to themselves are
  // shared by two groups of waves: those six chunks 32 us, 64 units of 33
  // blocks 40 us and 48 in stretches; not units of a few blocks (7: 19 us, by
  // one group 17), and not where two workgroups fit, which wait for each
  // other less (the 12288 keys again: 1140 us in halves).
  const bool alone = d <= 256 && units <= cus;
  if (p.many && units <= 16 * resident &&
      (unit_blocks <= 32 || (unit_blocks <= 64 && (units >= 2 * resident || (alone && units >= cus / 8)))))
    p.workgroups = int(units), p.join = false, p.whole = true, p.halves = alone && unit_blocks > 8 ? 2 : 1;
  // Few rows likewise, by 8 waves: 64 tokens under a window of 512, 32 / 8
  // heads of 128, take 34 us so and 36 in stretches, 4 tokens over 300 keys 9
  // and 11, 32 tokens over 2000 e4m3 keys 29 and 36; but over 2000 bf16 keys 8
  // tokens (64 units) 27 and 19, one token (2 units) 25 and 10.5. Wider heads leave 8 waves too few registers
  // (the window of 512 with heads of 256: 17 us and 12).
  if (!p.many && d <= 128 && (keys <= 544 || (keys <= 2048 && units >= cus)) && units <= 16 * resident)
    p.workgroups = int(units), p.join = false, p.whole = true;
  p.rows = int(rows < tile ? rows : tile);
  if (p.many) p.rows = (p.rows + 31) / 32 * 32;
  p.o_bytes = p.join ? align256(size_t(p.workgroups) * 2 * p.rows * d * sizeof(float)) : 0;
  p.ml_bytes = p.join ? align256(size_t(p.workgroups) * 2 * (p.many ? p.rows : kFewRows) * sizeof(float2)) : 0;
  p.owners = units < p.workgroups ? units : p.workgroups;
  p.tiles = units < p.workgroups ? int(tiles) : 0;
  p.owned_bytes = p.join ? align256(size_t(p.owners) * sizeof(Owned)) : 0;
  return p;
}

}  // namespace q4dec

extern "C" size_t paged_attention_workspace_bytes(int64_t n_seq, int64_t n_q, int64_t n_kv, int64_t head_dim,
                                                  int64_t max_q_len, int64_t max_kv_len, int64_t window) {
  using namespace q4dec;
  if (n_seq <= 0 || n_seq > 65535 || n_kv <= 0 || n_q <= 0 || n_q > kMaxHeads || n_q % n_kv || n_q / n_kv > kMaxGroup ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 512) || max_q_len <= 0 ||
      max_q_len >= (int64_t(1) << 30) / n_q || max_kv_len < 0 || max_kv_len > (int64_t(1) << 30) || window < 0)
    return 0;
  const AttnPlan p = plan_of(n_seq, n_q, n_kv, head_dim, max_q_len, max_kv_len, window);
  return p.o_bytes + p.ml_bytes + p.owned_bytes;
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
  int page_shift = 0;
  const int rc = check_attention(name, q, n_tok, n_q, n_kv, head_dim, k_cache, v_cache, kv_type, n_pages, page_size, k_scale,
                                 v_scale, page_table, table_stride, q_starts, kv_lens, n_seq, max_q_len, max_kv_len, scale,
                                 out, &page_shift);
  if (rc != Q4DEC_OK || n_seq == 0 || n_tok == 0) return rc;
  if (window < 0) return fail(Q4DEC_ERR_SHAPE, "%s: window must not be negative (got %lld)", name, (long long)window);
  const size_t need = paged_attention_workspace_bytes(n_seq, n_q, n_kv, head_dim, max_q_len, max_kv_len, window);
  if (need > 0 && !ws) return fail(Q4DEC_ERR_NULL, "%s: ws is NULL", name);
  if (ws_bytes < need)
    return fail(Q4DEC_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws_bytes, need);
  if (!aligned(ws, 256)) return fail(Q4DEC_ERR_ALIGN, "%s: ws must be 256-byte aligned", name);
  const AttnPlan p = plan_of(n_seq, n_q, n_kv, head_dim, max_q_len, max_kv_len, window);
  if (p.pieces >= (int64_t(1) << 31))
    return fail(Q4DEC_ERR_UNSUPPORTED, "%s: the bounds allow 2^31 pieces of work or more", name);
  AttnArgs a;
  a.q = q, a.out = out;
  a.k_cache = static_cast<const uint8_t*>(k_cache), a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale, a.v_scale = v_scale;
  a.page_table = page_table, a.q_starts = q_starts, a.kv_lens = kv_lens, a.err = err_flag;
  a.table_stride = table_stride;
  a.n_seq = int(n_seq), a.n_tok = int(n_tok), a.n_q = int(n_q), a.n_kv = int(n_kv), a.group = int(n_q / n_kv);
  a.n_pages = int(n_pages), a.page_shift = page_shift;
  a.max_q = int(max_q_len < n_tok ? max_q_len : n_tok), a.max_kv = int(max_kv_len);
  a.window = window, a.scale = scale;
  Partials part;
  part.o = static_cast<float*>(ws);
  part.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + p.o_bytes);
  part.owned = p.join ? reinterpret_cast<Owned*>(static_cast<uint8_t*>(ws) + p.o_bytes + p.ml_bytes) : nullptr;
  part.rows = p.rows, part.tiles = p.tiles;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool many_pieces = p.workgroups >= 64 * p.owners;  // a unit is likely to have
  auto go = [&](auto dim, auto f8) {
    constexpr int D = decltype(dim)::value;
    constexpr bool F8 = decltype(f8)::value;
    if (p.many) {
      auto launch = [&](auto halves) {
        constexpr int H = decltype(halves)::value;
        hipLaunchKernelGGL((attn_many_kernel<D, F8, H>), dim3(p.workgroups), dim3(ManyGeometry<D>::THREADS * H),
                           ManyGeometry<D>::kLds * H, st, a, part, p.workgroups, p.least);
      };
      if constexpr (D <= 256) {
        if (p.halves > 1) launch(std::integral_constant<int, 2>{});
        else launch(std::integral_constant<int, 1>{});
      } else {
        launch(std::integral_constant<int, 1>{});
      }
      if (!p.join) return;
      if (many_pieces)
        hipLaunchKernelGGL((attn_join_many_kernel<D, 4>), dim3(p.rows / 32 * (D / 8), unsigned(p.owners)),
                           dim3(kAttnThreads), 0, st, a, part);
      else
        hipLaunchKernelGGL((attn_join_many_kernel<D, 1>), dim3(p.rows / 32 * (D / 32), unsigned(p.owners)),
                           dim3(kAttnThreads), 0, st, a, part);
      return;
    }
    auto few = [&](auto whole) {
      constexpr bool W = decltype(whole)::value;
      constexpr int waves = FewGeometry<D, F8, W>::WAVES;
      hipLaunchKernelGGL((attn_few_kernel<D, F8, W>), dim3(p.workgroups), dim3(64 * waves),
                         size_t(waves) * p.rows * (D + 4) * sizeof(float), st, a, part, p.workgroups);
    };
    if constexpr (D <= 128)
      if (p.whole) return few(std::true_type{});
    few(std::false_type{});
    if (!p.join) return;
    if (many_pieces)
      hipLaunchKernelGGL((attn_join_kernel<D, 64, 16>), dim3(p.rows * (D / 64), unsigned(p.owners)), dim3(64 * 16), 0,
                         st, a, part);
    else
      hipLaunchKernelGGL((attn_join_kernel<D, D, 4>), dim3(p.rows, unsigned(p.owners)), dim3(64 * 4), 0, st, a, part);
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
