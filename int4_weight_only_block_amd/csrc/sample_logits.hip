// sample_logits: the first and the last of its launches, and its checks. What it
// computes and how is told in sample_kernels.h, with the other two.
#include "sample_kernels.h"

namespace q4dec {
Q4DEC_DEBUG_READER(sample_logits)

#pragma clang fp contract(off)

// 1: one wave per group.
__global__ __launch_bounds__(kGroupThreads) void sample_groups_kernel(SampleArgs a, RowWork* ws) {
  const GroupPlan gp = group_plan(a.vocab);
  Q4_DCHECK(int64_t(gridDim.x) * kGroupWaves >= gp.groups && gp.groups <= kGroups, kDbgSampleGrid);
  group_extremes(ws[blockIdx.y], row_at(a, int(blockIdx.y)), a.vocab);
}

// 4: one workgroup per row.
__global__ __launch_bounds__(kSampleThreads) void sample_draw_kernel(SampleArgs a, RowWork* ws) {
  __shared__ Shared sh;
  __shared__ u64 sums[kGroups];
  __shared__ uint2 small[kGroupThreads];
  __shared__ u64 small_w[kGroupThreads];
  __shared__ int chosen;
  const GroupPlan gp = group_plan(a.vocab);
  const int r = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = t >> 6;
  RowWork& w = ws[r];
  // (loaded before it is known whether it is there: what follows waits less)
  const uint2 first = w.list[t >> 2];
  const uint32_t listed = w.list_n;
  const Filters f = filters_of(a, r);
  const uint32_t n = f.borders() ? listed : 0;
  const RowInfo in = row_info(a.vocab, w, f, f.by_list() && n > kList);
  if (in.plain) {
    // the lowest index among the groups' first-ranked tokens
    for (int i = lane; i < (gp.groups + 63) / 64 * 64 && wave == 0; i += 64) {
      const u64 hit = __ballot(i < gp.groups && w.group_key[min(i, gp.groups - 1)] == in.max_key);
      if (hit) {
        if (lane == int(__ffsll(hit)) - 1) {
          a.idx_out[r] = in.max_key == 0 ? -1 : w.group_idx[i];
          if (a.prob_out) a.prob_out[r] = in.max_key == 0 ? NAN : 1.0f;
        }
        break;
      }
    }
    return;
  }
  const float* z = row_at(a, r);
  const Weights& wt = in.wt;

  if (f.by_list() && n <= kGroupThreads) {
    // four neighbouring threads a token, each compares it with a quarter
    const int at = t >> 2, part = t & 3;
    const uint2 me = at < int(n) ? first : make_uint2(0u, 0u);
    double x = 0.0;
    u64 own = 0;
    if (at < int(n)) {
      x = wt.weight(key_value(me.x));
      own = fixed(x);
      if (part == 0) {
        small[at] = me;
        small_w[at] = own;
      }
    }
    __syncthreads();
    const int count = at < int(n) ? int(n) : 0;
    int rank = 0;
    u64 better = 0;  // weight of the better-ranked
#pragma unroll 4
    for (int j = part; j < count; j += 4) {
      const uint2 o = small[j];
      const bool before = o.x > me.x || (o.x == me.x && o.y < me.y);
      rank += before;
      better += before ? small_w[j] : 0;
    }
    rank += __shfl_xor(rank, 1);
    rank += __shfl_xor(rank, 2);
    better += __shfl_xor(better, 1);
    better += __shfl_xor(better, 2);
    const bool in_k = at < int(n) && rank < f.top_k;
    const u64 s = wave_sum(in_k && part == 0 ? own : 0);
    if (lane == 0) sh.wave[wave] = s;
    __syncthreads();
    u64 whole = 0;  // of what top_k leaves
    for (int i = 0; i < kSampleWaves; ++i) whole += sh.wave[i];
    if (!in_k || (f.top_p < 1.0f && better >= top_p_target(f.top_p, whole)) || x < f.min_p) own = 0;
    if (at < int(n) && part == 0) small_w[at] = own;
    __syncthreads();
    u64 before = 0;
    whole = 0;
#pragma unroll 4
    for (int j = part; j < count; j += 4) {
      const u64 o = small_w[j];
      whole += o;
      before += small[j].y < me.y ? o : 0;
    }
    whole += __shfl_xor(whole, 1);
    whole += __shfl_xor(whole, 2);
    before += __shfl_xor(before, 1);
    before += __shfl_xor(before, 2);
    if (own > 0 && part == 0) {
      const u64 target = drawn_at(a.u[r], whole);
      if (before <= target && target < before + own) {
        a.idx_out[r] = int(me.y);
        if (a.prob_out) a.prob_out[r] = share_of(x, whole);
      }
    }
    return;
  }

  // kept: ranked up to (key_cut, idx_cut)
  uint32_t key_cut;
  int idx_cut;
  cut_row(sh, sums, f, in, w, z, a.vocab, n, key_cut, idx_cut);
  auto kept = [&](uint32_t k, int i) { return k > key_cut || (k == key_cut && i <= idx_cut); };
  __syncthreads();
  // the group that the drawn number falls in (the first-ranked token always stays: the whole is not 0)
  if (t < 64) {
    u64 c[4], own = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) own += c[i] = sums[4 * t + i];
    const u64 upto = wave_upto(own), whole = lane_value(upto, 63), target = drawn_at(a.u[r], whole);
    u64 before = upto - own;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (before <= target && target < before + c[i]) {
        chosen = 4 * t + i;
        sh.rest = target - before;
        sh.hist[0][0] = whole;
      }
      before += c[i];
    }
  }
  __syncthreads();
  u64 target = sh.rest;
  const u64 whole = sh.hist[0][0];
  const int lo = chosen * gp.per, hi = min(lo + gp.per, a.vocab);
  for (int base = lo; base < hi; base += kSampleThreads) {
    const int i = base + t;
    u64 own = 0;
    double x = 0.0;
    if (i < hi) {
      const uint32_t k = order_key(z[i]);
      if (k != 0 && kept(k, i)) {
        x = wt.weight(z[i]);
        own = x >= f.min_p ? fixed(x) : 0;
      }
    }
    const u64 upto = wave_upto(own);
    __syncthreads();
    if (lane == 63) sh.wave[wave] = upto;
    __syncthreads();
    u64 before = upto - own, all = 0;
    for (int v = 0; v < kSampleWaves; ++v) {
      if (v < wave) before += sh.wave[v];
      all += sh.wave[v];
    }
    if (before <= target && target < before + own) {
      a.idx_out[r] = i;
      if (a.prob_out) a.prob_out[r] = share_of(x, whole);
    }
    if (target < all) return;
    target -= all;
  }
}

}  // namespace q4dec

extern "C" size_t sample_logits_workspace_bytes(int64_t n_rows, int64_t vocab) {
  if (n_rows <= 0 || n_rows > 65535 || vocab <= 0 || vocab > (int64_t(1) << 20)) return 0;
  return size_t(n_rows) * sizeof(q4dec::RowWork);
}

extern "C" int sample_logits(const float* logits, int64_t n_rows, int64_t vocab, int64_t row_stride, float cap,
                             const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                             const float* u, void* ws, size_t ws_bytes, int32_t* idx_out, float* prob_out,
                             void* stream) {
  using namespace q4dec;
  const char* name = "sample_logits";
  if (n_rows < 0 || n_rows > 65535)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_rows must be in [0, 65535] (got %lld)", name, (long long)n_rows);
  if (vocab <= 0 || vocab > (int64_t(1) << 20))
    return fail(Q4DEC_ERR_SHAPE, "%s: vocab must be in [1, 2^20] (got %lld)", name, (long long)vocab);
  if (row_stride < vocab)
    return fail(Q4DEC_ERR_SHAPE, "%s: row_stride must be at least vocab (got %lld)", name, (long long)row_stride);
  if (n_rows == 0) return Q4DEC_OK;
  if (!logits) return fail(Q4DEC_ERR_NULL, "%s: logits is NULL", name);
  if (!u) return fail(Q4DEC_ERR_NULL, "%s: u is NULL", name);
  if (!idx_out) return fail(Q4DEC_ERR_NULL, "%s: idx_out is NULL", name);
  if (!aligned(logits, 4) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
      !aligned(min_p, 4) || !aligned(idx_out, 4) || !aligned(prob_out, 4))
    return fail(Q4DEC_ERR_ALIGN, "%s: logits, parameters and outputs must be 4-byte aligned", name);
  const size_t need = sample_logits_workspace_bytes(n_rows, vocab);
  if (need > 0 && !ws) return fail(Q4DEC_ERR_NULL, "%s: ws is NULL", name);
  if (ws_bytes < need)
    return fail(Q4DEC_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws_bytes, need);
  if (!aligned(ws, 256)) return fail(Q4DEC_ERR_ALIGN, "%s: ws must be 256-byte aligned", name);
  const SampleArgs a = {logits, row_stride, int(vocab), double(cap), cap > 0.0f ? 1.0 / double(cap) : 0.0, temperature, top_k, top_p, min_p, u, idx_out, prob_out};
  RowWork* work = static_cast<RowWork*>(ws);
  const GroupPlan gp = group_plan(a.vocab);
  const dim3 grid(unsigned((gp.groups + kGroupWaves - 1) / kGroupWaves), unsigned(n_rows));
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(sample_groups_kernel, grid, dim3(kGroupThreads), 0, st, a, work);
  hipLaunchKernelGGL(sample_bins_kernel<SampleArgs>, grid, dim3(kGroupThreads), 0, st, a, work);
  hipLaunchKernelGGL(sample_sums_kernel<SampleArgs>, grid, dim3(kGroupThreads), 0, st, a, work);
  hipLaunchKernelGGL(sample_draw_kernel, dim3(unsigned(n_rows)), dim3(kSampleThreads), 0, st, a, work);
  return launch_status(name);
}
