// verify_drafts: draft x of a row stays if u q(x) < p(x); at the first that
// does not, a token is drawn from max(0, p - q), else from the last row's p.
// p and q are the distributions of sample_logits, whose first three launches
// (sample_kernels.h) run over the target's and the drafter's rows together:
// each row's filters end up as a cut in its ranking and sums of what stays.
//  1. to 3. as there: group maxima; list or histogram; sums;
//  4. a workgroup a row finds the row's cut and the probability of its draft;
//  5. where a sequence stops at a draft that is taken back, the sums of
//     max(0, p - q) over each group of that row's tokens, in 60-bit fixed
//     point (integers: their order does not matter). Groups in which p has
//     nothing are left out: under a small top_k that is nearly all of them;
//  6. a workgroup a sequence draws: the group by the sums, then in the group.
#include "sample_kernels.h"

#include "q4dec_rollout.h"

namespace q4dec {
Q4DEC_DEBUG_READER(verify_drafts)

#pragma clang fp contract(off)

constexpr int64_t kMaxVerifyRows = 32767;  // twice as many are a grid's

// What a row's filters leave: kind 0 nothing, 1 the token idx_cut alone
// (greedy), 2 the tokens ranked up to (key_cut, idx_cut) and not lighter than
// min_p.
struct RowCut {
  double steep, top, min_p;
  u64 whole;
  double draft_share;  // the draft's probability
  float z_max;
  uint32_t key_cut;
  int32_t idx_cut, kind;
};

struct VerifyArgs {
  const float* logits;
  const float* draft_logits;
  int64_t row_stride, draft_stride;
  int vocab, n_rows, n_seq;
  double cap, inv_cap, draft_cap, draft_inv_cap;
  const int32_t* drafts;
  const int32_t* starts;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  const float* u_draw;
  int32_t* tokens;
  float* prob;
  int32_t* count;
  int32_t* err;
  int32_t* seq_of;  // of each row (the drafter's from n_rows on); -1: not used
  RowCut* cuts;
  u64* rest;  // [n_seq][kGroups]: sums of max(0, p - q)
};
__device__ __forceinline__ bool row_used(const VerifyArgs& a, int r) { return a.seq_of[r] >= 0; }
__device__ __forceinline__ const float* row_at(const VerifyArgs& a, int r) {
  return r < a.n_rows ? a.logits + size_t(r) * a.row_stride : a.draft_logits + size_t(r - a.n_rows) * a.draft_stride;
}
__device__ __forceinline__ Filters filters_of(const VerifyArgs& a, int r) {
  const bool target = r < a.n_rows;
  return filters_at(a, a.seq_of[r], target ? a.cap : a.draft_cap, target ? a.inv_cap : a.draft_inv_cap);
}

// The rows of sequence b; false if its bounds are not valid.
__device__ __forceinline__ bool rows_of(const VerifyArgs& a, int b, int& start, int& n) {
  start = a.starts[b];
  const int end = a.starts[b + 1];
  n = 0;
  if (start < 0 || end < start || end > a.n_rows) return false;
  n = end - start;
  return true;
}

// The first launch finds each row's sequence: the last that starts at the row
// or before, by all lanes of a wave, 64 of the starts at a time.
struct FirstArgs : VerifyArgs {};
__device__ __forceinline__ bool row_used(const FirstArgs& a, int r) {
  const int lane = threadIdx.x & 63, row = r < a.n_rows ? r : r - a.n_rows;
  int b = 0, wide = a.n_seq;  // it is among b .. b + wide - 1, if any
  while (wide > 0) {
    const int step = (wide + 63) / 64, at = b + lane * step;
    const u64 low = __ballot(lane * step < wide && a.starts[min(at, a.n_seq)] <= row);
    if (low == 0) break;
    const int last = 63 - __clzll(low);
    wide = step > 1 ? min(step, wide - last * step) : 0;
    b += last * step;
  }
  int start, n;
  const bool in = rows_of(a, b, start, n) && row >= start && row - start < n && !(r >= a.n_rows && row - start == n - 1);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.seq_of[r] = in ? b : -1;
  return in;
}

// The probability of token i with logit z in a row.
__device__ __forceinline__ double share_in(const RowCut& c, double inv_cap, float z, int i) {
  if (c.kind != 2) return c.kind == 1 && i == c.idx_cut ? 1.0 : 0.0;
  const Weights wt = {inv_cap, c.steep, c.top, c.z_max};
  const uint32_t key = order_key(z);
  const double x = wt.weight(z);
  const bool stays = key != 0 && (key > c.key_cut || (key == c.key_cut && i <= c.idx_cut)) && x >= c.min_p && fixed(x) > 0;
  return stays ? x * double(1ull << kFracBits) / double(c.whole) : 0.0;
}

// 4: one workgroup per row.
__global__ __launch_bounds__(kSampleThreads) void verify_rows_kernel(VerifyArgs a, RowWork* ws) {
  __shared__ Shared sh;
  __shared__ u64 sums[kGroups];
  __shared__ uint2 small[kGroupThreads];
  __shared__ u64 small_w[kGroupThreads];
  __shared__ int last;
  const GroupPlan gp = group_plan(a.vocab);
  Q4_DCHECK(gp.groups <= kGroups && int(gridDim.x) <= 2 * a.n_rows, kDbgVerifyGrid);
  const int r = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int seq = a.seq_of[r];
  if (seq < 0) return;
  RowWork& w = ws[r];
  const uint2 first = w.list[t >> 2];
  const uint32_t listed = w.list_n;
  const Filters f = filters_of(a, r);
  const uint32_t n = f.borders() ? listed : 0;
  const RowInfo in = row_info(a.vocab, w, f, f.by_list() && n > kList);
  const float* z = row_at(a, r);
  RowCut c = {in.wt.steep, in.wt.top, f.min_p, 0, 0.0, in.wt.z_max, 0, -1, in.max_key == 0 ? 0 : in.plain ? 1 : 2};
  if (in.plain) {
    if (wave == 0 && in.max_key != 0)
      for (int i = lane; i < (gp.groups + 63) / 64 * 64; i += 64) {
        const u64 hit = __ballot(i < gp.groups && w.group_key[min(i, gp.groups - 1)] == in.max_key);
        if (hit) {
          c.idx_cut = w.group_idx[i - lane + int(__ffsll(hit)) - 1];
          break;
        }
      }
  } else {
    if (t < kGroups) sums[t] = t < gp.groups && !f.by_list() ? w.group_sum[t] : 0;
    if (f.by_list() && n <= kGroupThreads) {
      // four neighbouring threads a token, each compares it with a quarter
      const int at = t >> 2, part = t & 3;
      const uint2 me = at < int(n) ? first : make_uint2(0u, 0u);
      double x = 0.0;
      u64 own = 0;
      if (at < int(n)) {
        x = in.wt.weight(key_value(me.x));
        own = fixed(x);
        if (part == 0) {
          small[at] = me;
          small_w[at] = own;
        }
      }
      if (t == 0) last = 0;
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
      const bool stays = in_k && !(f.top_p < 1.0f && better >= top_p_target(f.top_p, whole));
      if (stays && part == 0) {
        atomicMax(&last, rank);
        if (x >= f.min_p) atomicAdd(&sums[int(me.y) / gp.per], own);
      }
      __syncthreads();
      if (stays && part == 0 && rank == last) sh.digit = me.x, sh.rest = me.y;
      __syncthreads();
      c.key_cut = sh.digit, c.idx_cut = int(sh.rest);
    } else {
      cut_row(sh, sums, f, in, w, z, a.vocab, n, c.key_cut, c.idx_cut);
      __syncthreads();
    }
    if (t < gp.groups) w.group_sum[t] = sums[t];
    if (t < 64) {
      u64 own = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) own += sums[4 * t + i];
      c.whole = wave_sum(own);
    }
  }
  if (t == 0) {
    const int row = r < a.n_rows ? r : r - a.n_rows, x = a.drafts[row];
    const bool there = x >= 0 && x < a.vocab;
    c.draft_share = there ? share_in(c, f.inv_cap, z[there ? x : 0], x) : 0.0;
    a.cuts[r] = c;
  }
}

__device__ __forceinline__ double unit(float u) { return u > 0.0f ? fmin(double(u), 1.0) : 0.0; }

// Sequence b's first row whose draft does not stay, from its first row on (its
// last row where all stay). By each wave for itself.
__device__ __forceinline__ int stop_of(const VerifyArgs& a, int b, int start, int n) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < n - 1; base += 64) {
    const int i = base + lane, r = start + min(i, n - 2);
    const bool known = a.seq_of[r] == b;
    const double p = known ? a.cuts[r].draft_share : 0.0;
    const double q = !a.draft_logits ? 1.0 : a.seq_of[a.n_rows + r] == b ? a.cuts[a.n_rows + r].draft_share : 0.0;
    const u64 out = __ballot(i < n - 1 && !(unit(a.u[r]) * q < p));
    if (out) return base + int(__ffsll(out)) - 1;
  }
  return n - 1;
}

// max(0, p - q) of tokens with logits zp and zq, in 2^-60
template <int N>
__device__ __forceinline__ void rest_of(const RowCut& p, const RowCut& q, double p_inv_cap, double q_inv_cap, const float (&zp)[N],
                                        const float (&zq)[N], const int (&idx)[N], u64 (&out)[N]) {
  auto shares = [&](const RowCut& c, double inv_cap, const float (&z)[N], double (&x)[N]) {
    if (c.kind != 2) {
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = c.kind == 1 && idx[j] == c.idx_cut ? 1.0 : 0.0;
      return;
    }
    const Weights wt = {inv_cap, c.steep, c.top, c.z_max};
    const double scale = double(1ull << kFracBits) / double(c.whole);
    wt.weights(z, x);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t key = order_key(z[j]);
      const bool stays = key != 0 && (key > c.key_cut || (key == c.key_cut && idx[j] <= c.idx_cut)) && x[j] >= c.min_p && fixed(x[j]) > 0;
      x[j] = stays ? x[j] * scale : 0.0;
    }
  };
  double x[N], y[N];
  shares(p, p_inv_cap, zp, x);
  shares(q, q_inv_cap, zq, y);
#pragma unroll
  for (int j = 0; j < N; ++j) out[j] = x[j] > y[j] ? u64(rint((x[j] - y[j]) * 0x1p60)) : 0;
}

// 5: one wave per group of the row that each sequence stops at.
__global__ __launch_bounds__(kGroupThreads) void verify_rest_kernel(VerifyArgs a, RowWork* ws) {
  const GroupPlan gp = group_plan(a.vocab);
  Q4_DCHECK(int64_t(gridDim.x) * kGroupWaves >= gp.groups && gp.groups <= kGroups, kDbgVerifyGrid);
  const int b = blockIdx.y, lane = threadIdx.x & 63, group = blockIdx.x * kGroupWaves + int(threadIdx.x >> 6);
  int start, n;
  if (!rows_of(a, b, start, n) || n == 0 || group >= gp.groups) return;
  const int stop = stop_of(a, b, start, n), r = start + stop;
  if (stop == n - 1 || a.seq_of[r] != b || a.seq_of[a.n_rows + r] != b) return;
  const RowCut p = a.cuts[r], q = a.cuts[a.n_rows + r];
  if (p.kind != 2) return;
  u64 sum = 0;
  if (ws[r].group_sum[group] > 0) {
    const float* zp = row_at(a, r);
    const float* zq = row_at(a, a.n_rows + r);
    const int lo = group * gp.per, hi = min(lo + gp.per, a.vocab);
    for (int base = lo + lane; base - lane < hi; base += 64 * kSide) {
      float vp[kSide], vq[kSide];
      int idx[kSide];
      bool any = false;
#pragma unroll
      for (int j = 0; j < kSide; ++j) {
        idx[j] = base + 64 * j;
        vp[j] = idx[j] < hi ? zp[idx[j]] : -INFINITY;
        vq[j] = idx[j] < hi ? zq[idx[j]] : -INFINITY;
        any = any || order_key(vp[j]) >= p.key_cut;
      }
      if (__ballot(any) == 0) continue;
      u64 x[kSide];
      rest_of(p, q, a.inv_cap, a.draft_inv_cap, vp, vq, idx, x);
#pragma unroll
      for (int j = 0; j < kSide; ++j) sum += x[j];
    }
  }
  sum = wave_sum(sum);
  if (lane == 0) a.rest[size_t(b) * kGroups + group] = sum;
}

// 6: one workgroup per sequence.
__global__ __launch_bounds__(kSampleThreads) void verify_draw_kernel(VerifyArgs a, RowWork* ws) {
  __shared__ u64 part[kSampleWaves];
  __shared__ u64 shared_rest;
  __shared__ int chosen;
  const GroupPlan gp = group_plan(a.vocab);
  const int b = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int start, n;
  if (!rows_of(a, b, start, n)) {
    if (a.err && t == 0) *a.err = 1;
    return;
  }
  const int stop = n > 0 ? stop_of(a, b, start, n) : -1;
  if (t == 0) a.count[b] = stop + 1;
  if (n == 0) return;
  for (int i = t; i < n; i += kSampleThreads) {
    const int x = a.drafts[start + i];
    if (i < n - 1 && (x < 0 || x >= a.vocab) && a.err) *a.err = 1;
    if (i == stop) continue;
    a.tokens[start + i] = i < stop ? x : -1;
    if (a.prob) a.prob[start + i] = i < stop ? float(a.cuts[start + i].draft_share) : 0.0f;
  }
  const int r = start + stop;
  RowCut p = a.cuts[r];
  if (a.seq_of[r] != b) p.kind = 0;
  if (p.kind != 2) {
    if (t == 0) {
      a.tokens[r] = p.kind == 1 ? p.idx_cut : -1;
      if (a.prob) a.prob[r] = p.kind == 1 ? 1.0f : NAN;
    }
    return;
  }
  const float* zp = row_at(a, r);
  const Weights wt = {a.inv_cap, p.steep, p.top, p.z_max};
  auto stays = [&](float z, int i, double x) {
    const uint32_t key = order_key(z);
    return key != 0 && (key > p.key_cut || (key == p.key_cut && i <= p.idx_cut)) && x >= p.min_p;
  };
  // what is taken off: the drafter's whole distribution (`both`), or all of the draft
  const bool back = stop < n - 1;
  const bool both = back && a.draft_logits && a.seq_of[a.n_rows + r] == b;
  const int x_draft = a.drafts[r];
  int without = back && !a.draft_logits && x_draft >= 0 && x_draft < a.vocab ? x_draft : -1;
  u64 off = 0;  // its weight
  if (without >= 0) {
    const double x = wt.weight(zp[without]);
    off = stays(zp[without], without, x) ? fixed(x) : 0;
  }
  bool rests = false;
  // the group that the drawn number falls in, by the first wave: of max(0, p - q), or where that is nothing, of p
  if (t < 64) {
    u64 c[4], upto = 0, whole = 0, own = 0;
    for (int pass = both || without >= 0 ? 0 : 1; pass < 2; ++pass) {
      own = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = 4 * t + i;
        c[i] = g >= gp.groups ? 0 : both && pass == 0 ? a.rest[size_t(b) * kGroups + g] : ws[r].group_sum[g];
        if (pass == 0 && without >= 0 && without / gp.per == g) c[i] -= off;
        own += c[i];
      }
      upto = wave_upto(own), whole = lane_value(upto, 63);
      if (whole > 0) {
        rests = pass == 0;
        break;
      }
    }
    const u64 target = drawn_at(a.u_draw[b], whole);
    u64 before = upto - own;
    if (t == 0) chosen = rests ? -2 : -1;  // (nothing at all: not reached, the first-ranked token stays)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (before <= target && target < before + c[i]) {
        chosen = (4 * t + i) << 1 | int(rests);
        shared_rest = target - before;
      }
      before += c[i];
    }
  }
  __syncthreads();
  if (chosen < 0) return;
  rests = chosen & 1;
  u64 target = shared_rest;
  const int group = chosen >> 1, lo = group * gp.per, hi = min(lo + gp.per, a.vocab);
  const RowCut q = both ? a.cuts[a.n_rows + r] : p;
  const float* zq = both ? row_at(a, a.n_rows + r) : zp;
  if (!rests) without = -1;
  for (int base = lo; base < hi; base += kSampleThreads) {
    const int i = base + t;
    u64 own = 0;
    double x = 0.0;
    if (i < hi) {
      const float z = zp[i];
      x = wt.weight(z);
      if (rests && both) {
        const float vp[1] = {z}, vq[1] = {zq[i]};
        const int idx[1] = {i};
        u64 y[1];
        rest_of(p, q, a.inv_cap, a.draft_inv_cap, vp, vq, idx, y);
        own = y[0];
      } else {
        own = stays(z, i, x) && i != without ? fixed(x) : 0;
      }
    }
    const u64 upto = wave_upto(own);
    __syncthreads();
    if (lane == 63) part[wave] = upto;
    __syncthreads();
    u64 before = upto - own, all = 0;
    for (int v = 0; v < kSampleWaves; ++v) {
      if (v < wave) before += part[v];
      all += part[v];
    }
    if (before <= target && target < before + own) {
      a.tokens[r] = i;
      if (a.prob) a.prob[r] = share_of(x, p.whole);
    }
    if (target < all) return;
    target -= all;
  }
}

struct VerifyPlan {
  int64_t rows;  // with the drafter's
  size_t work, cuts, rest, seq_of;
};
static VerifyPlan verify_plan(int64_t n_rows, int64_t n_seq, bool drafter) {
  VerifyPlan p;
  p.rows = drafter ? 2 * n_rows : n_rows;
  p.work = align256(size_t(p.rows) * sizeof(RowWork));
  p.cuts = align256(size_t(p.rows) * sizeof(RowCut));
  p.rest = drafter ? align256(size_t(n_seq) * kGroups * sizeof(u64)) : 0;
  p.seq_of = align256(size_t(p.rows) * sizeof(int32_t));
  return p;
}

}  // namespace q4dec

extern "C" size_t verify_drafts_workspace_bytes(int64_t n_rows, int64_t n_seq, int64_t vocab, int32_t has_draft_logits) {
  using namespace q4dec;
  if (n_rows <= 0 || n_rows > kMaxVerifyRows || n_seq <= 0 || n_seq > kMaxVerifyRows || vocab <= 0 ||
      vocab > (int64_t(1) << 20))
    return 0;
  const VerifyPlan p = verify_plan(n_rows, n_seq, has_draft_logits != 0);
  return p.work + p.cuts + p.rest + p.seq_of;
}

extern "C" int verify_drafts(const float* logits, int64_t n_rows, int64_t vocab, int64_t row_stride, float cap,
                             const float* draft_logits, int64_t draft_stride, float draft_cap, const int32_t* drafts,
                             const int32_t* starts, int64_t n_seq, const float* temperature, const int32_t* top_k,
                             const float* top_p, const float* min_p, const float* u, const float* u_draw, void* ws,
                             size_t ws_bytes, int32_t* tokens_out, float* prob_out, int32_t* count_out, int32_t* err_flag,
                             void* stream) {
  using namespace q4dec;
  const char* name = "verify_drafts";
  if (n_rows < 0 || n_rows > kMaxVerifyRows)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_rows must be in [0, 32767] (got %lld)", name, (long long)n_rows);
  if (n_seq < 0 || n_seq > kMaxVerifyRows)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_seq must be in [0, 32767] (got %lld)", name, (long long)n_seq);
  if (vocab <= 0 || vocab > (int64_t(1) << 20))
    return fail(Q4DEC_ERR_SHAPE, "%s: vocab must be in [1, 2^20] (got %lld)", name, (long long)vocab);
  if (row_stride < vocab)
    return fail(Q4DEC_ERR_SHAPE, "%s: row_stride must be at least vocab (got %lld)", name, (long long)row_stride);
  if (draft_logits && draft_stride < vocab)
    return fail(Q4DEC_ERR_SHAPE, "%s: draft_stride must be at least vocab (got %lld)", name, (long long)draft_stride);
  if (n_rows == 0 || n_seq == 0) return Q4DEC_OK;
  if (!logits) return fail(Q4DEC_ERR_NULL, "%s: logits is NULL", name);
  if (!drafts) return fail(Q4DEC_ERR_NULL, "%s: drafts is NULL", name);
  if (!starts) return fail(Q4DEC_ERR_NULL, "%s: starts is NULL", name);
  if (!u) return fail(Q4DEC_ERR_NULL, "%s: u is NULL", name);
  if (!u_draw) return fail(Q4DEC_ERR_NULL, "%s: u_draw is NULL", name);
  if (!tokens_out) return fail(Q4DEC_ERR_NULL, "%s: tokens_out is NULL", name);
  if (!count_out) return fail(Q4DEC_ERR_NULL, "%s: count_out is NULL", name);
  for (const void* x : {(const void*)logits, (const void*)draft_logits, (const void*)drafts, (const void*)starts,
                        (const void*)temperature, (const void*)top_k, (const void*)top_p, (const void*)min_p, (const void*)u,
                        (const void*)u_draw, (const void*)tokens_out, (const void*)prob_out, (const void*)count_out,
                        (const void*)err_flag})
    if (!aligned(x, 4)) return fail(Q4DEC_ERR_ALIGN, "%s: inputs and outputs must be 4-byte aligned", name);
  const size_t need = verify_drafts_workspace_bytes(n_rows, n_seq, vocab, draft_logits ? 1 : 0);
  if (need > 0 && !ws) return fail(Q4DEC_ERR_NULL, "%s: ws is NULL", name);
  if (ws_bytes < need)
    return fail(Q4DEC_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws_bytes, need);
  if (!aligned(ws, 256)) return fail(Q4DEC_ERR_ALIGN, "%s: ws must be 256-byte aligned", name);
  const VerifyPlan p = verify_plan(n_rows, n_seq, draft_logits != nullptr);
  FirstArgs a;
  a.logits = logits, a.draft_logits = draft_logits, a.row_stride = row_stride, a.draft_stride = draft_stride;
  a.vocab = int(vocab), a.n_rows = int(n_rows), a.n_seq = int(n_seq);
  a.cap = double(cap), a.inv_cap = cap > 0.0f ? 1.0 / double(cap) : 0.0;
  a.draft_cap = double(draft_cap), a.draft_inv_cap = draft_cap > 0.0f ? 1.0 / double(draft_cap) : 0.0;
  a.drafts = drafts, a.starts = starts, a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p;
  a.u = u, a.u_draw = u_draw, a.tokens = tokens_out, a.prob = prob_out, a.count = count_out, a.err = err_flag;
  uint8_t* at = static_cast<uint8_t*>(ws);
  RowWork* work = reinterpret_cast<RowWork*>(at);
  a.cuts = reinterpret_cast<RowCut*>(at + p.work);
  a.rest = reinterpret_cast<u64*>(at + p.work + p.cuts);
  a.seq_of = reinterpret_cast<int32_t*>(at + p.work + p.cuts + p.rest);
  const VerifyArgs& v = a;
  const GroupPlan gp = group_plan(a.vocab);
  const unsigned across = unsigned((gp.groups + kGroupWaves - 1) / kGroupWaves);
  const dim3 grid(across, unsigned(p.rows));
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(sample_groups_kernel<FirstArgs>, grid, dim3(kGroupThreads), 0, st, a, work);
  hipLaunchKernelGGL(sample_bins_kernel<VerifyArgs>, grid, dim3(kGroupThreads), 0, st, v, work);
  hipLaunchKernelGGL(sample_sums_kernel<VerifyArgs>, grid, dim3(kGroupThreads), 0, st, v, work);
  hipLaunchKernelGGL(verify_rows_kernel, dim3(unsigned(p.rows)), dim3(kSampleThreads), 0, st, v, work);
  if (draft_logits)
    hipLaunchKernelGGL(verify_rest_kernel, dim3(across, unsigned(n_seq)), dim3(kGroupThreads), 0, st, v, work);
  hipLaunchKernelGGL(verify_draw_kernel, dim3(unsigned(n_seq)), dim3(kSampleThreads), 0, st, v, work);
  return launch_status(name);
}
