// verify_drafts: draft x of a row stays if u q(x) < p(x); at the first that
// does not, a token is drawn from max(0, p - q), else from the last row's p.
// p and q are the distributions of sample_logits; each row of the target and
// the drafter ends up as a cut in its ranking and sums of what stays.
//  1. a wave a group of V / 256 logits: its largest, and in a call without
//     filters the sum of its weights relative to it, so that a row is read once
//     (before it, where there are more than 64 sequences, each row's sequence);
//  2. and 3. in a call with filters sample_logits' list or histogram, and sums
//     (sample_kernels.h);
//  4. a workgroup a row finds the row's cut and the probability of its draft;
//  5. where a sequence stops at a draft that is taken back, the sums of
//     max(0, p - q) over each group of that row's tokens, in 60-bit fixed
//     point (integers: their order does not matter). Groups in which p has
//     nothing are left out: under a small top_k that is nearly all of them;
//  6. a workgroup a sequence draws: the group by the sums, then in the group.
// Measured: one sequence of 4 drafts, top-k 64 and top-p, 28 us (a chain of six
// launches); 24 of up to 4 with mixed filters 157 us, of which the histograms take
// 62 and the sums 36 as in sample_logits; 64 of 3 without filters 228 us: 470 MB in
// 194 us (2.4 TB/s; the reading alone takes 87), then max(0, p - q) of 64 pairs of
// rows in 44. The vector units are busy 72% of the 194: 638 instructions a wave for
// 16 logits a lane, of which the weights are about 26 a logit and the rest finds the
// group's largest and its tanh; at 262144 logits that is one chain of loads, maximum
// and weights a wave, with nothing after it to run beside its waits.
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
  bool open;  // without filters
  int32_t* seq_of;  // of each row (the drafter's from n_rows on); -1: not used
  GroupPlan gp;
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

// In a call without filters every token that may be drawn stays, but for greedy
// rows. (Of calls with filters the rows without them are left to the sums' launch:
// with both ways in the first launch's code it has registers for half as many
// waves, 24 sequences of up to 5 rows with mixed filters 29 us and 23.)
__device__ __forceinline__ bool open_row(const VerifyArgs& a, const Filters& f) { return a.open && f.heat > 0.0f; }
__device__ __forceinline__ bool sums_known(const VerifyArgs& a, const Filters& f) { return open_row(a, f); }

// The sequence of each row: the first that has it, -1 if none has or, of the
// drafter's rows, it is the last of one. No search by the order of the starts: a
// bad one among them is to spoil no sequence but those that it bounds. Up to 64
// sequences each wave of the first launch asks them all at once; more are asked
// by a launch before it, a workgroup for 1024 rows (65 sequences of 2 rows of 2000
// take 1.2 us longer by that; 10000 of 1000, where a search in each workgroup of
// the first launch took 782 us in all, 741).
constexpr int kAskedAtOnce = 64;
__device__ __forceinline__ int sequence_at(const VerifyArgs& a, int r) {
  if (a.n_seq > kAskedAtOnce) return a.seq_of[r];
  const int b = threadIdx.x & 63, row = r < a.n_rows ? r : r - a.n_rows;
  int start = 0, n = 0;
  const bool in = b < a.n_seq && rows_of(a, b, start, n) && row >= start && row - start < n;
  const u64 who = __ballot(in);
  const u64 last = __ballot(row - start == n - 1);
  if (who == 0) return -1;
  const int first = int(__ffsll(who)) - 1;
  return r >= a.n_rows && (last >> first & 1) ? -1 : first;
}
constexpr int kOwnThreads = 1024;
__global__ __launch_bounds__(kOwnThreads) void verify_sequences_kernel(VerifyArgs a, int rows) {
  __shared__ int own[kOwnThreads];
  const int t = threadIdx.x, from = blockIdx.x * kOwnThreads, upto = min(from + kOwnThreads, a.n_rows), row = from + t;
  own[t] = 0x7FFFFFFF;
  __syncthreads();
  for (int b = t; b < a.n_seq; b += kOwnThreads) {
    int start, n;
    if (!rows_of(a, b, start, n)) continue;
    for (int i = max(start, from); i < min(start + n, upto); ++i) atomicMin(&own[i - from], b);
  }
  __syncthreads();
  if (row >= upto) return;
  const int b = own[t] == 0x7FFFFFFF ? -1 : own[t];
  a.seq_of[row] = b;
  if (rows > a.n_rows) a.seq_of[a.n_rows + row] = b < 0 || a.starts[b + 1] - 1 == row ? -1 : b;
}

// Weights::weights to 2^-33 of their value, for sums over all of a row (so near
// that a drawn number of 24 bits hardly ever falls between the two). Such a
// launch is bound by its vector instructions, so there are as few as can be:
//  - a logit goes to octaves, steep * (tanh(z / cap) - top), without the tanh
//    for itself: z * (steep / cap) times the polynomial in (z / cap)^2 that
//    tanh_abs has, less a constant. It is off by 2^-44.6 of the octaves from 0,
//    so of a weight by up to ln 2 * 2048 * 2^-44.6 = 2^-34.1, and the constant's
//    rounding by 2^-42;
//  - 2^y by the polynomial through 8 nodes, 2^-34.1 of it; y is rounded by
//    adding 1.5 * 2^52, whose low bits then hold the whole number for the exponent.
// That is for logits within 0.45 of the cap, and where the constant is less than
// 2048 octaves; others have Weights::weights. Which goes by the token alone, so
// that every launch has the same bits for it. 0 for tokens that are never drawn.
struct Quick {
  Weights wt;
  double slope, shift;
  bool on;
  __device__ __forceinline__ explicit Quick(const Weights& w)
      : wt(w), slope(w.inv_cap > 0.0 ? w.inv_cap * w.steep : w.steep), shift(-w.steep * w.top), on(fabs(shift) < 2048.0) {}
  // (far: the tokens whose weights are not what `out` says)
  template <bool CAPPED, int N>
  __device__ __forceinline__ bool weigh(const float (&z)[N], double (&out)[N], bool (&far)[N]) const {
    constexpr double kTanh[] = {-0.0010586183492814069, 0.003469517587012053, -0.008842871160416817, 0.021867589319773756,
                                -0.05396815710836195,   0.13333333089707022,  -0.3333333333099173,   0.999999999999963};
    constexpr double kExp[] = {1.5303700711365693e-05, 0.00015469729214118296, 0.0013333478473685416, 0.009618025613318034,
                               0.055504109063258665,   0.24022651213498092,    0.6931471805568324,    0.9999999999595618};
    double y[N], p[N], n[N];
    bool any = !on;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const double x = double(z[j]);
      y[j] = x * slope;
      n[j] = CAPPED ? x * wt.inv_cap : x;
      far[j] = !(fabs(n[j]) <= (CAPPED ? 0.45 : 3.5e38));
      any = any || far[j];
      p[j] = CAPPED ? kTanh[0] : 1.0;
    }
    if constexpr (CAPPED) {
#pragma unroll
      for (int j = 0; j < N; ++j) n[j] = n[j] * n[j];
#pragma unroll
      for (int i = 1; i < int(sizeof(kTanh) / sizeof(double)); ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = fma(p[j], n[j], kTanh[i]);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      y[j] = fmax(fma(y[j], p[j], shift), -64.0);
      n[j] = y[j] + 0x1.8p52;
      y[j] = y[j] - (n[j] - 0x1.8p52);
      p[j] = kExp[0];
    }
#pragma unroll
    for (int i = 1; i < int(sizeof(kExp) / sizeof(double)); ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) p[j] = fma(p[j], y[j], kExp[i]);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      u32x2 b = __builtin_bit_cast(u32x2, p[j]);
      b.y += __builtin_bit_cast(u32x2, n[j]).x << 20;
      out[j] = __builtin_bit_cast(double, b);
    }
    return any;
  }
  template <int N>
  __device__ __forceinline__ void weights(const float (&z)[N], double (&out)[N]) const {
    bool far[N];
    bool any = wt.inv_cap > 0.0 ? weigh<true>(z, out, far) : weigh<false>(z, out, far);
    if (__ballot(any) == 0) return;
    any = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      far[j] = (far[j] || !on) && z[j] > -INFINITY;
      any = any || far[j];
      out[j] = z[j] > -INFINITY ? out[j] : 0.0;
    }
    if (__ballot(any) == 0) return;
    double x[N];
    wt.weights(z, x);
#pragma unroll
    for (int j = 0; j < N; ++j) out[j] = far[j] ? x[j] : out[j];
  }
};
// the sum over the lanes, in the last one
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
  return __builtin_bit_cast(double, moved<CTRL, ROWS>(__builtin_bit_cast(u64, v)));
}
__device__ __forceinline__ double sum_in_last(double v) {
  v += moved<0x111, 0xF>(v);
  v += moved<0x112, 0xF>(v);
  v += moved<0x114, 0xF>(v);
  v += moved<0x118, 0xF>(v);
  v += moved<0x142, 0xA>(v);
  v += moved<0x143, 0xC>(v);
  return v;
}

// 1: one wave per group.
__global__ __launch_bounds__(kGroupThreads) void verify_extremes_kernel(VerifyArgs a, RowWork* ws) {
  Q4_DCHECK(int64_t(gridDim.x) * kGroupWaves >= a.gp.groups && a.gp.groups <= kGroups, kDbgVerifyGrid);
  const int r = blockIdx.y, b = sequence_at(a, r);
  if (a.n_seq <= kAskedAtOnce && blockIdx.x == 0 && threadIdx.x == 0) a.seq_of[r] = b;
  if (b >= 0) group_extremes(ws[r], row_at(a, r), a.vocab);
}
// The same without filters, with the sums. (Registers for four waves; with fewer
// for more the products spill: 229 us become 305.)
__global__ __launch_bounds__(kGroupThreads, 4) void verify_groups_kernel(VerifyArgs a, RowWork* ws) {
  __shared__ int row_seq;
  __shared__ bool row_open;
  __shared__ double row_steep;
  Q4_DCHECK(int64_t(gridDim.x) * kGroupWaves >= a.gp.groups && a.gp.groups <= kGroups, kDbgVerifyGrid);
  const int r = blockIdx.y, lane = threadIdx.x & 63, group = blockIdx.x * kGroupWaves + int(threadIdx.x >> 6);
  const bool target = r < a.n_rows;
  const double inv_cap = target ? a.inv_cap : a.draft_inv_cap;
  if (threadIdx.x < 64) {  // what is the row's, by one wave
    const int b = sequence_at(a, r);
    if (b >= 0) {
      const Filters f = filters_at(a, b, target ? a.cap : a.draft_cap, inv_cap);
      row_open = open_row(a, f);
      row_steep = steep_of(f);
    }
    row_seq = b;
    if (a.n_seq <= kAskedAtOnce && blockIdx.x == 0 && threadIdx.x == 0) a.seq_of[r] = b;
  }
  __syncthreads();
  if (row_seq < 0) return;
  const float* z = row_at(a, r);
  RowWork& w = ws[r];
  if (!row_open) {
    group_extremes(w, z, a.vocab);
    return;
  }
  if (group >= a.gp.groups) return;
  const int lo = group * a.gp.per, hi = min(lo + a.gp.per, a.vocab);
  uint32_t best = 0;
  double sum = 0.0;  // of this lane, relative to `best`
  for (int base = lo; base < hi; base += 16 * 64) {
    float v[16 / kSide][kSide], top = -INFINITY;
    const float* from = z + base + lane;
    if (base + 16 * 64 <= hi) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e / kSide][e % kSide] = from[64 * e];
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e / kSide][e % kSide] = base + lane + 64 * e < hi ? from[64 * e] : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, v[e / kSide][e % kSide]);  // (leaves a NaN out)
    const uint32_t key = wave_max(order_key(top));
    if (key == 0) continue;
    const uint32_t was = best;
    best = max(best, key);
    const Quick quick(weights_of(row_steep, inv_cap, best));
    if (was != 0 && best != was) sum *= quick.wt.weight(key_value(was));
#pragma unroll
    for (int e = 0; e < 16 / kSide; ++e) {
      if (base + 64 * kSide * e >= hi) break;
      double x[kSide];
      quick.weights(v[e], x);
#pragma unroll
      for (int j = 0; j < kSide; ++j) sum += x[j];
    }
  }
  sum = sum_in_last(sum);
  if (lane == 63) {
    w.group_key[group] = best;
    w.weight[group] = __builtin_bit_cast(u64, sum);
  }
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
  const GroupPlan gp = a.gp;
  Q4_DCHECK(gp.groups <= kGroups && int(gridDim.x) <= 2 * a.n_rows, kDbgVerifyGrid);
  const int r = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int seq = a.seq_of[r];
  if (seq < 0) return;
  RowWork& w = ws[r];
  const uint2 first = w.list[t >> 2];
  const uint32_t listed = w.list_n;
  const Filters f = filters_of(a, r);
  const bool open = open_row(a, f);
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
    if (t < kGroups) sums[t] = t < gp.groups && !f.by_list() && !open ? w.group_sum[t] : 0;
    if (open) {
      // (a group whose heaviest token rounds to nothing has none that may be drawn)
      const double x = t < gp.groups && w.group_key[t] != 0 ? in.wt.weight(key_value(w.group_key[t])) : 0.0;
      if (fixed(x) > 0) sums[t] = max(u64(rint(__builtin_bit_cast(double, w.weight[t]) * x * double(1ull << kFracBits))), u64(1));
      c.key_cut = 1, c.idx_cut = 0x7FFFFFFF;
      __syncthreads();
    } else if (f.by_list() && n <= kGroupThreads) {
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

// (below 1, so that equal probabilities always stay)
__device__ __forceinline__ double unit(float u) { return u > 0.0f ? double(fminf(u, 0x1.fffffep-1f)) : 0.0; }

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

// max(0, p - q) of tokens with logits zp and zq, in 2^-60.
struct RestOf {
  RowCut p, q;
  Quick p_quick, q_quick;
  double p_scale, q_scale;
  __device__ __forceinline__ RestOf(const RowCut& p, const RowCut& q, double p_inv_cap, double q_inv_cap)
      : p(p),
        q(q),
        p_quick(Weights{p_inv_cap, p.steep, p.top, p.z_max}),
        q_quick(Weights{q_inv_cap, q.steep, q.top, q.z_max}),
        p_scale(double(1ull << kFracBits) / double(p.whole)),
        q_scale(double(1ull << kFracBits) / double(q.whole)) {}
  template <int N>
  static __device__ __forceinline__ void shares(const RowCut& c, const Quick& quick, double scale, const float (&z)[N],
                                                const int (&idx)[N], double (&x)[N]) {
    if (c.kind != 2) {
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = c.kind == 1 && idx[j] == c.idx_cut ? 1.0 : 0.0;
      return;
    }
    if (c.key_cut == 1 && c.min_p == 0.0) {  // nothing filtered
      quick.weights(z, x);
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = x[j] > 0x1p-43 ? x[j] * scale : 0.0;
      return;
    }
    quick.wt.weights(z, x);  // (which min_p is compared with)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t key = order_key(z[j]);
      const bool stays = key != 0 && (key > c.key_cut || (key == c.key_cut && idx[j] <= c.idx_cut)) && x[j] >= c.min_p && x[j] > 0x1p-43;
      x[j] = stays ? x[j] * scale : 0.0;
    }
  }
  template <int N>
  __device__ __forceinline__ void operator()(const float (&zp)[N], const float (&zq)[N], const int (&idx)[N], u64 (&out)[N]) const {
    double x[N], y[N];
    shares(p, p_quick, p_scale, zp, idx, x);
    shares(q, q_quick, q_scale, zq, idx, y);
#pragma unroll
    for (int j = 0; j < N; ++j) out[j] = x[j] > y[j] ? u64(rint((x[j] - y[j]) * 0x1p60)) : 0;
  }
};

// 5: one wave per group of the row that each sequence stops at.
__global__ __launch_bounds__(kGroupThreads) void verify_rest_kernel(VerifyArgs a, RowWork* ws) {
  const GroupPlan gp = a.gp;
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
    const RestOf rest(p, q, a.inv_cap, a.draft_inv_cap);
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
      rest(vp, vq, idx, x);
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
  const GroupPlan gp = a.gp;
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
  auto own_of = [&](float z, int i) {
    const double x = wt.weight(z);
    return stays(z, i, x) ? fixed(x) : 0;
  };
  // The weight of its group without it: counted, since a sum less a weight that
  // is nearly all of it is mostly their roundings.
  u64 others = 0;
  if (without >= 0) {
    const int lo = without / gp.per * gp.per, hi = min(lo + gp.per, a.vocab);
    for (int i = lo + t; i < hi; i += kSampleThreads) others += i != without ? own_of(zp[i], i) : 0;
    others = wave_sum(others);
    if (lane == 0) part[wave] = others;
    __syncthreads();
    others = 0;
    for (int v = 0; v < kSampleWaves; ++v) others += part[v];
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
        if (pass == 0 && without >= 0 && without / gp.per == g) c[i] = others;
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
  const RestOf rest(p, both ? a.cuts[a.n_rows + r] : p, a.inv_cap, a.draft_inv_cap);
  const float* zq = both ? row_at(a, a.n_rows + r) : zp;
  if (!rests) without = -1;
  int end = -1;  // this thread's last token that may be drawn
  float end_z = 0.0f;
  for (int base = lo; base < hi; base += kSampleThreads) {
    const int i = base + t;
    u64 own = 0;
    float z = -INFINITY;
    if (i < hi) {
      z = zp[i];
      if (rests && both) {
        const float vp[1] = {z}, vq[1] = {zq[i]};
        const int idx[1] = {i};
        u64 y[1];
        rest(vp, vq, idx, y);
        own = y[0];
      } else {
        own = i != without ? own_of(z, i) : 0;
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
      if (a.prob) a.prob[r] = share_of(wt.weight(z), p.whole);
    }
    if (own > 0) end = i, end_z = z;
    if (target < all) return;
    target -= all;
  }
  // A group's sum is not always its tokens' to the last bit: the number fell
  // behind the last of them.
  if (t == 0) chosen = -1;
  __syncthreads();
  if (end >= 0) atomicMax(&chosen, end);
  __syncthreads();
  if (end >= 0 && end == chosen) {
    a.tokens[r] = end;
    if (a.prob) a.prob[r] = share_of(wt.weight(end_z), p.whole);
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
  VerifyArgs a;
  a.logits = logits, a.draft_logits = draft_logits, a.row_stride = row_stride, a.draft_stride = draft_stride;
  a.vocab = int(vocab), a.n_rows = int(n_rows), a.n_seq = int(n_seq);
  a.cap = double(cap), a.inv_cap = cap > 0.0f ? 1.0 / double(cap) : 0.0;
  a.draft_cap = double(draft_cap), a.draft_inv_cap = draft_cap > 0.0f ? 1.0 / double(draft_cap) : 0.0;
  a.drafts = drafts, a.starts = starts, a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p;
  a.u = u, a.u_draw = u_draw, a.tokens = tokens_out, a.prob = prob_out, a.count = count_out, a.err = err_flag;
  a.open = !top_k && !top_p && !min_p;
  uint8_t* at = static_cast<uint8_t*>(ws);
  RowWork* work = reinterpret_cast<RowWork*>(at);
  a.cuts = reinterpret_cast<RowCut*>(at + p.work);
  a.rest = reinterpret_cast<u64*>(at + p.work + p.cuts);
  a.seq_of = reinterpret_cast<int32_t*>(at + p.work + p.cuts + p.rest);
  const GroupPlan gp = a.gp = group_plan(a.vocab);
  const unsigned across = unsigned((gp.groups + kGroupWaves - 1) / kGroupWaves);
  const dim3 grid(across, unsigned(p.rows));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (n_seq > kAskedAtOnce)
    hipLaunchKernelGGL(verify_sequences_kernel, dim3(unsigned((n_rows + kOwnThreads - 1) / kOwnThreads)), dim3(kOwnThreads), 0, st,
                       a, int(p.rows));
  hipLaunchKernelGGL(a.open ? verify_groups_kernel : verify_extremes_kernel, grid, dim3(kGroupThreads), 0, st, a, work);
  if (top_k || top_p) hipLaunchKernelGGL(sample_bins_kernel<VerifyArgs>, grid, dim3(kGroupThreads), 0, st, a, work);
  if (!a.open) hipLaunchKernelGGL(sample_sums_kernel<VerifyArgs>, grid, dim3(kGroupThreads), 0, st, a, work);
  hipLaunchKernelGGL(verify_rows_kernel, dim3(unsigned(p.rows)), dim3(kSampleThreads), 0, st, a, work);
  if (draft_logits)
    hipLaunchKernelGGL(verify_rest_kernel, dim3(across, unsigned(n_seq)), dim3(kGroupThreads), 0, st, a, work);
  hipLaunchKernelGGL(verify_draw_kernel, dim3(unsigned(n_seq)), dim3(kSampleThreads), 0, st, a, work);
  return launch_status(name);
}
