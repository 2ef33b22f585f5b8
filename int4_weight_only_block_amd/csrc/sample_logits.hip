// sample_logits: temperature, top-k, top-p and min-p over a row of logits and
// one draw from what they leave.
//
// Order and arithmetic. Tokens are ranked by an integer key that orders like
// the fp32 logit (equal logits: lower index first). A weight
// exp(l - l_max), formed in fp64, enters every sum as a 42-bit fixed-point
// fraction, so sums of up to 2^20 weights are exact 64-bit integers: they do
// not depend on the order of the additions (atomics included) and a border
// falls in the same place every time.
//
// A cut (key, index) keeps the tokens ranked up to it. Top-k and top-p both
// keep a prefix of the ranking while the sum of a measure (1, or the weight)
// over the better-ranked tokens is below a target, so one radix descent over
// the key's digits, and over the index's among equal keys, finds either.
//
// Four launches; what is left after each is less by orders of magnitude:
//  1. groups of V / 256 logits: largest and smallest key of each;
//  2. a histogram over 512 steps of log2(w), from the largest weight down to
//     2^-44 (or to the row's smallest): count, weight and largest key of each.
//     With top_k <= 256 the k-th largest of the group maxima bounds the k-th
//     largest logit from below, so all but about k logits are left out here
//     by one comparison;
//  3. the histogram says in which step each filter's border lies: tokens
//     above it are summed per group, those in it (a few to a few thousand)
//     go on a list;
//  4. one workgroup per row finds the borders among the list's tokens, adds
//     what they keep to the group sums, finds the group that the drawn number
//     falls in and walks it in index order.
// A list that is too long (thousands of equal logits at a border) makes the
// last step find the borders in the row itself.
#include <math.h>

#include "q4dec_internal.h"
#include "q4dec_serve.h"

namespace q4dec {
Q4DEC_DEBUG_READER(sample_logits)

typedef unsigned long long u64;

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kFracBits = 42;

struct SampleArgs {
  const float* logits;
  int64_t row_stride;
  int vocab;
  float cap;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* idx_out;
  float* prob_out;
};

// fp32 -> integer that orders like the value (-0 as +0); 0 for NaN and
// -infinity, which are never drawn (every other value is above it).
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.0f);
  const uint32_t key = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (z > -INFINITY) ? key : 0u;
}

// 2^y for y in [-1000, 60], to 2^-46 of the value: the Taylor polynomial of
// degree 11 of 2^f, |f| <= 1/2 (its first left-out term is below 2^-47).
__device__ __forceinline__ double exp2_poly(double y) {
  const double n = rint(y), f = (y - n) * 0.6931471805599453;
  double p = 1.0 / 39916800.0;
  p = fma(p, f, 1.0 / 3628800.0);
  p = fma(p, f, 1.0 / 362880.0);
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  p = fma(p, f, 1.0);
  return ldexp(p, int(n));
}

// tanh to 2^-45 absolute: 1 - 2 / (e^2x + 1), the quotient by two Newton steps
__device__ __forceinline__ double tanh_abs(double x) {
  const double e = exp2_poly(fmin(fmax(x, -20.0), 20.0) * 2.8853900817779268) + 1.0;
  double r = __builtin_amdgcn_rcp(e);
  r = fma(fma(-e, r, 1.0), r, r);
  r = fma(fma(-e, r, 1.0), r, r);
  return fma(-2.0, r, 1.0);
}

struct Weights {
  double cap, inv_cap, scale, top;  // scale = log2(e) / T, top = cap * tanh(z_max / cap)
  float z_max;
  __device__ __forceinline__ double capped(float z) const { return cap > 0.0 ? cap * tanh_abs(double(z) * inv_cap) : double(z); }
  // how many octaves below the largest weight; 0 for the largest logit, also where it is +infinity
  __device__ __forceinline__ double octaves(float z) const { return z == z_max ? 0.0 : (top - capped(z)) * scale; }
  static __device__ __forceinline__ double weight_at(double oct) { return oct < 64.0 ? exp2_poly(-oct) : 0.0; }
  __device__ __forceinline__ double weight(float z) const { return weight_at(octaves(z)); }
};
__device__ __forceinline__ float key_value(uint32_t key) {
  return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ Weights weights_of(float cap, float heat, uint32_t max_key) {
  Weights w;
  w.cap = double(cap);
  w.inv_cap = 1.0 / w.cap;
  w.scale = 1.4426950408889634 / double(heat);
  w.z_max = key_value(max_key);
  w.top = w.capped(w.z_max);
  return w;
}

__device__ __forceinline__ u64 fixed(double w) { return u64(rint(w * double(1ull << kFracBits))); }

__device__ __forceinline__ u64 wave_sum(u64 v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

struct Shared {
  u64 hist[256];
  u64 wave[kSampleWaves];
  u64 rest;
  uint32_t digit;
};

// In the histogram of a digit: the digit, from 255 down (or from 0 up for
// ASC), at which the running sum passes `target`, and what is left of the
// target there. target <= sum of the histogram.
template <bool ASC>
__device__ __forceinline__ void find_digit(Shared& sh, u64 target) {
  __syncthreads();
  if (threadIdx.x < 64) {
    u64 c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = int(threadIdx.x) * 4 + i;
      c[i] = sh.hist[ASC ? d : 255 - d];
      sum += c[i];
    }
    u64 before = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const u64 o = __shfl_up(before, off);
      if (int(threadIdx.x) >= off) before += o;
    }
    before -= sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = int(threadIdx.x) * 4 + i;
      if (before < target && target <= before + c[i]) {
        sh.digit = ASC ? d : 255 - d;
        sh.rest = target - before;
      }
      before += c[i];
    }
  }
  __syncthreads();
}

// The last token, in rank order, before which the measure's sum is below
// `target` (1 <= target <= the measure's whole sum); over the tokens that
// each(f) calls f(key, index, weight as a function) for, in any order.
template <bool WEIGHTED, class EACH>
__device__ __forceinline__ void find_cut(Shared& sh, u64 target, uint32_t key_lo, uint32_t key_hi, const Weights& wt,
                                         EACH each, uint32_t& key_cut, int& idx_cut) {
  // all keys lie in [key_lo, key_hi]: only the digits of the difference
  const int bits = key_hi > key_lo ? 32 - __clz(int(key_hi - key_lo)) : 1;
  uint32_t rel = 0;
  if (threadIdx.x == 0) sh.digit = 0, sh.rest = 1;
  for (int shift = (bits - 1) / 8 * 8; shift >= 0; shift -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0;
    __syncthreads();
    each([&](uint32_t key, int, float z) {
      const uint32_t k = key - key_lo;
      if (((k ^ rel) >> shift) >> 8) return;  // another higher digit
      const u64 w = WEIGHTED ? fixed(wt.weight(z)) : 1ull;
      if (w) atomicAdd(&sh.hist[(k >> shift) & 255u], w);
    });
    find_digit<false>(sh, target);
    rel |= sh.digit << shift;
    target = sh.rest;
  }
  const uint32_t key = key_lo + rel;
  // the ties of that key, by index: each weighs the same
  u64 ties = target, whole = sh.hist[sh.digit];
  if (WEIGHTED) {
    const u64 w = max(fixed(wt.weight(key_value(key))), u64(1));
    ties = (target + w - 1) / w;
    whole /= w;
  }
  uint32_t idx = 0x7FFFFFFF;
  if (ties < whole) {
    idx = 0;
    for (int shift = 16; shift >= 0; shift -= 8) {
      __syncthreads();
      if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0;
      __syncthreads();
      each([&](uint32_t k, int i, float) {
        if (k == key && (uint32_t(i) >> (shift + 8)) == (idx >> (shift + 8)))
          atomicAdd(&sh.hist[(uint32_t(i) >> shift) & 255u], 1ull);
      });
      find_digit<true>(sh, ties);
      idx |= sh.digit << shift;
      ties = sh.rest;
    }
  }
  __syncthreads();
  key_cut = key;
  idx_cut = int(idx);
}

// ------------------------------------------------------- the row's workspace
constexpr int kGroups = 256;  // at most; groups of 64 * e logits
constexpr int kBins = 512;
constexpr double kOctaves = 44.0;  // a weight 2^-44 rounds to nothing
constexpr int kList = 8192;
constexpr int kPerThread = kList / kSampleThreads;

struct RowWork {
  uint32_t group_key[kGroups];  // largest key of each group, and its index
  int32_t group_idx[kGroups];
  uint32_t group_min[kGroups];  // smallest key that may be drawn
  u64 group_sum[kGroups];       // weights that stay for certain
  u64 weight[kBins];
  uint32_t count[kBins];
  uint32_t top_key[kBins];
  uint32_t list_n;
  uint32_t pad[31];
  uint2 list[kList];  // (key, index)
};

struct GroupPlan {
  int per, groups;  // logits of a group (a multiple of 64), groups of a row
};
__host__ __device__ inline GroupPlan group_plan(int vocab) {
  const int e = (vocab + 64 * kGroups - 1) / (64 * kGroups);
  return {64 * e, (vocab + 64 * e - 1) / (64 * e)};
}

constexpr int kGroupThreads = 256;  // launches 1 to 3: a wave per group
constexpr int kGroupWaves = kGroupThreads / 64;

// 1: one wave per group.
__global__ __launch_bounds__(kGroupThreads) void sample_groups_kernel(SampleArgs a, RowWork* ws) {
  const GroupPlan gp = group_plan(a.vocab);
  Q4_DCHECK(int64_t(gridDim.x) * kGroupWaves >= gp.groups && gp.groups <= kGroups, kDbgSampleGrid);
  const int lane = threadIdx.x & 63, group = blockIdx.x * kGroupWaves + int(threadIdx.x >> 6);
  RowWork& w = ws[blockIdx.y];
  for (int i = blockIdx.x * kGroupThreads + threadIdx.x; i < kBins; i += gridDim.x * kGroupThreads) {
    w.weight[i] = 0;
    w.count[i] = 0;
    w.top_key[i] = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) w.list_n = 0;
  if (group >= gp.groups) return;
  const float* z = a.logits + size_t(blockIdx.y) * a.row_stride;
  const int lo = group * gp.per, hi = min(lo + gp.per, a.vocab);
  uint32_t best = 0, least = 0xFFFFFFFFu;
  int bidx = -1;
#pragma unroll 16
  for (int i = lo + lane; i < hi; i += 64) {
    const uint32_t k = order_key(z[i]);
    if (k > best) best = k, bidx = i;
    if (k != 0) least = min(least, k);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const uint32_t ok = __shfl_xor(best, off);
    const int oi = __shfl_xor(bidx, off);
    if (ok > best || (ok == best && ok != 0 && oi < bidx)) best = ok, bidx = oi;
    least = min(least, uint32_t(__shfl_xor(least, off)));
  }
  if (lane == 0) {
    w.group_key[group] = best;
    w.group_idx[group] = bidx;
    w.group_min[group] = least;
  }
}

// What every later launch derives again from the groups: the first-ranked
// token, a bound below the top-k border, and the histogram's scale.
struct RowInfo {
  uint32_t max_key, floor_key;  // keys below floor_key are not among the top_k
  int max_idx;
  bool plain;  // nothing to draw: no token, or greedy
  Weights wt;
  double bins;  // per octave
};
struct InfoShared {
  uint32_t key[kGroups], least[4], best[4], floor;
  int idx[4];
};

// top_k as a filter: 0 if it is off
__device__ __forceinline__ int top_k_of(const SampleArgs& a, int r) {
  const int k = a.top_k ? a.top_k[r] : 0;
  return k > 0 && k < a.vocab ? k : 0;
}

// Called by every thread; the first 256 hold a group each.
__device__ __forceinline__ RowInfo row_info(const SampleArgs& a, const RowWork& w, int r, InfoShared& sh) {
  const GroupPlan gp = group_plan(a.vocab);
  const int t = threadIdx.x, lane = t & 63;
  if (t < kGroups) {
    const bool in = t < gp.groups;
    uint32_t best = in ? w.group_key[t] : 0u, least = in ? w.group_min[t] : 0xFFFFFFFFu;
    int bidx = in ? w.group_idx[t] : -1;
    sh.key[t] = best;
    if (t == 0) sh.floor = 0;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const uint32_t ok = __shfl_xor(best, off);
      const int oi = __shfl_xor(bidx, off);
      if (ok > best || (ok == best && ok != 0 && oi < bidx)) best = ok, bidx = oi;
      least = min(least, uint32_t(__shfl_xor(least, off)));
    }
    if (lane == 0) sh.best[t >> 6] = best, sh.idx[t >> 6] = bidx, sh.least[t >> 6] = least;
  }
  __syncthreads();
  const int top_k = top_k_of(a, r);
  if (top_k > 0 && top_k <= gp.groups && t < gp.groups) {
    // the top_k-th largest of the group maxima: at least top_k logits reach it
    const uint32_t mine = sh.key[t];
    int above = 0, ties = 0;
#pragma unroll 8
    for (int i = 0; i < gp.groups; ++i) {
      above += sh.key[i] > mine;
      ties += sh.key[i] == mine;
    }
    if (above < top_k && top_k <= above + ties) sh.floor = mine;  // (the same value from every tie)
  }
  __syncthreads();
  RowInfo o;
  o.max_key = sh.best[0], o.max_idx = sh.idx[0];
  uint32_t least = sh.least[0];
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    if (sh.best[i] > o.max_key) o.max_key = sh.best[i], o.max_idx = sh.idx[i];  // (later groups, later indices)
    least = min(least, sh.least[i]);
  }
  o.floor_key = max(sh.floor, least);
  const float heat = a.temperature ? a.temperature[r] : 1.0f;
  o.plain = o.max_key == 0 || !(heat > 0.0f);
  if (!o.plain) {
    o.wt = weights_of(a.cap, heat, o.max_key);
    const double range = o.wt.octaves(key_value(o.floor_key));
    o.bins = double(kBins - 1) / fmax(range < kOctaves ? range : kOctaves, 0x1p-40);
  }
  return o;
}

__device__ __forceinline__ float top_p_of(const SampleArgs& a, int r) {
  const float p = a.top_p ? a.top_p[r] : 1.0f;
  return p < 1.0f ? fmaxf(p, 0.0f) : 1.0f;  // (a NaN switches it off)
}
__device__ __forceinline__ double min_p_of(const SampleArgs& a, int r) {
  const float p = a.min_p ? a.min_p[r] : 0.0f;
  return p > 0.0f ? fmin(double(p), 1.0) : 0.0;
}

// 2: the histogram.
__global__ __launch_bounds__(kGroupThreads) void sample_bins_kernel(SampleArgs a, RowWork* ws) {
  __shared__ InfoShared info_sh;
  __shared__ u64 weight[kBins];
  __shared__ uint32_t count[kBins], top_key[kBins];
  const GroupPlan gp = group_plan(a.vocab);
  const int r = blockIdx.y, lane = threadIdx.x & 63;
  if (top_k_of(a, r) == 0 && !(top_p_of(a, r) < 1.0f)) return;  // no border to find
  for (int i = threadIdx.x; i < kBins; i += kGroupThreads) weight[i] = 0, count[i] = 0, top_key[i] = 0;
  RowWork& w = ws[r];
  const RowInfo in = row_info(a, w, r, info_sh);
  if (in.plain) return;
  const float* z = a.logits + size_t(r) * a.row_stride;
  const int group = blockIdx.x * kGroupWaves + int(threadIdx.x >> 6);
  if (group < gp.groups && info_sh.key[group] >= in.floor_key) {
    const int lo = group * gp.per, hi = min(lo + gp.per, a.vocab);
    for (int base = lo; base < hi; base += 16 * 64) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = base + 64 * e + lane < hi ? z[base + 64 * e + lane] : -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t k = order_key(v[e]);
        if (k == 0 || k < in.floor_key) continue;
        const double oct = in.wt.octaves(v[e]);
        const int bin = int(fmin(oct * in.bins, double(kBins - 1)));
        atomicAdd(&count[bin], 1u);
        atomicMax(&top_key[bin], k);
        const u64 f = fixed(Weights::weight_at(oct));
        if (f) atomicAdd(&weight[bin], f);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kGroupThreads)
    if (count[i]) {
      atomicAdd(&w.count[i], count[i]);
      atomicMax(&w.top_key[i], top_key[i]);
      if (weight[i]) atomicAdd(&w.weight[i], weight[i]);
    }
}

// Where the borders lie. Keys in (a_lo, a_hi] may hold the top-p border, keys
// in (b_lo, b_hi] hold the top-k one; of the rest those above `sure` stay.
struct Borders {
  uint32_t sure, a_lo, a_hi, b_lo, b_hi;
  u64 k_rest;     // tokens of the top-k step that stay; 0: top_k is off
  u64 above_k;    // weight of the better steps
  bool p_on;
};
struct BorderShared {
  u64 weight[kBins + 1];  // of the better steps
  uint32_t count[kBins + 1], top_key[kBins + 1];
  u64 wave_w[4];
  uint32_t wave_c[4];
  int bin_k, bin_lo, bin_hi, next_k, next_hi;
};

// the step that `target` > 0 of the weight falls in: call with every thread
__device__ __forceinline__ bool in_step(const u64* sums, int i, u64 target) { return sums[i] < target && target <= sums[i + 1]; }

// Called by every thread; the first 256 hold two steps each.
__device__ __forceinline__ Borders find_borders(const SampleArgs& a, const RowWork& w, int r, uint32_t floor_key,
                                                BorderShared& sh) {
  const int t = threadIdx.x, lane = t & 63;
  u64 w0 = 0, w1 = 0, ws = 0;
  uint32_t c0 = 0, c1 = 0, cs = 0;
  if (t < kBins / 2) {
    w0 = w.weight[2 * t], w1 = w.weight[2 * t + 1];
    c0 = w.count[2 * t], c1 = w.count[2 * t + 1];
    sh.top_key[2 * t] = w.top_key[2 * t];
    sh.top_key[2 * t + 1] = w.top_key[2 * t + 1];
    ws = w0 + w1, cs = c0 + c1;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const u64 ow = __shfl_up(ws, off);
      const uint32_t oc = __shfl_up(cs, off);
      if (lane >= off) ws += ow, cs += oc;
    }
    if (lane == 63) sh.wave_w[t >> 6] = ws, sh.wave_c[t >> 6] = cs;
  }
  if (t == 0) sh.bin_k = sh.bin_lo = sh.bin_hi = -1, sh.next_k = sh.next_hi = kBins, sh.top_key[kBins] = 0;
  __syncthreads();
  if (t < kBins / 2) {
    for (int i = 0; i < t >> 6; ++i) ws += sh.wave_w[i], cs += sh.wave_c[i];
    sh.weight[2 * t] = ws - w1 - w0, sh.weight[2 * t + 1] = ws - w1;
    sh.count[2 * t] = cs - c1 - c0, sh.count[2 * t + 1] = cs - c1;
    if (t == kBins / 2 - 1) sh.weight[kBins] = ws, sh.count[kBins] = cs;
  }
  __syncthreads();
  const uint32_t top_k = top_k_of(a, r);
  for (int i = t; i < kBins; i += blockDim.x)
    if (top_k > 0 && sh.count[i] < top_k && top_k <= sh.count[i + 1]) sh.bin_k = i;
  __syncthreads();
  // The last step that top_k leaves something of (-1: it leaves all), and
  // whether its border cuts it: not if the border is the step's end, and not
  // if the step has no weight.
  const int end = sh.bin_k;
  const bool cut = end >= 0 && sh.count[end + 1] > top_k && sh.weight[end + 1] > sh.weight[end];
  const u64 s_hi = sh.weight[end >= 0 ? end + 1 : kBins], s_lo = cut ? sh.weight[end] : s_hi;
  const float top_p = top_p_of(a, r);
  const bool p_on = top_p < 1.0f;
  const u64 t_lo = u64(fmax(ceil(double(top_p) * double(s_lo)), 1.0));
  const u64 t_hi = u64(fmax(ceil(double(top_p) * double(s_hi)), 1.0));
  for (int i = t; i < kBins; i += blockDim.x) {
    if (p_on && in_step(sh.weight, i, t_lo)) sh.bin_lo = i;
    if (p_on && in_step(sh.weight, i, t_hi)) sh.bin_hi = i;
  }
  __syncthreads();
  const int lo = sh.bin_lo, hi = sh.bin_hi;
  for (int i = t; i < kBins; i += blockDim.x)
    if (sh.count[i + 1] > sh.count[i]) {
      if (i > hi) atomicMin(&sh.next_hi, i);
      if (i > end) atomicMin(&sh.next_k, i);
    }
  __syncthreads();
  Borders o = {};
  o.p_on = p_on;
  o.k_rest = cut ? top_k - sh.count[end] : 0;
  o.above_k = s_lo;
  // (tokens below the floor are in no step)
  const uint32_t floor = floor_key - 1, below_k = max(sh.top_key[sh.next_k], floor);
  o.sure = end >= 0 ? below_k : floor;
  if (cut) o.b_hi = sh.top_key[end], o.b_lo = below_k, o.sure = o.b_hi;
  if (p_on) o.a_hi = sh.top_key[lo], o.a_lo = max(sh.top_key[sh.next_hi], floor), o.sure = o.a_hi;
  return o;
}

// 3: sums of what stays for certain, and the list of what may.
__global__ __launch_bounds__(kGroupThreads) void sample_sums_kernel(SampleArgs a, RowWork* ws) {
  __shared__ InfoShared info_sh;
  __shared__ BorderShared border_sh;
  const GroupPlan gp = group_plan(a.vocab);
  const int r = blockIdx.y, lane = threadIdx.x & 63;
  RowWork& w = ws[r];
  const RowInfo in = row_info(a, w, r, info_sh);
  if (in.plain) return;
  Borders b = {};
  if (top_k_of(a, r) > 0 || top_p_of(a, r) < 1.0f) b = find_borders(a, w, r, in.floor_key, border_sh);
  const double min_p = min_p_of(a, r);
  const float* z = a.logits + size_t(r) * a.row_stride;
  const int group = blockIdx.x * kGroupWaves + int(threadIdx.x >> 6);
  if (group >= gp.groups) return;
  u64 sum = 0;
  const uint32_t lowest = min(b.sure, min(b.a_hi > b.a_lo ? b.a_lo : ~0u, b.b_hi > b.b_lo ? b.b_lo : ~0u));
  if (info_sh.key[group] > lowest) {
    const int lo = group * gp.per, hi = min(lo + gp.per, a.vocab);
    for (int base = lo; base < hi; base += 16 * 64) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = base + 64 * e + lane < hi ? z[base + 64 * e + lane] : -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t k = order_key(v[e]);
        if (k > b.sure) {
          const double x = in.wt.weight(v[e]);
          if (x >= min_p) sum += fixed(x);
        } else if ((k > b.a_lo && k <= b.a_hi) || (k > b.b_lo && k <= b.b_hi)) {
          const uint32_t at = atomicAdd(&w.list_n, 1u);
          if (at < kList) w.list[at] = make_uint2(k, uint32_t(base + 64 * e + lane));
        }
      }
    }
  }
  sum = wave_sum(sum);
  if (lane == 0) w.group_sum[group] = sum;
}

// 4: one workgroup per row.
__global__ __launch_bounds__(kSampleThreads) void sample_draw_kernel(SampleArgs a, RowWork* ws) {
  __shared__ InfoShared info_sh;
  __shared__ BorderShared border_sh;
  __shared__ Shared sh;
  __shared__ u64 sums[kGroups];
  __shared__ int chosen;
  const GroupPlan gp = group_plan(a.vocab);
  const int r = blockIdx.x, t = threadIdx.x, lane = t & 63, wave = t >> 6;
  RowWork& w = ws[r];
  const RowInfo in = row_info(a, w, r, info_sh);
  if (in.plain) {
    if (t == 0) {
      a.idx_out[r] = in.max_idx;
      if (a.prob_out) a.prob_out[r] = in.max_key == 0 ? NAN : 1.0f;
    }
    return;
  }
  const float* z = a.logits + size_t(r) * a.row_stride;
  const Weights& wt = in.wt;
  const double min_p = min_p_of(a, r);
  const bool filtered = top_k_of(a, r) > 0 || top_p_of(a, r) < 1.0f;
  Borders b = {};
  if (filtered) b = find_borders(a, w, r, in.floor_key, border_sh);
  if (t < kGroups) sums[t] = t < gp.groups ? w.group_sum[t] : 0;
  // kept: ranked up to (key_cut, idx_cut)
  uint32_t key_cut = b.sure + 1;
  int idx_cut = 0x7FFFFFFF;
  auto kept = [&](uint32_t k, int i) { return k > key_cut || (k == key_cut && i <= idx_cut); };
  const uint32_t n = filtered ? w.list_n : 0;
  if (n > 0) {
    uint2 mine[kPerThread];
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const uint32_t at = e * kSampleThreads + t;
      mine[e] = at < min(n, uint32_t(kList)) ? w.list[at] : make_uint2(0u, 0u);
    }
    // the tokens with keys in (lo, hi]: from the list, or where it has no
    // room for them all, from the row
    auto between = [&](uint32_t lo, uint32_t hi) {
      return [&, lo, hi](auto f) {
        if (n <= kList) {
#pragma unroll
          for (int e = 0; e < kPerThread; ++e)
            if (mine[e].x > lo && mine[e].x <= hi) f(mine[e].x, int(mine[e].y), key_value(mine[e].x));
        } else {
          for (int i = t; i < a.vocab; i += kSampleThreads) {
            const uint32_t k = order_key(z[i]);
            if (k > lo && k <= hi) f(k, i, key_value(k));
          }
        }
      };
    };
    u64 whole = b.above_k;  // weight of what top_k leaves
    if (b.k_rest > 0) {
      find_cut<false>(sh, b.k_rest, b.b_lo + 1, b.b_hi, wt, between(b.b_lo, b.b_hi), key_cut, idx_cut);
      if (b.p_on) {
        u64 s = 0;
        between(b.b_lo, b.b_hi)([&](uint32_t k, int i, float v) {
          if (kept(k, i)) s += fixed(wt.weight(v));
        });
        s = wave_sum(s);
        if (lane == 0) sh.wave[wave] = s;
        __syncthreads();
        for (int i = 0; i < kSampleWaves; ++i) whole += sh.wave[i];
      }
    }
    if (b.p_on) {
      const u64 target = u64(fmax(ceil(double(top_p_of(a, r)) * double(whole)), 1.0));
      if (t == 0) border_sh.next_hi = kBins;
      __syncthreads();
      for (int i = t; i < kBins; i += kSampleThreads)
        if (in_step(border_sh.weight, i, target)) border_sh.bin_hi = i;
      __syncthreads();
      const int bin = border_sh.bin_hi;
      for (int i = t; i < kBins; i += kSampleThreads)
        if (i > bin && border_sh.count[i + 1] > border_sh.count[i]) atomicMin(&border_sh.next_hi, i);
      __syncthreads();
      const uint32_t lo = border_sh.top_key[border_sh.next_hi], hi = border_sh.top_key[bin];
      find_cut<true>(sh, target - border_sh.weight[bin], lo + 1, hi, wt, between(lo, hi), key_cut, idx_cut);
    }
    // what the list's tokens add to their groups
    between(0, b.sure)([&](uint32_t k, int i, float v) {
      if (!kept(k, i)) return;
      const double x = wt.weight(v);
      if (x >= min_p) atomicAdd(&sums[i / gp.per], fixed(x));
    });
  }
  __syncthreads();
  // the group that the drawn number falls in (the first-ranked token always stays: the whole is not 0)
  if (t < 64) {
    u64 c[4], own = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) own += c[i] = sums[4 * t + i];
    u64 upto = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const u64 o = __shfl_up(upto, off);
      if (lane >= off) upto += o;
    }
    const u64 whole = __shfl(upto, 63);
    const float uf = a.u[r];
    const double u = uf > 0.0f ? fmin(double(uf), 1.0) : 0.0;
    u64 target = u64(u * double(whole));
    if (target >= whole) target = whole - 1;
    u64 before = upto - own;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (before <= target && target < before + c[i]) {
        chosen = 4 * t + i;
        sh.rest = target - before;
        sh.hist[0] = whole;
      }
      before += c[i];
    }
  }
  __syncthreads();
  u64 target = sh.rest;
  const u64 whole = sh.hist[0];
  const int lo = chosen * gp.per, hi = min(lo + gp.per, a.vocab);
  for (int base = lo; base < hi; base += kSampleThreads) {
    const int i = base + t;
    u64 own = 0;
    double x = 0.0;
    if (i < hi) {
      const uint32_t k = order_key(z[i]);
      if (k != 0 && kept(k, i)) {
        x = wt.weight(z[i]);
        own = x >= min_p ? fixed(x) : 0;
      }
    }
    u64 upto = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const u64 o = __shfl_up(upto, off);
      if (lane >= off) upto += o;
    }
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
      if (a.prob_out) a.prob_out[r] = float(x * double(1ull << kFracBits) / double(whole));
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
  const SampleArgs a = {logits, row_stride, int(vocab), cap, temperature, top_k, top_p, min_p, u, idx_out, prob_out};
  RowWork* work = static_cast<RowWork*>(ws);
  const GroupPlan gp = group_plan(a.vocab);
  const dim3 grid(unsigned((gp.groups + kGroupWaves - 1) / kGroupWaves), unsigned(n_rows));
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(sample_groups_kernel, grid, dim3(kGroupThreads), 0, st, a, work);
  hipLaunchKernelGGL(sample_bins_kernel, grid, dim3(kGroupThreads), 0, st, a, work);
  hipLaunchKernelGGL(sample_sums_kernel, grid, dim3(kGroupThreads), 0, st, a, work);
  hipLaunchKernelGGL(sample_draw_kernel, dim3(unsigned(n_rows)), dim3(kSampleThreads), 0, st, a, work);
  return launch_status(name);
}
