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
//  2. with top_k <= 256 the k-th largest of the group maxima bounds the k-th
//     largest logit from below: the logits that reach it, a little more than
//     k, go on a list, and the next launch has nothing to do. Otherwise a
//     histogram over 512 steps of log2(w), from the largest weight down to
//     2^-44 (or to the row's smallest): count, weight and largest key of each;
//  3. the histogram says in which step each filter's border lies: tokens
//     above it are summed per group, those in it (a few to a few thousand)
//     go on the list;
//  4. one workgroup per row finds the borders among the list's tokens and
//     draws: up to 256 tokens by comparing all with all, else by adding what
//     the borders leave to the group sums and walking the group that the
//     drawn number falls in.
// A list that is too long makes the last step find the borders in the row
// itself. Thousands of equal logits at a border do that, and so do finite masks
// under a small top_k that fewer groups than top_k rise above: one row of 262144
// of which 40 are not -1e4, top-k 64, 2500 us (21 with -infinity); rows of fewer
// groups than top_k (50257 logits are 197), top-k 200, 260 us.
//
// What launches 2 to 4 derive again from the groups or the histogram one wave
// derives in registers; sharing the work out over waves costs more barriers
// than it saves.
//
// Measured: one row of 262144 with top-k 64 and top-p 16.0 us, five of 100003
// without a filter 14.9 us (chains of four launches), 64 of 262144 with mixed
// filters 72 us, without one 55 us (67 MB, 13 us at a copy's rate): there a
// weight is about 65 vector instructions, most of them fp64, and each of 4096
// workgroups has some 5 us of chained loads and sums before its first weight.
#pragma once

#include <math.h>

#include <type_traits>

#include "q4dec_internal.h"
#include "q4dec_serve.h"
#include "serve_internal.h"

namespace q4dec {

typedef unsigned long long u64;

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kFracBits = 42;
constexpr int kGroups = 256;  // of a row, at most; groups of 64 * e logits

// The second and third launch and the parts of all are verify_drafts' too, whose
// rows have other places, settings and caps: what they ask of their arguments
// are row_used, row_at, filters_of and sums_known.
struct SampleArgs {
  const float* logits;
  int64_t row_stride;
  int vocab;
  double cap, inv_cap;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* idx_out;
  float* prob_out;
};
__device__ __forceinline__ bool row_used(const SampleArgs&, int) { return true; }
__device__ __forceinline__ const float* row_at(const SampleArgs& a, int r) { return a.logits + size_t(r) * a.row_stride; }

// fp32 -> integer that orders like the value (-0 as +0); 0 for NaN and
// -infinity, which are never drawn (every other value is above it).
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.0f);
  const uint32_t key = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (z > -INFINITY) ? key : 0u;
}

// The weights are computed for N tokens side by side. Every launch gets the
// same bits for a token, whatever its neighbours: no contraction that the
// compiler may choose or not, and each branch's result is selected per token.
#pragma clang fp contract(off)

// 2^y for y in [-1000, 60], to 2^-51 of the value: the polynomial that meets
// 2^f in the 11 Chebyshev nodes of [-1/2, 1/2] (in 60-digit arithmetic).
template <int N>
__device__ __forceinline__ void exp2_poly(const double (&y)[N], double (&out)[N]) {
  constexpr double kC[] = {1.0208690299958306e-07, 1.321544258792169e-06, 1.5252657260200837e-05,
                           0.0001540353044173605,  0.0013333558230164974, 0.009618129107606888,
                           0.05550410866444772,    0.24022650695910097,   0.69314718055995, 1.0};
  double n[N], f[N], p[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    n[j] = rint(y[j]);
    f[j] = y[j] - n[j];
    p[j] = 7.072585949269223e-09;
  }
#pragma unroll
  for (int i = 0; i < 10; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = fma(p[j], f[j], kC[i]);
#pragma unroll
  for (int j = 0; j < N; ++j) out[j] = ldexp(p[j], int(n[j]));
}

// tanh to 2^-45 absolute. Small arguments (logits within 0.45 of the cap, most
// of them) by the polynomial that meets tanh(x) / x in the 8 Chebyshev nodes
// of x^2 in [0, 0.45^2]; else 1 - 2 / (e^2x + 1), the quotient by two Newton
// steps.
template <int N>
__device__ __forceinline__ void tanh_abs(const double (&x)[N], double (&out)[N]) {
  constexpr double kC[] = {0.003469517587012053, -0.008842871160416817, 0.021867589319773756, -0.05396815710836195,
                           0.13333333089707022,  -0.3333333333099173,   0.999999999999963};
  double y[N], p[N];
  bool big = false;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    big = big || !(fabs(x[j]) <= 0.45);
    y[j] = x[j] * x[j];
    p[j] = -0.0010586183492814069;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = fma(p[j], y[j], kC[i]);
#pragma unroll
  for (int j = 0; j < N; ++j) out[j] = p[j] * x[j];
  if (__ballot(big) == 0) return;
  double e[N], r[N];
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = fmin(fmax(x[j], -20.0), 20.0) * 2.8853900817779268;
  exp2_poly(e, e);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    e[j] = e[j] + 1.0;
    r[j] = __builtin_amdgcn_rcp(e[j]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) r[j] = fma(fma(-e[j], r[j], 1.0), r[j], r[j]);
#pragma unroll
  for (int j = 0; j < N; ++j) out[j] = fabs(x[j]) <= 0.45 ? out[j] : fma(-2.0, r[j], 1.0);
}

struct Weights {
  double inv_cap, steep, top;  // octaves = steep * (top - t), t = tanh(z / cap), or z where there is no cap; top the largest t
  float z_max;
  template <int N>
  __device__ __forceinline__ void capped(const float (&z)[N], double (&t)[N]) const {
    if (inv_cap > 0.0) {
      double x[N];
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = double(z[j]) * inv_cap;
      tanh_abs(x, t);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) t[j] = double(z[j]);
    }
  }
  // How many octaves below the largest weight; 0 for the largest logit, also
  // where it is +infinity. The difference comes first, so that equal t's (far
  // above the cap every t is 1) are 0 octaves apart whatever `steep` is:
  // steep * top - steep * t as one fma leaves the rounding of steep * top,
  // which can be negative. A t above top by its own last bit counts as top: a
  // step of the histogram is never below 0, a weight never above 1.
  template <int N>
  __device__ __forceinline__ void octaves(const float (&z)[N], double (&o)[N]) const {
    capped(z, o);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const double d = steep * (top - o[j]);  // (a NaN stays one)
      o[j] = z[j] == z_max || d < 0.0 ? 0.0 : d;
    }
  }
  // 2^-octaves; 2^-64, which rounds to nothing, from 64 octaves on (and for a NaN)
  template <int N>
  static __device__ __forceinline__ void weights_at(const double (&oct)[N], double (&x)[N]) {
    double y[N];
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] = fmax(-oct[j], -64.0);
    exp2_poly(y, x);
  }
  template <int N>
  __device__ __forceinline__ void weights(const float (&z)[N], double (&x)[N]) const {
    double o[N];
    octaves(z, o);
    weights_at(o, x);
  }
  __device__ __forceinline__ double octaves(float z) const {
    const float zs[1] = {z};
    double o[1];
    octaves(zs, o);
    return o[0];
  }
  // A logit below which every weight certainly rounds to nothing (-infinity:
  // none is known): far down a row (low temperatures) a comparison then saves
  // the fp64. The inverse of the softcap, 46 octaves down, is taken in fp32,
  // and what it gives has to be 45 down by the weights' own arithmetic.
  __device__ __forceinline__ float far_below() const {
    double z = top - 46.0 / steep;
    if (inv_cap > 0.0) {
      const float t = float(z);
      z = double(0.34657359f * __builtin_amdgcn_logf((1.0f + t) / (1.0f - t))) / inv_cap;  // atanh
    }
    const float at = float(z);
    return at < z_max && octaves(at) > 45.0 ? at : -INFINITY;
  }
  __device__ __forceinline__ double weight(float z) const {
    const float zs[1] = {z};
    double x[1];
    weights(zs, x);
    return x[0];
  }
};
__device__ __forceinline__ float key_value(uint32_t key) {
  return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// The filters of a row; top_k is 0 and top_p is 1 where they are off.
struct Filters {
  int top_k;
  float heat, top_p;
  double min_p;
  double cap, inv_cap;  // the latter 0: none
  __device__ bool borders() const { return top_k > 0 || top_p < 1.0f; }
  // top-k from the group maxima, without a histogram
  __device__ bool by_list() const { return top_k > 0 && top_k <= kGroups; }
};
// (r: of the settings, which a sequence's rows may have in common)
template <class ARGS>
__device__ __forceinline__ Filters filters_at(const ARGS& a, int r, double cap, double inv_cap) {
  const int k = a.top_k ? a.top_k[r] : 0;
  const float p = a.top_p ? a.top_p[r] : 1.0f, m = a.min_p ? a.min_p[r] : 0.0f;
  Filters f;
  f.cap = cap, f.inv_cap = inv_cap;
  f.heat = a.temperature ? a.temperature[r] : 1.0f;
  f.top_k = k > 0 && k < a.vocab ? k : 0;
  f.top_p = p < 1.0f ? fmaxf(p, 0.0f) : 1.0f;  // (a NaN switches it off)
  f.min_p = m > 0.0f ? fmin(double(m), 1.0) : 0.0;
  return f;
}
__device__ __forceinline__ Filters filters_of(const SampleArgs& a, int r) { return filters_at(a, r, a.cap, a.inv_cap); }
__device__ __forceinline__ bool sums_known(const SampleArgs&, const Filters&) { return false; }

__device__ __forceinline__ double steep_of(const Filters& f) {
  return 1.4426950408889634 / double(f.heat) * (f.inv_cap > 0.0 ? f.cap : 1.0);
}
__device__ __forceinline__ Weights weights_of(double steep, double inv_cap, uint32_t max_key) {
  Weights w;
  w.inv_cap = inv_cap;
  w.steep = steep;
  w.z_max = key_value(max_key);
  const float top[1] = {w.z_max};
  double t[1];
  w.capped(top, t);
  w.top = t[0];
  return w;
}
__device__ __forceinline__ Weights weights_of(const Filters& f, uint32_t max_key) {
  return weights_of(steep_of(f), f.inv_cap, max_key);
}

// w * 2^42 for w in [0, 1], rounded: 2^52 leaves no fraction bits
__device__ __forceinline__ u64 fixed(double w) {
  return __builtin_bit_cast(u64, fma(w, double(1ull << kFracBits), 0x1p52)) & ((1ull << 52) - 1);
}

// Sums and maxima over a wave by lane moves in the vector unit (a shuffle
// through LDS takes several times as long, and these come in long chains).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v) {  // 0 where nothing is moved to
  return __builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 moved(u64 v) {
  return u64(moved<CTRL, ROWS>(uint32_t(v >> 32))) << 32 | moved<CTRL, ROWS>(uint32_t(v));
}
// sum over the lanes up to this one
template <class T>
__device__ __forceinline__ T wave_upto(T v) {
  v += moved<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
  v += moved<0x112, 0xF>(v);
  v += moved<0x114, 0xF>(v);
  v += moved<0x118, 0xF>(v);
  v += moved<0x142, 0xA>(v);  // row_bcast 15, 31
  v += moved<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {  // (lane uniform)
  return __builtin_amdgcn_readlane(int(v), lane);
}
__device__ __forceinline__ u64 lane_value(u64 v, int lane) {
  return u64(lane_value(uint32_t(v >> 32), lane)) << 32 | lane_value(uint32_t(v), lane);
}
__device__ __forceinline__ u64 wave_sum(u64 v) { return lane_value(wave_upto(v), 63); }
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, moved<0x111, 0xF>(v));
  v = max(v, moved<0x112, 0xF>(v));
  v = max(v, moved<0x114, 0xF>(v));
  v = max(v, moved<0x118, 0xF>(v));
  v = max(v, moved<0x142, 0xA>(v));
  v = max(v, moved<0x143, 0xC>(v));
  return lane_value(v, 63);
}

struct Shared {
  u64 hist[2][256];
  u64 wave[kSampleWaves];
  u64 rest;
  uint32_t digit;
};

// In the histogram of a digit: the digit, from 255 down (or from 0 up for
// ASC), at which the running sum passes `target`, and what is left of the
// target there. target <= sum of the histogram. Clears the other histogram.
template <bool ASC>
__device__ __forceinline__ void find_digit(Shared& sh, int which, u64 target) {
  __syncthreads();
  if (threadIdx.x < 64) {
    u64 c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = int(threadIdx.x) * 4 + i;
      c[i] = sh.hist[which][ASC ? d : 255 - d];
      sum += c[i];
    }
    u64 before = wave_upto(sum) - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = int(threadIdx.x) * 4 + i;
      if (before < target && target <= before + c[i]) {
        sh.digit = ASC ? d : 255 - d;
        sh.rest = target - before;
      }
      before += c[i];
    }
  } else if (threadIdx.x < 64 + 256) {
    sh.hist[which ^ 1][threadIdx.x - 64] = 0;
  }
  __syncthreads();
}

// set beside the weight of a token that min_p leaves out
constexpr u64 kLight = 1ull << 63;

// The last token, in rank order, before which the measure's sum is below
// `target` (1 <= target <= the measure's whole sum); over the tokens that
// each(f) calls f(key, index, weight) for, in any order.
template <bool WEIGHTED, class EACH>
__device__ __forceinline__ void find_cut(Shared& sh, u64 target, uint32_t key_lo, uint32_t key_hi, const Weights& wt,
                                         EACH each, uint32_t& key_cut, int& idx_cut) {
  // all keys lie in [key_lo, key_hi]: only the digits of the difference
  const int bits = key_hi > key_lo ? 32 - __clz(int(key_hi - key_lo)) : 1;
  uint32_t rel = 0;
  int which = 0;  // histogram of this digit
  if (threadIdx.x == 0) sh.digit = 0, sh.rest = 1;
  if (threadIdx.x < 256) sh.hist[0][threadIdx.x] = 0;
  __syncthreads();
  for (int shift = (bits - 1) / 8 * 8; shift >= 0; shift -= 8, which ^= 1) {
    each([&](uint32_t key, int, u64 x) {
      const uint32_t k = key - key_lo;
      if (((k ^ rel) >> shift) >> 8) return;  // another higher digit
      const u64 w = WEIGHTED ? x & ~kLight : 1ull;
      if (w) atomicAdd(&sh.hist[which][(k >> shift) & 255u], w);
    });
    find_digit<false>(sh, which, target);
    rel |= sh.digit << shift;
    target = sh.rest;
  }
  const uint32_t key = key_lo + rel;
  // the ties of that key, by index: each weighs the same
  u64 ties = target, whole = sh.hist[which ^ 1][sh.digit];
  if (WEIGHTED) {
    const u64 w = max(fixed(wt.weight(key_value(key))), u64(1));
    ties = (target + w - 1) / w;
    whole /= w;
  }
  uint32_t idx = 0x7FFFFFFF;
  if (ties < whole) {
    idx = 0;
    for (int shift = 16; shift >= 0; shift -= 8, which ^= 1) {
      each([&](uint32_t k, int i, u64) {
        if (k == key && (uint32_t(i) >> (shift + 8)) == (idx >> (shift + 8)))
          atomicAdd(&sh.hist[which][(uint32_t(i) >> shift) & 255u], 1ull);
      });
      find_digit<true>(sh, which, ties);
      idx |= sh.digit << shift;
      ties = sh.rest;
    }
  }
  __syncthreads();
  key_cut = key;
  idx_cut = int(idx);
}

// ------------------------------------------------------- the row's workspace
constexpr int kBins = 512;
constexpr double kOctaves = 44.0;  // a weight 2^-44 rounds to nothing
constexpr int kList = 4096;
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
__device__ __forceinline__ void group_extremes(RowWork& w, const float* z, int vocab) {
  const GroupPlan gp = group_plan(vocab);
  const int lane = threadIdx.x & 63, group = blockIdx.x * kGroupWaves + int(threadIdx.x >> 6);
  for (int i = blockIdx.x * kGroupThreads + threadIdx.x; i < kBins; i += gridDim.x * kGroupThreads) {
    w.weight[i] = 0;
    w.count[i] = 0;
    w.top_key[i] = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) w.list_n = 0;
  if (group >= gp.groups) return;
  const int lo = group * gp.per, hi = min(lo + gp.per, vocab);
  uint32_t best = 0, least = 0xFFFFFFFFu;
  int bidx = -1;
#pragma unroll 16
  for (int i = lo + lane; i < hi; i += 64) {
    const uint32_t k = order_key(z[i]);
    if (k > best) best = k, bidx = i;
    if (k != 0) least = min(least, k);
  }
  const uint32_t top = wave_max(best);
  const uint32_t idx = ~wave_max(best == top ? ~uint32_t(bidx) : 0u);  // the lowest; -1 if there is none
  least = ~wave_max(~least);
  if (lane == 0) {
    w.group_key[group] = top;
    w.group_idx[group] = int(idx);
    w.group_min[group] = least;
  }
}

// Each wave for itself, four groups a lane. floor_key: no key below it is
// among the top_k (with by_list()), or may be drawn at all.
struct RowInfo {
  uint32_t max_key, floor_key;
  bool plain;  // nothing to draw from: no token, or greedy
  Weights wt;
};
__device__ __forceinline__ RowInfo row_info(int vocab, const RowWork& w, const Filters& f, bool floor) {
  const int groups = group_plan(vocab).groups, lane = threadIdx.x & 63;
  const uint4 kv = reinterpret_cast<const uint4*>(w.group_key)[lane];
  uint32_t k[4] = {kv.x, kv.y, kv.z, kv.w};  // (groups past the last hold leftovers)
#pragma unroll
  for (int i = 0; i < 4; ++i) k[i] = 4 * lane + i < groups ? k[i] : 0u;
  RowInfo o;
  o.max_key = wave_max(max(max(k[0], k[1]), max(k[2], k[3])));
  o.plain = o.max_key == 0 || !(f.heat > 0.0f);
  o.floor_key = 1;
  if (floor) {
    // the top_k-th largest of the maxima to 16 bits, rounded down: at least
    // top_k logits reach it
    uint32_t at = 0;
#pragma unroll 1
    for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1) {
      const uint32_t next = at | bit;
      int n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) n += __popcll(__ballot(k[i] >= next));
      if (n >= f.top_k) at = next;
    }
    o.floor_key = max(at, 1u);
  }
  if (!o.plain) o.wt = weights_of(f, o.max_key);
  return o;
}

// Steps of the histogram per octave: it spans the row's weights, at most 2^44.
__device__ __forceinline__ double steps_of(int vocab, const RowWork& w, const Weights& wt) {
  const int groups = group_plan(vocab).groups, lane = threadIdx.x & 63;
  const uint4 kv = reinterpret_cast<const uint4*>(w.group_min)[lane];
  const uint32_t k[4] = {kv.x, kv.y, kv.z, kv.w};
  uint32_t inv = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) inv = max(inv, 4 * lane + i < groups ? ~k[i] : 0u);
  const double range = wt.octaves(key_value(~wave_max(inv)));
  return double(kBins - 2) / fmax(range < kOctaves ? range : kOctaves, 0x1p-40);
}

// Tokens on their way to the row's list: a wave gathers those of 1024 logits
// in LDS and takes its place in the list once (an atomic per token on the one
// counter took a microsecond each, one after the other).
struct Gather {
  uint2* buf;  // of this wave, 1024 entries
  int n;
  __device__ __forceinline__ void add(bool take, uint32_t key, int idx) {
    const u64 who = __ballot(take);
    if (take) buf[n + __popcll(who & ((1ull << (threadIdx.x & 63)) - 1))] = make_uint2(key, uint32_t(idx));
    n += __popcll(who);
  }
  __device__ __forceinline__ void flush(RowWork& w) {
    if (n == 0) return;
    const int lane = threadIdx.x & 63;
    uint32_t at = 0;
    if (lane == 0) at = atomicAdd(&w.list_n, uint32_t(n));
    at = lane_value(at, 0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int i = lane; i < n; i += 64)
      if (at + i < uint32_t(kList)) w.list[at + i] = buf[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    n = 0;
  }
};

// f(logits, first index) for the group's logits, kSide of a lane (64 apart) at
// a time, -infinity past its end; after() after every 1024
constexpr int kSide = 4;
template <class F, class AFTER>
__device__ __forceinline__ void for_group(const float* z, const GroupPlan& gp, int vocab, int group, F f, AFTER after) {
  const int lane = threadIdx.x & 63, lo = group * gp.per, hi = min(lo + gp.per, vocab);
  for (int base = lo; base < hi; base += 16 * 64) {
    float v[16 / kSide][kSide];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int i = base + lane + 64 * e;
      v[e / kSide][e % kSide] = i < hi ? z[i] : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < 16 / kSide; ++e) f(v[e], base + lane + 64 * kSide * e);
    after();
  }
}

// 2: the list of a small top_k, or the histogram.
template <class ARGS>
__global__ __launch_bounds__(kGroupThreads) void sample_bins_kernel(ARGS a, RowWork* ws) {
  __shared__ __align__(16) uint8_t room[kGroupWaves * 1024 * sizeof(uint2)];
  u64* weight = reinterpret_cast<u64*>(room);
  uint32_t* count = reinterpret_cast<uint32_t*>(room + kBins * 8);
  uint32_t* top_key = count + kBins;
  Gather gather = {reinterpret_cast<uint2*>(room) + (threadIdx.x >> 6) * 1024, 0};
  const GroupPlan gp = group_plan(a.vocab);
  const int r = blockIdx.y, group = blockIdx.x * kGroupWaves + int(threadIdx.x >> 6);
  if (!row_used(a, r)) return;
  const Filters f = filters_of(a, r);
  if (!f.borders()) return;
  RowWork& w = ws[r];
  const float* z = row_at(a, r);
  if (f.by_list()) {
    const RowInfo in = row_info(a.vocab, w, f, true);
    if (in.plain) return;
    if (group < gp.groups && w.group_key[group] >= in.floor_key)
        for_group(z, gp, a.vocab, group, [&](const float (&v)[kSide], int i) {
#pragma unroll
          for (int j = 0; j < kSide; ++j) {
            const uint32_t k = order_key(v[j]);
            gather.add(k >= in.floor_key, k, i + 64 * j);
          }
        }, [&] { gather.flush(w); });
    return;
  }
  // (one wave derives these for the four: 64 rows with top-p 121 -> 117 us)
  __shared__ RowInfo row;
  __shared__ double row_steps;
  __shared__ float row_far;
  if (threadIdx.x < 64) {
    const RowInfo in = row_info(a.vocab, w, f, false);
    if (!in.plain) {
      const double steps = steps_of(a.vocab, w, in.wt);
      const float far = in.wt.far_below();
      if (threadIdx.x == 0) row_steps = steps, row_far = far;
    }
    if (threadIdx.x == 0) row = in;
  } else {
    for (int i = threadIdx.x - 64; i < kBins; i += kGroupThreads - 64) weight[i] = 0, count[i] = 0, top_key[i] = 0;
  }
  __syncthreads();
  const RowInfo in = row;
  if (in.plain) return;
  const double steps = row_steps;
  const float far = row_far;
  {
    // the last step is that of weights that round to nothing: its largest key
    // is all that is wanted, and on a cold row nearly every token is there
    uint32_t tail = 0;
    if (group < gp.groups) for_group(z, gp, a.vocab, group, [&](const float (&v)[kSide], int) {
      uint32_t k[kSide];
      bool near = false;
#pragma unroll
      for (int j = 0; j < kSide; ++j) {
        k[j] = order_key(v[j]);
        near = near || (k[j] != 0 && !(v[j] < far));
      }
      double oct[kSide], x[kSide];
      if (__ballot(near)) {
        in.wt.octaves(v, oct);
        Weights::weights_at(oct, x);
      } else {
#pragma unroll
        for (int j = 0; j < kSide; ++j) oct[j] = x[j] = 0.0;
      }
#pragma unroll
      for (int j = 0; j < kSide; ++j) {
        const u64 y = k[j] ? fixed(x[j]) : 0;
        if (y == 0) {
          tail = max(tail, k[j]);
          continue;
        }
        const int bin = int(fmin(oct[j] * steps, double(kBins - 2)));
        Q4_DCHECK(bin >= 0 && bin <= kBins - 2, kDbgSampleGrid);
        if (f.top_k > 0) atomicAdd(&count[bin], 1u);
        atomicMax(&top_key[bin], k[j]);
        atomicAdd(&weight[bin], y);
      }
    }, [] {});
    tail = wave_max(tail);
    if ((threadIdx.x & 63) == 0 && tail) atomicMax(&top_key[kBins - 1], tail);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kGroupThreads)
    if (top_key[i]) {
      if (count[i]) atomicAdd(&w.count[i], count[i]);
      atomicMax(&w.top_key[i], top_key[i]);
      if (weight[i]) atomicAdd(&w.weight[i], weight[i]);
    }
}

// The histogram in a wave's registers, 8 steps a lane, with running sums.
struct Steps {
  static constexpr int N = kBins / 64;
  u64 before[N + 1];  // weight of the better steps; [N]: with this lane's last
  uint32_t count[N + 1];
  uint32_t key[N];  // largest key of the step, 0: empty

  __device__ __forceinline__ void load(const RowWork& w) {
    const int lane = threadIdx.x & 63;
    u64 x[N];
    uint32_t c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = w.weight[lane * N + i], c[i] = w.count[lane * N + i], key[i] = w.top_key[lane * N + i];
    u64 sx = 0;
    uint32_t sc = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) sx += x[i], sc += c[i];
    before[0] = wave_upto(sx) - sx, count[0] = wave_upto(sc) - sc;
#pragma unroll
    for (int i = 0; i < N; ++i) before[i + 1] = before[i] + x[i], count[i + 1] = count[i] + c[i];
  }
  __device__ __forceinline__ u64 whole() const { return lane_value(before[N], 63); }

  struct At {
    int step;  // -1: none
    uint32_t key, count;
    u64 before, upto;
    uint32_t count_upto;
  };
  // the only step, if any, that `is` holds for
  template <class IS>
  __device__ __forceinline__ At find(IS is) const {
    At mine = {-1, 0, 0, 0, 0, 0};
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (is(i)) mine = {lane * N + i, key[i], count[i], before[i], before[i + 1], count[i + 1]};
    const u64 who = __ballot(mine.step >= 0);
    const int src = who ? __ffsll(who) - 1 : 0;
    At o;
    o.step = int(lane_value(uint32_t(mine.step), src));
    o.key = lane_value(mine.key, src);
    o.count = lane_value(mine.count, src);
    o.before = lane_value(mine.before, src);
    o.upto = lane_value(mine.upto, src);
    o.count_upto = lane_value(mine.count_upto, src);
    return o;
  }
  // the step that the target-th part (from 1) of the weight falls in
  __device__ __forceinline__ At at_weight(u64 target) const {
    return find([&](int i) { return before[i] < target && target <= before[i + 1]; });
  }
  __device__ __forceinline__ At at_count(uint32_t target) const {
    return find([&](int i) { return count[i] < target && target <= count[i + 1]; });
  }
  // largest key of the steps after `step`; 0 if they are empty
  __device__ __forceinline__ uint32_t key_below(int step) const {
    const int lane = threadIdx.x & 63;
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) best = max(best, lane * N + i > step ? key[i] : 0u);
    return wave_max(best);
  }
};

// Where the borders lie. Keys in (a_lo, a_hi] may hold the top-p border, keys
// in (b_lo, b_hi] hold the top-k one; of the rest those above `sure` stay.
struct Borders {
  uint32_t sure, a_lo, a_hi, b_lo, b_hi;
  u64 k_rest;   // tokens from (b_lo, b_hi] that top_k leaves; 0: it cuts nothing there
  u64 above_k;  // weight of what it leaves of better ones
};

__device__ __forceinline__ u64 top_p_target(float top_p, u64 whole) {
  return u64(fmax(ceil(double(top_p) * double(whole)), 1.0));
}

__device__ __forceinline__ Borders borders_of(const Filters& f, const Steps& st) {
  // The last step that top_k leaves something of (-1: it leaves all that has
  // weight), and whether its border cuts it: not if the border is its end.
  const Steps::At end = f.top_k > 0 ? st.at_count(f.top_k) : Steps::At{-1, 0, 0, 0, 0, 0};
  const bool cut = end.step >= 0 && end.count_upto > uint32_t(f.top_k);
  const u64 s_hi = end.step >= 0 ? end.upto : st.whole(), s_lo = cut ? end.before : s_hi;
  const uint32_t below = st.key_below(end.step >= 0 ? end.step : kBins - 2);
  Borders o = {};
  o.k_rest = cut ? f.top_k - end.count : 0;
  o.above_k = s_lo;
  o.sure = below;
  if (cut) o.b_hi = end.key, o.b_lo = below, o.sure = end.key;
  if (f.top_p < 1.0f) {
    const Steps::At lo = st.at_weight(top_p_target(f.top_p, s_lo)), hi = st.at_weight(top_p_target(f.top_p, s_hi));
    o.a_hi = lo.key, o.a_lo = st.key_below(hi.step), o.sure = lo.key;
  }
  return o;
}

// 3: sums of what stays for certain, and the list of what may.
template <class ARGS>
__global__ __launch_bounds__(kGroupThreads) void sample_sums_kernel(ARGS a, RowWork* ws) {
  const GroupPlan gp = group_plan(a.vocab);
  const int r = blockIdx.y, lane = threadIdx.x & 63, group = blockIdx.x * kGroupWaves + int(threadIdx.x >> 6);
  __shared__ uint2 gathered[kGroupWaves][1024];
  Gather gather = {gathered[threadIdx.x >> 6], 0};
  if (!row_used(a, r)) return;
  const Filters f = filters_of(a, r);
  if (f.by_list() || sums_known(a, f)) return;
  RowWork& w = ws[r];
  __shared__ RowInfo row;  // derived by one wave, as above
  __shared__ Borders row_borders;
  __shared__ float row_far;
  if (threadIdx.x < 64) {
    const RowInfo in = row_info(a.vocab, w, f, false);
    if (!in.plain) {
      Borders b = {};
      if (f.borders()) {
        Steps st;
        st.load(w);
        b = borders_of(f, st);
      }
      const float far = in.wt.far_below();
      if (lane == 0) row_borders = b, row_far = far;
    }
    if (lane == 0) row = in;
  }
  __syncthreads();
  const RowInfo in = row;
  if (in.plain || group >= gp.groups) return;
  const Borders b = row_borders;
  const float far = row_far;
  const float* z = row_at(a, r);
  const uint32_t lowest = min(b.sure, min(b.a_hi > b.a_lo ? b.a_lo : ~0u, b.b_hi > b.b_lo ? b.b_lo : ~0u));
  {
    u64 sum = 0;
    if (w.group_key[group] > lowest) {
      if (!f.borders()) {
        for_group(z, gp, a.vocab, group, [&](const float (&v)[kSide], int) {
          bool near = false;
#pragma unroll
          for (int j = 0; j < kSide; ++j) near = near || !(v[j] < far);
          if (__ballot(near) == 0) return;
          double x[kSide];
          in.wt.weights(v, x);
#pragma unroll
          for (int j = 0; j < kSide; ++j) sum += order_key(v[j]) != 0 && x[j] >= f.min_p ? fixed(x[j]) : 0;
        }, [] {});
      } else {
        // Few of the logits stay (top_p 0.9 leaves a twentieth of a normal
        // row): those that do are moved together at the end of the wave's
        // buffer first, so that fp64 is done for them alone (64 such rows of
        // 262144: 57 us without it).
        uint2* const end = gather.buf + 1023;
        int m = 0;
        for_group(z, gp, a.vocab, group, [&](const float (&v)[kSide], int i) {
#pragma unroll
          for (int j = 0; j < kSide; ++j) {
            const uint32_t k = order_key(v[j]);
            gather.add(k <= b.sure && ((k > b.a_lo && k <= b.a_hi) || (k > b.b_lo && k <= b.b_hi)), k, i + 64 * j);
            const bool stays = k > b.sure && !(v[j] < far);
            const u64 who = __ballot(stays);
            if (stays) end[-m - __popcll(who & ((1ull << lane) - 1))].x = __builtin_bit_cast(uint32_t, v[j]);
            m += __popcll(who);
          }
        }, [&] {
          gather.flush(w);
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          for (int at = lane; at - lane < m; at += 64 * kSide) {
            float v[kSide];
            double x[kSide];
#pragma unroll
            for (int j = 0; j < kSide; ++j) v[j] = at + 64 * j < m ? __builtin_bit_cast(float, end[-at - 64 * j].x) : in.wt.z_max;
            in.wt.weights(v, x);
#pragma unroll
            for (int j = 0; j < kSide; ++j) sum += at + 64 * j < m && x[j] >= f.min_p ? fixed(x[j]) : 0;
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          m = 0;
        });
      }
    }
    sum = wave_sum(sum);
    if (lane == 0) w.group_sum[group] = sum;
  }
}

// A workgroup finds where a row's borders lie among the `n` tokens of its list:
// it keeps the tokens ranked up to (key_cut, idx_cut), but for those that min_p
// leaves out. `sums`: the weight that stays of each group (complete after the
// next barrier).
__device__ __forceinline__ void cut_row(Shared& sh, u64* sums, const Filters& f, const RowInfo& in, const RowWork& w,
                                        const float* z, int vocab, uint32_t n, uint32_t& key_cut, int& idx_cut) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const GroupPlan gp = group_plan(vocab);
  const Weights& wt = in.wt;
  Borders b = {};
  Steps st;
  if (f.by_list()) {
    b.sure = in.max_key, b.b_lo = in.floor_key - 1, b.b_hi = in.max_key;
    b.k_rest = min(u64(f.top_k), u64(n));
  } else if (f.borders()) {
    st.load(w);
    b = borders_of(f, st);
  }
  if (t < kGroups) sums[t] = t < gp.groups && !f.by_list() ? w.group_sum[t] : 0;
  key_cut = b.sure + 1;
  idx_cut = 0x7FFFFFFF;
  auto kept = [&](uint32_t k, int i) { return k > key_cut || (k == key_cut && i <= idx_cut); };
  if (n > 0) {
    uint2 mine[kPerThread];
    u64 mine_w[kPerThread];
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const uint32_t at = e * kSampleThreads + t;
      mine[e] = at < min(n, uint32_t(kList)) ? w.list[at] : make_uint2(0u, 0u);
    }
    auto weigh = [&](auto count) {
      constexpr int N = decltype(count)::value;
      float v[N];
      double x[N];
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = mine[e].x ? key_value(mine[e].x) : wt.z_max;
      wt.weights(v, x);
#pragma unroll
      for (int e = 0; e < N; ++e) mine_w[e] = x[e] >= f.min_p ? fixed(x[e]) : fixed(x[e]) | kLight;
    };
#pragma unroll
    for (int e = 1; e < kPerThread; ++e) mine_w[e] = 0;
    if (n <= kSampleThreads) weigh(std::integral_constant<int, 1>{});
    else weigh(std::integral_constant<int, kPerThread>{});
    // the tokens with keys in (lo, hi]: from the list, or where it has no
    // room for them all, from the row
    auto between = [&](uint32_t lo, uint32_t hi) {
      return [&, lo, hi](auto each) {
        if (n <= kList) {
#pragma unroll
          for (int e = 0; e < kPerThread; ++e)
            if (mine[e].x > lo && mine[e].x <= hi) each(mine[e].x, int(mine[e].y), mine_w[e]);
        } else {
          for (int i = t; i < vocab; i += kSampleThreads) {
            const uint32_t k = order_key(z[i]);
            if (k > lo && k <= hi) {
              const double x = wt.weight(key_value(k));
              each(k, i, x >= f.min_p ? fixed(x) : fixed(x) | kLight);
            }
          }
        }
      };
    };
    u64 whole = b.above_k;  // weight of what top_k leaves
    if (b.k_rest > 0) {
      find_cut<false>(sh, b.k_rest, b.b_lo + 1, b.b_hi, wt, between(b.b_lo, b.b_hi), key_cut, idx_cut);
      if (f.top_p < 1.0f) {
        u64 s = 0;
        between(b.b_lo, b.b_hi)([&](uint32_t k, int i, u64 x) {
          if (kept(k, i)) s += x & ~kLight;
        });
        s = wave_sum(s);
        if (lane == 0) sh.wave[wave] = s;
        __syncthreads();
        for (int i = 0; i < kSampleWaves; ++i) whole += sh.wave[i];
      }
    }
    if (f.top_p < 1.0f) {
      u64 target = top_p_target(f.top_p, whole);
      uint32_t lo = b.b_lo, hi = b.b_hi;
      if (!f.by_list()) {
        const Steps::At at = st.at_weight(target);
        lo = st.key_below(at.step), hi = at.key;
        target -= at.before;
      }
      find_cut<true>(sh, target, lo + 1, hi, wt, between(lo, hi), key_cut, idx_cut);
    }
    // what the list's tokens add to their groups
    between(0, b.sure)([&](uint32_t k, int i, u64 x) {
      if (kept(k, i) && !(x & kLight)) atomicAdd(&sums[i / gp.per], x);
    });
  }
}

// The drawn number's place in `whole`.
__device__ __forceinline__ u64 drawn_at(float uf, u64 whole) {
  const double u = uf > 0.0f ? fmin(double(uf), 1.0) : 0.0;
  const u64 t = u64(u * double(whole));
  return t < whole ? t : whole - 1;
}

__device__ __forceinline__ float share_of(double x, u64 whole) { return float(x * double(1ull << kFracBits) / double(whole)); }

}  // namespace q4dec
