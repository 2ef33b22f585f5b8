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

struct Weights {
  double cap, inv_t, top;  // top = cap * tanh(z_max / cap)
  float z_max;
  __device__ __forceinline__ double capped(float z) const { return cap > 0.0 ? cap * tanh(double(z) / cap) : double(z); }
  // exp(l - l_max); 1 for the largest logit, also where it is +infinity
  __device__ __forceinline__ double weight(float z) const {
    return z == z_max ? 1.0 : exp((capped(z) - top) * inv_t);
  }
};

__device__ __forceinline__ u64 fixed(double w) { return u64(__double2ull_rn(w * double(1ull << kFracBits))); }

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
  uint32_t key[kSampleWaves];
  int idx[kSampleWaves];
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
// `target` (1 <= target <= the measure's whole sum).
template <bool WEIGHTED>
__device__ __forceinline__ void find_cut(Shared& sh, const float* z, int vocab, const Weights& wt, u64 target,
                                         uint32_t& key_cut, int& idx_cut) {
  uint32_t key = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < vocab; i += kSampleThreads) {
      const uint32_t k = order_key(z[i]);
      if (k == 0 || (shift < 24 && (k >> (shift + 8)) != (key >> (shift + 8)))) continue;
      const u64 m = WEIGHTED ? fixed(wt.weight(z[i])) : 1ull;
      if (m) atomicAdd(&sh.hist[(k >> shift) & 255u], m);
    }
    find_digit<false>(sh, target);
    key |= sh.digit << shift;
    target = sh.rest;
  }
  // the ties of that key, by index: each weighs the same
  const uint32_t bits = key & 0x80000000u ? key & 0x7FFFFFFFu : ~key;
  u64 ties = 1;
  if (WEIGHTED) {
    const u64 m = fixed(wt.weight(__builtin_bit_cast(float, bits)));
    ties = (target + m - 1) / m;
  } else {
    ties = target;
  }
  uint32_t idx = 0;
  for (int shift = 16; shift >= 0; shift -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < vocab; i += kSampleThreads)
      if (order_key(z[i]) == key && (uint32_t(i) >> (shift + 8)) == (idx >> (shift + 8)))
        atomicAdd(&sh.hist[(uint32_t(i) >> shift) & 255u], 1ull);
    find_digit<true>(sh, ties);
    idx |= sh.digit << shift;
    ties = sh.rest;
  }
  key_cut = key;
  idx_cut = int(idx);
}

__global__ __launch_bounds__(kSampleThreads) void sample_row_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int r = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float* z = a.logits + size_t(r) * a.row_stride;

  // first-ranked token
  uint32_t best = 0;
  int bidx = -1;
  for (int i = threadIdx.x; i < a.vocab; i += kSampleThreads) {
    const uint32_t k = order_key(z[i]);
    if (k > best) best = k, bidx = i;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const uint32_t ok = __shfl_xor(best, off);
    const int oi = __shfl_xor(bidx, off);
    if (ok > best || (ok == best && ok != 0 && oi < bidx)) best = ok, bidx = oi;
  }
  if (lane == 0) sh.key[wave] = best, sh.idx[wave] = bidx;
  __syncthreads();
  best = sh.key[0], bidx = sh.idx[0];
  for (int w = 1; w < kSampleWaves; ++w)
    if (sh.key[w] > best || (sh.key[w] == best && best != 0 && sh.idx[w] < bidx)) best = sh.key[w], bidx = sh.idx[w];
  const float heat = a.temperature ? a.temperature[r] : 1.0f;
  if (best == 0 || !(heat > 0.0f)) {
    if (threadIdx.x == 0) {
      a.idx_out[r] = bidx;
      if (a.prob_out) a.prob_out[r] = best == 0 ? NAN : 1.0f;
    }
    return;
  }
  Weights wt;
  wt.cap = double(a.cap);
  wt.inv_t = 1.0 / double(heat);
  wt.z_max = __builtin_bit_cast(float, best & 0x80000000u ? best & 0x7FFFFFFFu : ~best);
  wt.top = wt.capped(wt.z_max);

  uint32_t key_cut = 0;  // everything
  int idx_cut = 0x7FFFFFFF;
  auto kept = [&](uint32_t k, int i) { return k > key_cut || (k == key_cut && i <= idx_cut); };
  // sums a value over the workgroup
  auto total = [&](u64 v) {
    v = wave_sum(v);
    __syncthreads();
    if (lane == 0) sh.wave[wave] = v;
    __syncthreads();
    u64 s = 0;
    for (int w = 0; w < kSampleWaves; ++w) s += sh.wave[w];
    return s;
  };

  const int top_k = a.top_k ? a.top_k[r] : 0;
  if (top_k > 0 && top_k < a.vocab) {
    u64 n = 0;
    for (int i = threadIdx.x; i < a.vocab; i += kSampleThreads) n += order_key(z[i]) != 0;
    if (total(n) > u64(top_k)) find_cut<false>(sh, z, a.vocab, wt, u64(top_k), key_cut, idx_cut);
  }
  const float top_p = a.top_p ? a.top_p[r] : 1.0f;
  if (top_p < 1.0f) {
    u64 s = 0;
    for (int i = threadIdx.x; i < a.vocab; i += kSampleThreads) {
      const uint32_t k = order_key(z[i]);
      if (k != 0 && kept(k, i)) s += fixed(wt.weight(z[i]));
    }
    s = total(s);
    const u64 target = u64(ceil(fmax(double(top_p), 0.0) * double(s)));
    find_cut<true>(sh, z, a.vocab, wt, target > 0 ? target : 1, key_cut, idx_cut);
  }
  const float mp = a.min_p ? a.min_p[r] : 0.0f;
  const double min_p = mp > 0.0f ? fmin(double(mp), 1.0) : 0.0;
  auto drawn_weight = [&](int i) {
    const uint32_t k = order_key(z[i]);
    if (k == 0 || !kept(k, i)) return u64(0);
    const double w = wt.weight(z[i]);
    return w >= min_p ? fixed(w) : u64(0);
  };

  // each wave sums its own stretch of the row; the stretch that the target
  // falls in is then walked in index order
  const int per = ((a.vocab + kSampleWaves - 1) / kSampleWaves + 63) / 64 * 64;
  const int lo = min(wave * per, a.vocab), hi = min(lo + per, a.vocab);
  u64 s = 0;
  for (int i = lo + lane; i < hi; i += 64) s += drawn_weight(i);
  s = wave_sum(s);
  __syncthreads();
  if (lane == 0) sh.wave[wave] = s;
  __syncthreads();
  u64 whole = 0, before = 0;
  for (int w = 0; w < kSampleWaves; ++w) {
    if (w < wave) before += sh.wave[w];
    whole += sh.wave[w];
  }
  const float uf = a.u[r];
  const double u = uf > 0.0f ? fmin(double(uf), 1.0) : 0.0;
  u64 target = u64(u * double(whole));
  if (target >= whole) target = whole - 1;
  if (target < before || target >= before + s) return;
  for (int base = lo; base < hi; base += 64) {
    const u64 w = base + lane < hi ? drawn_weight(base + lane) : 0;
    u64 upto = w;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const u64 o = __shfl_up(upto, off);
      if (lane >= off) upto += o;
    }
    const u64 hit = __ballot(before + upto > target);
    if (hit) {
      if (lane == int(__ffsll(hit)) - 1) {
        a.idx_out[r] = base + lane;
        if (a.prob_out) a.prob_out[r] = float(wt.weight(z[base + lane]) * double(1ull << kFracBits) / double(whole));
      }
      return;
    }
    before += __shfl(upto, 63);
  }
}

}  // namespace q4dec

extern "C" size_t sample_logits_workspace_bytes(int64_t n_rows, int64_t vocab) { return 0; }

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
  hipLaunchKernelGGL(sample_row_kernel, dim3(unsigned(n_rows)), dim3(kSampleThreads), 0,
                     static_cast<hipStream_t>(stream), a);
  return launch_status(name);
}
