// paged_attention: softmax(scale q k^T) v of the new tokens of several
// sequences over their paged keys and values (causal, optional window,
// grouped heads), in base 2: p_j = 2^(s_j - m) with s = scale * log2(e) * q.k
// and the running maximum m; sums of p and of p v are rescaled when m grows.
//
// The rows of one sequence and key/value head are its new tokens times its
// group of query heads (row = token * group + head of the group), so the
// keys and values are read once for all of them.
//
// Few rows (decode, drafted tokens): attn_few_kernel. Bound by reading the
// cache, so keys and values go from memory straight into matrix-core
// operands, no LDS on the way:
//  - scores come transposed, S^T = K Q^T: a lane's 16-byte piece of a key row
//    is its A operand as it is. Lane (c, g) (c = lane % 16, g = lane / 16)
//    then holds for row c of Q the scores of keys 4g .. 4g+3 of each 16;
//  - O^T = V^T P^T sums over keys, and the order of a sum's terms is free: the
//    contraction slots of lane group g are given the keys 4g .. 4g+3 of each
//    16, so the probabilities are the B operand where they are. The A operand
//    wants one column of V for those keys: the lane reads a piece of each of
//    its 4 (or 8) rows and transposes it in registers (v_perm, half an
//    instruction per element; the VALU has room to spare here).
// The work, blocks of keys of every (sequence, key/value head, 16 rows) in
// turn, is cut into equal stretches, one a workgroup, from the lengths on the
// device: a batch of unlike lengths fills the card as one long sequence does,
// and a captured call stays balanced when its lengths change. A unit that
// several workgroups share is joined by attn_join_kernel in a fixed order.
// Measured: one token over 131072 keys of 512 57 us and 9 us to join (4.7
// TB/s of keys and values; a large copy moves 5.1), 48 tokens over e4m3 keys
// of 256 54 and 5 us (4.4 TB/s), 16 over 4096 keys of 128 54 us in all (5.0
// TB/s), one token's window of 512 8 and 4 us: one chain of loads, each lookup
// of a page and Q waited for on the way, and two launches.
#include <math.h>

#include <type_traits>

#include "q4dec_internal.h"
#include "q4dec_serve.h"
#include "serve_internal.h"

namespace q4dec {
Q4DEC_DEBUG_READER(paged_attention)

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;

struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* q_starts;
  const int32_t* kv_lens;
  int32_t* err;
  int64_t table_stride;
  int n_seq, n_tok, n_q, n_kv, group, n_pages, page_shift;
  int max_q, max_kv;
  int64_t window;
  float scale;
};

// Bounds of sequence b; false if they are not valid.
__device__ __forceinline__ bool sequence_of(const AttnArgs& a, int b, int& start, int& q_len, int& kv_len) {
  start = a.q_starts[b];
  q_len = int(uint32_t(a.q_starts[b + 1]) - uint32_t(start));
  kv_len = a.kv_lens[b];
  const bool ok = start >= 0 && q_len >= 0 && start <= a.n_tok && q_len <= a.n_tok - start && q_len <= a.max_q &&
                  kv_len >= 0 && kv_len <= a.max_kv;
  return ok;
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFewRows = 16;  // rows of a tile of attn_few_kernel

// What one workgroup's rows r0 .. r0 + n - 1 of (sequence b) see: positions
// [lo, hi), the last row's first being lo_max, the first row's end hi_min.
struct Span {
  int lo, hi, lo_max, hi_min;
};
// A value that all lanes agree on, in a scalar register: the compiler does not
// see through the search for a workgroup's stretch that it is one, and would
// keep it, and every address made from it, in vector registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ Span uniform(const Span& s) {
  return {uniform(s.lo), uniform(s.hi), uniform(s.lo_max), uniform(s.hi_min)};
}
__device__ __forceinline__ Span span_of(const AttnArgs& a, int q_len, int kv_len, int first_row, int last_row) {
  const int p0 = kv_len - q_len + first_row / a.group, p1 = kv_len - q_len + last_row / a.group;
  auto low = [&](int p) { return a.window > 0 && p >= a.window ? int(p - a.window + 1) : 0; };
  return {low(p0), p1 + 1, low(p1), p0 + 1};
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
// two e4m3 values (the low or high half of w) as a bf16 pair, exact
template <bool HI>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}
// not 0 if one of the elements is NaN or infinite: an exponent (e4m3: all bits
// but the sign) of ones carries into the sign bit when one is added at its end
template <bool F8>
__device__ __forceinline__ uint32_t nonfinite(uint32_t x) {
  return F8 ? ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u : ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

// the bits of the elements that nonfinite() marked
template <bool F8>
__device__ __forceinline__ uint32_t spread(uint32_t n) {
  return F8 ? (n >> 7) * 0xFFu : (n >> 15 & 1u) * 0xFFFFu | (n >> 31) * 0xFFFF0000u;
}

__device__ __forceinline__ f32x4 mfma16(const uint32_t (&a)[4], const uint32_t (&b)[4], f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ f32x4 mfma16(const uint32_t (&a)[2], const uint32_t (&b)[2], f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a), __builtin_bit_cast(s16x4, b), c, 0, 0,
                                                   0);
}

// Partial results: sums of p v relative to m, and (m, sum of p). A workgroup
// has two slots, for the first unit of its stretch and for the last one; the
// one whose stretch holds a shared unit's beginning says where its pieces are:
// in its slot `slot` and in slot 0 of the next pieces - 1 workgroups.
struct Owned {
  int wg, pieces, slot;  // pieces = 0: it owns none
  int start, h, r0, n;
};
struct Partials {
  float* o;
  float2* ml;
  Owned* owned;  // NULL: nothing to join (few rows: one workgroup; many: one a unit)
  // Where units are fewer than workgroups `owned` has one entry a unit (of
  // the most there can be), else one a workgroup.
  int tiles;  // 0, or tiles a head can have: by unit
  int rows;   // of a slot
  __device__ __forceinline__ void own(const Owned& o, bool begins, bool ends_stretch, int b, int n_kv, int tile) const {
    if (!owned || threadIdx.x != 0) return;
    if (tiles) {
      if (begins) owned[(size_t(b) * n_kv + o.h) * tiles + tile] = o;
    } else if (ends_stretch) {
      owned[o.wg] = o;
    }
  }
  // the entry of a join's workgroup; pieces = 0 where there is nothing to do
  __device__ __forceinline__ Owned find(const AttnArgs& a, int at, int tile_rows) const {
    if (tiles) {
      int start, q_len, kv_len;
      const int b = at / (a.n_kv * tiles), tile = at % tiles;
      if (!sequence_of(a, b, start, q_len, kv_len) || tile * tile_rows >= q_len * a.group) return Owned{0, 0, 0, 0, 0, 0, 0};
    }
    return owned[at];
  }
};
// of a unit whose blocks up to k1 are in this stretch, the last of it if not all
__device__ __forceinline__ int pieces_of(bool begins, int k1, int blocks, int per) {
  return begins && k1 < blocks ? 1 + (blocks - k1 + per - 1) / per : 0;
}

constexpr int few_waves(bool whole) { return whole ? 2 * kAttnWaves : kAttnWaves; }

template <int D, bool F8, bool WHOLE>
struct FewGeometry {
  static constexpr int WAVES = few_waves(WHOLE);
  static constexpr int TS = D >= 256 && !F8 ? 1 : 2;  // groups of 16 keys in a step (what registers allow)
  static constexpr int CW = F8 ? (D / 16 < 16 ? D / 16 : 16) : (D / 16 < 8 ? D / 16 : 8);  // columns of V a lane reads
  static constexpr int NB = D / (16 * CW);
  static constexpr int KW = F8 ? D / 64 : D / 32;  // 16-byte pieces of a key row per lane
  static constexpr int VW = CW * (F8 ? 1 : 2) / 4;  // dwords of a piece of V
  static constexpr int kBlock = 16 * TS * WAVES;  // keys: a step of every wave
};

// N dwords by the widest loads
template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

// ---- values that are not finite
// The products cannot be trusted with them: a probability of zero, a key that a
// row does not see or (few rows) the second part of a probability makes NaN of
// an infinity. Where a wave's sums have come out as NaN, or values were left
// out on the way, it looks at its keys once more after it has put the sums
// down: those of a row and column that met such values become their sum.

// x * f, but an infinity is one whatever its weight: for a join's second try,
// where its sums are NaN.
__device__ __forceinline__ f32x4 scaled(f32x4 x, float f) {
  f32x4 y = x * f;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = fabsf(x[e]) == INFINITY ? x[e] : y[e];
  return y;
}
__device__ __forceinline__ bool any_nan(f32x4 x) { return (x[0] != x[0]) | (x[1] != x[1]) | (x[2] != x[2]) | (x[3] != x[3]); }

// For `count` keys key_of(0 .. count - 1), those below `hi`, and the columns
// col .. col + COLS - 1: put(row, column, x, anew) for each value x that is not finite
// and each of the rows 0 .. rows - 1 that sees its key, once with `anew` (the
// sum starts with it) and once without. Lane r holds what row r sees: the
// positions lo_row .. lo_row + row_wide - 1. e4m3 has no infinity, and there is
// nothing that a NaN does not make NaN: there the sums are only added to.
template <int D, bool F8, int COLS, class KEY, class PUT>
__device__ __forceinline__ void put_nonfinite(const AttnArgs& a, const int32_t* table, int h, int col, int rows, int lo_row,
                                              uint32_t row_wide, int count, int hi, KEY key_of, PUT put) {
  constexpr int ES = F8 ? 1 : 2;
  const int lane = threadIdx.x & 63, page_mask = (1 << a.page_shift) - 1;
  auto row_of = [&](int page, int key) {
    return a.v_cache + ((((size_t(page) * a.n_kv + h) << a.page_shift) + size_t(key & page_mask)) * D + col) * ES;
  };
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // the wave's sums are in their place
  __builtin_amdgcn_wave_barrier();
#pragma unroll 1
  for (int anew = F8 ? 0 : 1; anew >= 0; --anew) {
#pragma unroll 1
    for (int base = 0; base < count; base += 64) {  // a key a lane
      const int key = key_of(base + lane);
      const int page = table[min(key, hi - 1) >> a.page_shift];
      const bool there = (base + lane < count) & (key < hi) & (uint32_t(page) < uint32_t(a.n_pages));
      const uint8_t* v = row_of(there ? page : 0, there ? key : 0);
      uint32_t bad = 0;
#pragma unroll 4
      for (int i = 0; i < COLS * ES; i += 16) {
        const uint4 x = *reinterpret_cast<const uint4*>(v + i);
        bad |= nonfinite<F8>(x.x) | nonfinite<F8>(x.y) | nonfinite<F8>(x.z) | nonfinite<F8>(x.w);
      }
#pragma unroll 1
      for (unsigned long long who = __ballot(there & (bad != 0)); who; who &= who - 1) {
        const int src = __ffsll(who) - 1, k = __builtin_amdgcn_readlane(key, src);
        const uint8_t* from = row_of(__builtin_amdgcn_readlane(page, src), k);
        const unsigned long long sees = __ballot((lane < rows) & (uint32_t(k - lo_row) < row_wide));
#pragma unroll 1
        for (int d = lane; d < COLS; d += 64) {
          const float x = F8 ? __builtin_amdgcn_cvt_f32_fp8(int(from[d]), 0)
                             : bf16_to_f32(reinterpret_cast<const uint16_t*>(from)[d]);
          if (isfinite(x)) continue;
#pragma unroll 1
          for (unsigned long long r = sees; r; r &= r - 1) put(__ffsll(r) - 1, d, x, anew != 0);
        }
      }
    }
  }
}

// ---- scores that are all -infinity
// Such a row has no largest score and a sum of weights of zero, as one that sees
// nothing has, but its quotient is 0 / 0. Where a lane's row has no largest
// score although some of the keys [k_lo, k_hi) lie within the positions that it
// may see, this says whether one of them lies in a page that is there. Partial
// results carry it as a sum of weights of kBlank, which weighs nothing beside a
// piece that has a largest score.
constexpr float kBlank = 1.0f;
// (its positions lo_row .. lo_row + row_wide - 1 end before k_hi)
__device__ __forceinline__ bool reaches(int lo_row, uint32_t row_wide, int k_lo) {
  return (row_wide > 0) & (lo_row + int(row_wide) > k_lo);
}
__device__ __forceinline__ bool sees_some(const AttnArgs& a, const int32_t* table, int lo_row, uint32_t row_wide, int k_lo,
                                          int k_hi) {
  const int lane = threadIdx.x & 63, last = (k_hi - 1) >> a.page_shift;
  const int from = max(lo_row, k_lo) >> a.page_shift, to = (lo_row + int(row_wide) - 1) >> a.page_shift;
  unsigned long long seen = 0;
#pragma unroll 1
  for (int base = k_lo >> a.page_shift; base <= last; base += 64) {  // a page a lane
    const uint32_t page = table[min(base + lane, last)];
    const unsigned long long good = __ballot((base + lane <= last) & (page < uint32_t(a.n_pages)));
    const int lo = max(from - base, 0), hi = min(to - base, 63);
    seen |= lo <= hi ? good & (~0ull >> (63 - hi)) & (~0ull << lo) : 0ull;
  }
  return seen != 0;
}

// ---- the cut into workgroups
// Each wave derives it for itself, a sequence a lane: the host sees to it that
// the blocks over all sequences stay below 2^31.

// sum of v over the lanes up to this one
__device__ __forceinline__ int lanes_upto(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15, 31
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// One sequence's units (key/value heads times tiles of 16 rows) and blocks of
// keys in each (all the positions that any row sees, at least one block: a
// row that sees nothing has to be written too).
struct SeqWork {
  int start, q_len, kv_len, units, blocks;
  Span span;
};
template <int BLOCK>
__device__ __forceinline__ SeqWork seq_work(const AttnArgs& a, bool ok, int start, int q_len, int kv_len) {
  SeqWork w;
  w.start = start, w.q_len = ok ? q_len : 0, w.kv_len = kv_len;
  const int rows = w.q_len * a.group;
  w.units = a.n_kv * ((rows + kFewRows - 1) / kFewRows);
  w.span = span_of(a, w.q_len, kv_len, 0, max(rows - 1, 0));
  w.blocks = rows > 0 ? max((w.span.hi - (w.span.lo & ~15) + BLOCK - 1) / BLOCK, 1) : 0;
  return w;
}
template <int BLOCK>
__device__ __forceinline__ SeqWork seq_work(const AttnArgs& a, int b) {
  int start = 0, q_len = 0, kv_len = 0;
  const bool ok = b < a.n_seq && sequence_of(a, b, start, q_len, kv_len);
  if (!ok && b < a.n_seq && a.err) *a.err = 1;
  return seq_work<BLOCK>(a, ok, start, q_len, kv_len);
}

// The blocks of all sequences and of one workgroup's stretch.
struct Cut {
  int total, per;
};
template <int BLOCK>
__device__ __forceinline__ Cut cut_of(const AttnArgs& a, int first64, int workgroups) {
  Cut c;
  c.total = __builtin_amdgcn_readlane(lanes_upto(first64), 63);
  for (int base = 64; base < a.n_seq; base += 64) {
    const SeqWork w = seq_work<BLOCK>(a, base + int(threadIdx.x & 63));
    c.total += __builtin_amdgcn_readlane(lanes_upto(w.units * w.blocks), 63);
  }
  c.per = __builtin_amdgcn_readfirstlane(int((uint32_t(c.total) + uint32_t(workgroups) - 1u) / uint32_t(workgroups)));
  if (c.per == 0) c.per = 1;
  return c;
}

// WHOLE: a workgroup takes one unit and all of its keys.
template <int D, bool F8, bool WHOLE>
__global__ __launch_bounds__(64 * few_waves(WHOLE), D >= 512 ? 1 : 2) void attn_few_kernel(AttnArgs a, Partials part,
                                                                                  int workgroups) {
  using G = FewGeometry<D, F8, WHOLE>;
  constexpr int TS = G::TS, CW = G::CW, NB = G::NB, KW = G::KW, VW = G::VW, ES = F8 ? 1 : 2, kBlock = G::kBlock, NW = G::WAVES;
  constexpr int NS = D / 32;  // contraction steps of a score
  constexpr int kStep = 16 * TS, kRowPad = D + 4;
  extern __shared__ float lds[];
  __shared__ float2 wave_ml[NW][16];
  __shared__ float row_l[16];
  __shared__ uint4 qf[NS][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  Q4_DCHECK(int(gridDim.x) <= workgroups && part.rows <= kFewRows, kDbgAttnGrid);

  // this workgroup's stretch: from block k0 of unit `unit` of sequence b on
  SeqWork sw;
  Cut cut = {0, 1};
  int b = 0, unit = 0, k0 = 0, left = 0;
  if constexpr (WHOLE) {
    const int tiles = workgroups / (a.n_seq * a.n_kv), tile = blockIdx.x % tiles, h = blockIdx.x / tiles % a.n_kv;
    b = blockIdx.x / tiles / a.n_kv;
    int start, q_len, kv_len;
    if (!sequence_of(a, b, start, q_len, kv_len)) {
      if (a.err && threadIdx.x == 0) *a.err = 1;
      return;
    }
    sw = seq_work<kBlock>(a, true, start, q_len, kv_len);
    if (tile >= sw.units / a.n_kv) return;
    unit = h * (sw.units / a.n_kv) + tile;
    left = sw.blocks;
  } else {
    sw = seq_work<kBlock>(a, lane);
    cut = cut_of<kBlock>(a, sw.units * sw.blocks, workgroups);
    const int64_t from64 = int64_t(blockIdx.x) * cut.per;
    if (from64 >= cut.total) {
      part.own(Owned{int(blockIdx.x), 0, 0, 0, 0, 0, 0}, false, true, 0, 0, 0);
      return;
    }
    const int from = int(from64);
    left = min(cut.per, cut.total - from);
    int skip = 0;
    for (int seen = 0;;) {
      const int cost = sw.units * sw.blocks, upto = seen + lanes_upto(cost);
      const unsigned long long hit = __ballot(upto - cost <= from && from < upto);
      if (hit) {
        const int src = __ffsll(hit) - 1;
        b += src;
        skip = from - __builtin_amdgcn_readlane(upto - cost, src);
        const int start = __builtin_amdgcn_readlane(sw.start, src), q_len = __builtin_amdgcn_readlane(sw.q_len, src);
        sw = seq_work<kBlock>(a, true, start, q_len, __builtin_amdgcn_readlane(sw.kv_len, src));
        break;
      }
      b += 64;
      if (b >= a.n_seq) return;  // (not reached: from < total)
      seen = __builtin_amdgcn_readlane(upto, 63);
      sw = seq_work<kBlock>(a, b + lane);
    }
    unit = __builtin_amdgcn_readfirstlane(int(uint32_t(skip) / uint32_t(sw.blocks)));
    k0 = skip - unit * sw.blocks;
  }

  for (bool first = true;; first = false) {
    // What a wave agrees on goes into scalar registers, so that its branches are
    // scalar too. At a branch of some lanes the compiler has lost values: see
    // Pages::checked, and a tuple of scores in accumulation registers of which
    // it set one element there for some lanes, and overwrote the other three.
    b = uniform(b), unit = uniform(unit), k0 = uniform(k0), left = uniform(left);
    sw = {uniform(sw.start), uniform(sw.q_len), uniform(sw.kv_len), uniform(sw.units), uniform(sw.blocks), uniform(sw.span)};
    const int k1 = left < sw.blocks - k0 ? k0 + left : sw.blocks;
    const bool whole = k0 == 0 && k1 == sw.blocks;
    const int tiles = sw.units / a.n_kv, h = unit / tiles, r0 = unit % tiles * kFewRows;
    const int start = sw.start, q_len = sw.q_len, kv_len = sw.kv_len;
    const int n = min(kFewRows, q_len * a.group - r0);
    const Span sp = span_of(a, q_len, kv_len, r0, r0 + n - 1);
    const int k_lo = (sw.span.lo & ~15) + k0 * kBlock;
    const int k_hi = min(sw.span.hi, (sw.span.lo & ~15) + k1 * kBlock);

    // this lane's row of Q (column c of the operand), and what it sees
    const bool live = c < n;
    const int row = r0 + min(c, n - 1), token = row / a.group, hq = h * a.group + row % a.group;
    const int p_row = live ? kv_len - q_len + token : -1;
    const int lo_row = a.window > 0 && p_row >= a.window ? int(p_row - a.window + 1) : 0;
    const uint32_t row_wide = max(min(p_row + 1, k_hi) - lo_row, 0);  // positions from lo_row on
    const uint16_t* q_row = a.q + (size_t(start + token) * a.n_q + hq) * D;
    // the B operands of the scores, the same for every wave, in lane order
    uint4 qv[(NS + NW - 1) / NW];
#pragma unroll
    for (int i = 0; i < (NS + NW - 1) / NW; ++i) {
      const int s = min(i * NW + wave, NS - 1);
      qv[i] = *reinterpret_cast<const uint4*>(q_row + (F8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g));
    }
    const float qs = a.scale * kLog2e * (F8 && a.k_scale ? a.k_scale[h] : 1.0f);

    const int32_t* table = a.page_table + b * a.table_stride;
    const int page_mask = (1 << a.page_shift) - 1;
    const size_t page_bytes = (size_t(a.n_kv) << a.page_shift) * (D * ES);
    const size_t head_bytes = (size_t(h) << a.page_shift) * (D * ES);
    // the page of the 16 keys from kb on; -1: nothing there to see
    auto page_of = [&](int kb) {
      if (kb >= k_hi) return -1;
      const int p = uniform(table[kb >> a.page_shift]);
      const bool good = uint32_t(p) < uint32_t(a.n_pages);
      if (!good && a.err) *a.err = 1;  // (by all lanes: see Pages::checked)
      return good ? p : -1;
    };
    auto offset_of = [&](int page, int kb) {
      return size_t(max(page, 0)) * page_bytes + head_bytes + size_t(page < 0 ? 0 : kb & page_mask) * (D * ES);
    };

    uint32_t kf[TS][KW][4], vf[4 * TS][NB][VW];
    auto load_k = [&](const int (&page)[TS], int kb) {
#pragma unroll
      for (int t = 0; t < TS; ++t) {
        const uint8_t* p = a.k_cache + offset_of(page[t], kb + 16 * t) + c * (D * ES) + 16 * g;
#pragma unroll
        for (int i = 0; i < KW; ++i) load_dwords<4>(p + 64 * i, kf[t][i]);
      }
    };
    auto load_v = [&](const int (&page)[TS], int kb) {
#pragma unroll
      for (int t = 0; t < TS; ++t) {
        const uint8_t* p = a.v_cache + offset_of(page[t], kb + 16 * t) + (4 * g) * (D * ES) + c * (CW * ES);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int i = 0; i < NB; ++i) load_dwords<VW>(p + r * (D * ES) + i * (16 * CW * ES), vf[4 * t + r][i]);
      }
    };

    f32x4 o[NB][CW];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < CW; ++j) o[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f;
    uint32_t odd = 0;  // set by a value left out (see below)

    auto step = [&](auto more_c, const int (&page)[TS], int kb, const int (&next)[TS], int kb_next) {
      constexpr bool MORE = decltype(more_c)::value;
      f32x4 s[TS];
#pragma unroll
      for (int t = 0; t < TS; ++t) s[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const uint4 qi = qf[i][lane];
        const uint32_t q4[4] = {qi.x, qi.y, qi.z, qi.w};
#pragma unroll
        for (int t = 0; t < TS; ++t) {
          if constexpr (F8) {
            const uint32_t w0 = kf[t][i >> 1][2 * (i & 1)], w1 = kf[t][i >> 1][2 * (i & 1) + 1];
            const uint32_t k4[4] = {e4m3_pair<false>(w0), e4m3_pair<true>(w0), e4m3_pair<false>(w1),
                                    e4m3_pair<true>(w1)};
            s[t] = mfma16(k4, q4, s[t]);
          } else {
            s[t] = mfma16(kf[t][i], q4, s[t]);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (MORE) load_k(next, kb_next);
      __builtin_amdgcn_sched_barrier(0);
      bool open = true;  // every row sees every key of the step
#pragma unroll
      for (int t = 0; t < TS; ++t) open = open && page[t] >= 0;
      open = open && kb >= sp.lo_max && kb + kStep <= min(sp.hi_min, k_hi);
#pragma unroll
      for (int t = 0; t < TS; ++t) {
        const uint32_t wide = page[t] >= 0 ? row_wide : 0u;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t at = uint32_t(kb + 16 * t + 4 * g + r - lo_row);
          s[t][r] = open || at < wide ? s[t][r] * qs : -INFINITY;
        }
      }
      float mx = m;
#pragma unroll
      for (int t = 0; t < TS; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) mx = fmaxf(mx, s[t][r]);  // (leaves a NaN score out; its p is NaN)
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float base = mx == -INFINITY ? 0.0f : mx;
      if (__ballot(mx > m)) {
        const float f = __builtin_amdgcn_exp2f(m - base);
        l *= f;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < CW; ++j) o[i][j] *= f;
        m = mx;
      }
      // the probabilities in two bf16 parts, so that their rounding adds
      // nothing to the output's own (the matrix cores are idle here anyway)
      uint32_t ph[2 * TS], pl[2 * TS];
#pragma unroll
      for (int t = 0; t < TS; ++t)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          const float p0 = __builtin_amdgcn_exp2f(s[t][r] - base), p1 = __builtin_amdgcn_exp2f(s[t][r + 1] - base);
          l += p0 + p1;
          const uint32_t hi = pack_bf16(p0, p1);
          ph[2 * t + r / 2] = hi;
          pl[2 * t + r / 2] = pack_bf16(p0 - bf16_to_f32(hi & 0xFFFFu), p1 - bf16_to_f32(hi >> 16));
        }
      if (!open) {
        // 0 * NaN is NaN: values at keys that no row sees become zero, and at
        // keys that only some see those that are not finite, added at the end
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = kb + 16 * t + 4 * g + r;
            const uint32_t any = page[t] >= 0 && uint32_t(key - sp.lo) < uint32_t(k_hi - sp.lo) ? ~0u : 0u;
            const uint32_t all = uint32_t(key - sp.lo_max) < uint32_t(max(sp.hi_min - sp.lo_max, 0)) ? ~0u : 0u;
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
              for (int w = 0; w < VW; ++w) {
                const uint32_t x = vf[4 * t + r][i][w] & any;
                const uint32_t out = nonfinite<F8>(x) & ~all;
                vf[4 * t + r][i][w] = x & ~spread<F8>(out);
                odd |= out;
              }
          }
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int w = 0; w < CW / 2; ++w) {  // columns 2w and 2w + 1 of the lane's piece
          uint32_t lo[2 * TS], hi[2 * TS];
#pragma unroll
          for (int kp = 0; kp < 2 * TS; ++kp) {
            uint32_t x0 = vf[2 * kp][i][F8 ? w >> 1 : w], x1 = vf[2 * kp + 1][i][F8 ? w >> 1 : w];
            if constexpr (F8) {
              x0 = w & 1 ? e4m3_pair<true>(x0) : e4m3_pair<false>(x0);
              x1 = w & 1 ? e4m3_pair<true>(x1) : e4m3_pair<false>(x1);
            }
            lo[kp] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
            hi[kp] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
          }
          o[i][2 * w] = mfma16(lo, ph, o[i][2 * w]);
          o[i][2 * w + 1] = mfma16(hi, ph, o[i][2 * w + 1]);
          o[i][2 * w] = mfma16(lo, pl, o[i][2 * w]);
          o[i][2 * w + 1] = mfma16(hi, pl, o[i][2 * w + 1]);
          __builtin_amdgcn_sched_barrier(0);
        }
      if constexpr (MORE) load_v(next, kb_next);
    };

    // The waves take the steps in turn, each at least one, of which it may see
    // nothing: with a branch round a wave that has none the compiler keeps
    // keys and values in scratch (512-wide heads, 122 registers).
    const int steps = k_hi > k_lo ? (k_hi - k_lo + kStep - 1) / kStep : 0;
    const int mine = steps > wave ? (steps - wave + NW - 1) / NW : 1;
    int kb = k_lo + wave * kStep;
    int page[TS], next[TS];
#pragma unroll
    for (int t = 0; t < TS; ++t) page[t] = page_of(kb + 16 * t);
    load_k(page, kb);
    load_v(page, kb);
#pragma unroll
    for (int t = 0; t < TS; ++t) next[t] = page_of(kb + NW * kStep + 16 * t);
#pragma unroll
    for (int i = 0; i < (NS + NW - 1) / NW; ++i)
      if (i * NW + wave < NS) qf[i * NW + wave][lane] = qv[i];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    for (int i = 1; i < mine; ++i) {
      const int kn = kb + NW * kStep;
      int after[TS];
#pragma unroll
      for (int t = 0; t < TS; ++t) after[t] = page_of(kn + NW * kStep + 16 * t);
      step(std::true_type{}, page, kb, next, kn);
      kb = kn;
#pragma unroll
      for (int t = 0; t < TS; ++t) page[t] = next[t], next[t] = after[t];
    }
    step(std::false_type{}, page, kb, next, kb);
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    // join the waves: sums relative to the largest of their maxima
    if (g == 0) wave_ml[wave][c] = make_float2(m, l);
    __syncthreads();
    float mt = -INFINITY, lt = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) mt = fmaxf(mt, wave_ml[w][c].x);
    const float bt = mt == -INFINITY ? 0.0f : mt;
#pragma unroll
    for (int w = 0; w < NW; ++w) lt += wave_ml[w][c].y * __builtin_amdgcn_exp2f(wave_ml[w][c].x - bt);
    const bool blank = (mt == -INFINITY) & (lt == 0.0f) & reaches(lo_row, row_wide, k_lo);
    if (__ballot(blank))
      lt = (blank & sees_some(a, table, lo_row, row_wide, k_lo, k_hi)) ? (whole ? NAN : kBlank) : lt;
    const float f = __builtin_amdgcn_exp2f(m - bt);
    float spoilt = 0.0f;  // NaN if one of the sums is
    if (live) {
      float* dst = lds + (wave * n + c) * kRowPad;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < CW; j += 4) {
            const f32x4 x = {o[i][j][r] * f, o[i][j + 1][r] * f, o[i][j + 2][r] * f, o[i][j + 3][r] * f};
            *reinterpret_cast<f32x4*>(dst + i * 16 * CW + CW * (4 * g + r) + j) = x;
            if constexpr (!F8) spoilt = fmaf(x[0] + x[1] + (x[2] + x[3]), 0.0f, spoilt);
          }
      if (l != l) spoilt = 0.0f;  // (all of the row is NaN)
    }
    if (k_hi > k_lo && __ballot((odd != 0) | (spoilt != spoilt)))
      put_nonfinite<D, F8, D>(
          a, table, h, 0, n, lo_row, row_wide, mine * kStep, k_hi,
          [&](int i) { return k_lo + (i / kStep * NW + wave) * kStep + i % kStep; },
          [&](int row, int d, float x, bool anew) {
            float* at = lds + (wave * n + row) * kRowPad + d;
            *at = anew ? 0.0f : *at + x;
          });
    const size_t slot = size_t(blockIdx.x) * 2 + (first ? 0 : 1);
    if (wave == 0 && g == 0) {
      row_l[c] = lt;
      if (!whole && live) part.ml[slot * kFewRows + c] = make_float2(mt, lt);
    }
    __syncthreads();
    const float vs = F8 && a.v_scale ? a.v_scale[h] : 1.0f;
    for (int e = threadIdx.x * 4; e < n * D; e += 64 * NW * 4) {
      const int rr = e / D, d = e % D;
      f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NW; ++w) x += *reinterpret_cast<const f32x4*>(lds + (w * n + rr) * kRowPad + d);
      if (!whole) {
        *reinterpret_cast<f32x4*>(part.o + (slot * part.rows + rr) * D + d) = x;
      } else {
        const float inv = row_l[rr] == 0.0f ? 0.0f : vs / row_l[rr];
        const int t = (r0 + rr) / a.group, q = h * a.group + (r0 + rr) % a.group;
        *reinterpret_cast<uint2*>(a.out + (size_t(start + t) * a.n_q + q) * D + d) =
            make_uint2(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv));
      }
    }

    left -= k1 - k0;
    part.own(Owned{int(blockIdx.x), pieces_of(k0 == 0, k1, sw.blocks, cut.per), first ? 0 : 1, start, h, r0, n}, k0 == 0,
             left <= 0, b, a.n_kv, r0 / kFewRows);
    if (left <= 0) return;
    k0 = 0;
    if (++unit == sw.units) {
      unit = 0;
      do {
        sw = seq_work<kBlock>(a, ++b);
      } while (sw.units == 0);  // (left > 0: there is one)
    }
    __syncthreads();  // LDS is free again
  }
}

// Joins the pieces of a unit that several workgroups share, in their order:
// one workgroup per row and COLS columns, groups of lanes taking the pieces in
// turn, four columns a lane. (The unit is the grid's slow index: workgroups
// that have something to do may be far apart, often by a multiple of 8, and
// would all run on one die.)
template <int D, int COLS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void attn_join_kernel(AttnArgs a, Partials part) {
  constexpr int kLanes = COLS / 4 < 64 ? COLS / 4 : 64, kTakers = WAVES * 64 / kLanes, kPieces = COLS / (4 * kLanes);
  __shared__ __align__(16) float sum[kTakers][COLS];
  const int lane = threadIdx.x & 63, taker = threadIdx.x / kLanes, col = threadIdx.x % kLanes * 4;
  const int rr = blockIdx.x / (D / COLS), c0 = blockIdx.x % (D / COLS) * COLS;
  const Owned u = part.find(a, blockIdx.y, kFewRows);
  if (rr >= u.n || u.pieces == 0) return;
  const int n = u.pieces;
  auto slot_of = [&](int i) { return size_t(u.wg + i) * 2 + (i == 0 ? u.slot : 0); };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 64) m = fmaxf(m, part.ml[slot_of(i) * kFewRows + rr].x);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  const float base = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  for (int i = lane; i < n; i += 64) {
    const float2 v = part.ml[slot_of(i) * kFewRows + rr];
    l += v.y * __builtin_amdgcn_exp2f(v.x - base);
  }
  l = group_sum<64>(l);
  if (m == -INFINITY) {
    bool blank = false;
    for (int i = lane; i < n; i += 64) blank |= part.ml[slot_of(i) * kFewRows + rr].y != 0.0f;
    if (__ballot(blank)) l = NAN;
  }
  f32x4 x[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) x[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int i = taker; i < n; i += kTakers) {
    const float f = __builtin_amdgcn_exp2f(part.ml[slot_of(i) * kFewRows + rr].x - base);
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
      x[p] += f * *reinterpret_cast<const f32x4*>(part.o + (slot_of(i) * part.rows + rr) * D + c0 + p * 256 + col);
  }
#pragma unroll
  for (int p = 0; p < kPieces; ++p)
    if (__ballot(any_nan(x[p]))) {
      x[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int i = taker; i < n; i += kTakers)
        x[p] += scaled(*reinterpret_cast<const f32x4*>(part.o + (slot_of(i) * part.rows + rr) * D + c0 + p * 256 + col),
                       __builtin_amdgcn_exp2f(part.ml[slot_of(i) * kFewRows + rr].x - base));
    }
#pragma unroll
  for (int p = 0; p < kPieces; ++p) *reinterpret_cast<f32x4*>(&sum[taker][p * 256 + col]) = x[p];
  __syncthreads();
  const float scale = l == 0.0f ? 0.0f : (a.v_scale ? a.v_scale[u.h] : 1.0f) / l;
  const int t = (u.r0 + rr) / a.group, q = u.h * a.group + (u.r0 + rr) % a.group;
  for (int d = threadIdx.x; d < COLS; d += 64 * WAVES) {
    float y = 0.0f;
#pragma unroll 16
    for (int i = 0; i < kTakers; ++i) y += sum[i][d];
    a.out[(size_t(u.start + t) * a.n_q + q) * D + c0 + d] = f32_to_bf16_rne(y * scale);
  }
}

// ---------------------------------------------------------------- many rows
// Prefill chunks: attn_many_kernel, bound by the matrix cores and the
// softmax's VALU work. A workgroup of four waves takes 128 rows, 32 a wave,
// and walks over the keys in tiles that all four read from LDS (filled by
// direct loads one tile ahead, two buffers). As above the scores come
// transposed, S^T = K Q^T with v_mfma_f32_32x32x16: lane (c, h) (c = lane % 32,
// h = lane / 32) holds for its row c the scores of keys 8i + 4h .. 8i + 4h + 3,
// so a row's maximum is a chain in the lane and one swap with lane ^ 32, and
// the packed probabilities are the B operand of O^T = V^T P^T as they are:
// contraction slot j of half h stands for key 16 s + 8 (j / 4) + 4h + j % 4.
// V's operand for those keys is two transposing LDS reads (4 keys x 16
// columns per 16 lanes).
//
// LDS holds a tile's rows in 16-byte pieces, piece x of row r at x ^ f(r):
// 16 rows' equal pieces (K's read) and 8 rows' equal 64 bytes (V's) then lie
// in different banks. Direct loads fill LDS in lane order, so the lanes
// permute the source address instead.
// Measured: five chunks of 2048 tokens over up to 12288 keys, 32 heads of 128,
// 880 us (884 TFLOP/s; a large library product reaches 1184); the matrix cores
// are busy 50% of the cycles and the VALU about 60%, hardly at the same time.
// 256-wide heads 470 TFLOP/s, bf16 or e4m3: an output of 32 x 256 a wave leaves
// no registers to run a second tile's products beside a softmax, and where
// units are cut the partial results are as many bytes as the keys. 512-wide
// heads 250 to 270.
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kManyRows = 128;
constexpr float kLazy = 8.0f;  // the maximum is followed once it has grown by 2^8

template <int D>
struct ManyGeometry {
  // 512-wide heads: two waves share 32 rows, each with half of the columns
  // (an output of 32 x 512 would take every register); they add their halves
  // of the scores through LDS.
  static constexpr int PARTS = D > 256 ? 2 : 1;
  static constexpr int DW = D / PARTS;           // columns of a wave
  static constexpr int WAVES = 4 * PARTS, THREADS = 64 * WAVES;
  static constexpr int KT = D <= 128 ? 64 : 32;  // keys of a tile
  static constexpr int CH = D / 8;               // 16-byte pieces of a row
  static constexpr int NL = KT * CH / THREADS;   // pieces a thread loads
  static constexpr int kTileBytes = KT * D * 2;
  // Q operands (of DW / 16) that live in LDS where registers run out: a spill
  // to scratch would have its reload queue behind the next tile's loads
  static constexpr int QL = DW == 256 ? 3 : 0;
  static constexpr int kLds = 4 * kTileBytes + QL * WAVES * 1024;  // two buffers of K and V, Q
  static __device__ __forceinline__ int swizzle(int row) {
    return D == 64 ? ((row >> 1) & 1) << 2 | ((row >> 2) & 3) : (row & 3) << 2 | ((row >> 2) & 3);
  }
};

// The pages of 64 groups of 16 keys, a group a lane: looked up ahead in one
// load, not group by group, since each wait for a lookup is also one for all
// the keys and values asked for before it (five chunks over up to 12288 keys:
// 921 us instead of 1035).
struct Pages {
  int now, raw;  // of these 64 groups, checked; of the 64 after them, as read
  __device__ __forceinline__ static int read(const AttnArgs& a, const int32_t* table, int key, int k_hi) {
    return table[min(key, k_hi - 1) >> a.page_shift];  // (lengths of up to 2^30: key does not overflow)
  }
  // -1: nothing there to see
  __device__ __forceinline__ static int checked(const AttnArgs& a, int page, int key, int k_hi) {
    // Without a branch of some lanes: the compiler has put a register's spill
    // where such a branch had not yet joined, and the other lanes lost theirs.
    const bool in = key < k_hi, good = uint32_t(page) < uint32_t(a.n_pages);
    if (__ballot(in & !good) && a.err) *a.err = 1;
    return (in & good) ? page : -1;
  }
  __device__ __forceinline__ int at(int group) const { return __builtin_amdgcn_readlane(now, group); }
};

// 16 bytes a lane from global memory at `k` and at `v` (uniform) + `at` straight
// into LDS at `to_k` and `to_v` (uniform) + 16 lane. Written out because the
// compiler has every transposed read of LDS wait for all such loads that it
// knows of, those into the other buffer too. They write no register, and a
// count of loads in flight that leaves them out makes the compiler's own waits
// longer, never shorter. m0 is the compiler's: it gets back what it held (a
// load takes it when it is issued). (The wait states are those of a scalar
// register that a vector instruction may just have written, and of m0.)
__device__ __forceinline__ void load_to_lds(const uint8_t* k, const uint8_t* v, uint32_t at, uint8_t* to_k, uint8_t* to_v) {
  const uint32_t lds_k = uint32_t(uintptr_t((__attribute__((address_space(3))) void*)to_k));
  const uint32_t lds_v = uint32_t(uintptr_t((__attribute__((address_space(3))) void*)to_v));
  uint32_t held;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 4\n\t"
      "global_load_lds_dwordx4 %3, %4\n\t"
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %3, %5\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(held)
      : "s"(lds_k), "s"(lds_v), "v"(at), "s"(k), "s"(v)
      : "memory");
}

// One tile of 128 rows of a sequence and head: what its rows see, in blocks of
// a tile of keys (at least one: a row that sees nothing has to be written too).
struct TileWork {
  Span span;
  int n, blocks;
};
template <int KT>
__device__ __forceinline__ TileWork tile_work(const AttnArgs& a, int q_len, int kv_len, int tile) {
  const int rows = q_len * a.group, r0 = tile * kManyRows;
  TileWork t;
  t.n = min(kManyRows, rows - r0);
  t.span = span_of(a, q_len, kv_len, r0, r0 + t.n - 1);
  t.blocks = max((t.span.hi - (t.span.lo & ~15) + KT - 1) / KT, 1);
  return t;
}
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int q_len) { return (q_len * a.group + kManyRows - 1) / kManyRows; }

// Blocks of one head of a sequence.
template <int KT>
__device__ __forceinline__ int head_blocks(const AttnArgs& a, int q_len, int kv_len) {
  int sum = 0;
  for (int t = tiles_of(a, q_len) - 1; t >= 0; --t) sum += tile_work<KT>(a, q_len, kv_len, t).blocks;
  return sum;
}

// A sequence a lane, as for few rows: its rows and the blocks of one of its heads.
struct SeqBlocks {
  int start, q_len, kv_len, head;
};
template <int KT>
__device__ __forceinline__ SeqBlocks seq_blocks(const AttnArgs& a, int b) {
  SeqBlocks w = {0, 0, 0, 0};
  if (b >= a.n_seq) return w;
  if (!sequence_of(a, b, w.start, w.q_len, w.kv_len)) {
    if (a.err) *a.err = 1;
    w.q_len = 0;
  }
  w.head = head_blocks<KT>(a, w.q_len, w.kv_len);
  return w;
}
// Stretches of less than `least` blocks do not pay: joining costs more.
template <int KT>
__device__ __forceinline__ Cut many_cut_of(const AttnArgs& a, int first64, int workgroups, int least) {
  Cut c;
  c.total = __builtin_amdgcn_readlane(lanes_upto(first64), 63);
  for (int base = 64; base < a.n_seq; base += 64)
    c.total += __builtin_amdgcn_readlane(lanes_upto(seq_blocks<KT>(a, base + int(threadIdx.x & 63)).head * a.n_kv), 63);
  c.per = max(__builtin_amdgcn_readfirstlane(int((uint32_t(c.total) + uint32_t(workgroups) - 1u) / uint32_t(workgroups))), least);
  return c;
}

// Partial results of the many-rows kernel: 32 rows `block` of slot x at
// (x * blocks + block); o as the lanes hold it, [D / 8][64 lanes][4], ml [32].
__device__ __forceinline__ size_t block_at(const Partials& p, size_t slot, int block) { return slot * (p.rows / 32) + block; }

// x of this lane and of lane ^ 32. The instruction exchanges the halves of two
// registers; the compiler's builtin for it has returned one register for both
// results here where both operands held the same value. (The wait state is
// the one it puts between a write of an operand and the exchange.)
__device__ __forceinline__ void both_halves(float x, float& lo, float& hi) {
  lo = x;
  hi = x;
  asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(lo), "+v"(hi));
}
__device__ __forceinline__ float swap_max(float x) {
  float lo, hi;
  both_halves(x, lo, hi);
  return fmaxf(lo, hi);
}
__device__ __forceinline__ float swap_sum(float x) {
  float lo, hi;
  both_halves(x, lo, hi);
  return lo + hi;
}

// HALVES = 2: two groups of waves take the keys' tiles in turn, each with its
// own buffers, and join through LDS at the end.
template <int D, bool F8, int HALVES>
__global__ __launch_bounds__(ManyGeometry<D>::THREADS * HALVES, 2) void attn_many_kernel(AttnArgs a, Partials part,
                                                                                int workgroups, int least) {
  using G = ManyGeometry<D>;
  constexpr int KT = G::KT, CH = G::CH, NL = G::NL, DW = G::DW, NW = G::WAVES, NG = KT / 16, NB = DW / 32,
                NK = KT / 32, ES = F8 ? 1 : 2;
  extern __shared__ __align__(16) uint8_t room[];
  __shared__ int flagged;
  const int lane = threadIdx.x & 63, wave_of_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int keys = HALVES > 1 ? wave_of_all / NW : 0, wave = wave_of_all - keys * NW;  // which half of the keys
  uint8_t* const tiles = room + keys * G::kLds;
  const int c = lane & 31, half = lane >> 5, my_rows = wave & 3, my_part = G::PARTS > 1 ? wave >> 2 : 0;
  Q4_DCHECK(int(gridDim.x) <= workgroups && part.rows <= kManyRows && part.rows % 32 == 0, kDbgAttnGrid);
  // Workgroups go to the 8 dies in turn; give each die a contiguous stretch
  // of them, so that the tiles of one head share its L2.
  const int n_wg = gridDim.x, per_die = n_wg / 8, over = n_wg % 8, die = blockIdx.x % 8;
  const int wg = die * per_die + min(die, over) + int(blockIdx.x) / 8;

  // this workgroup's stretch: from block k0 of row tile `tile` of head h of sequence b on
  int b = 0, h = 0, tile = 0, k0 = 0, left = 0;
  SeqBlocks sb;
  Cut cut = {0, 1};
  TileWork tw;
  if (part.owned == nullptr) {
    // a unit each, the last tiles of a head, which see most, first
    const int tiles = workgroups / (a.n_seq * a.n_kv), unit = wg / tiles;
    b = unit / a.n_kv, h = unit % a.n_kv, tile = tiles - 1 - wg % tiles;
    if (!sequence_of(a, b, sb.start, sb.q_len, sb.kv_len)) {
      if (a.err && threadIdx.x == 0) *a.err = 1;
      return;
    }
    if (tile >= tiles_of(a, sb.q_len)) return;
    tw = tile_work<KT>(a, sb.q_len, sb.kv_len, tile);
    left = tw.blocks;
  } else {
    sb = seq_blocks<KT>(a, lane);
    cut = many_cut_of<KT>(a, sb.head * a.n_kv, workgroups, least);
    const int64_t from64 = int64_t(wg) * cut.per;
    if (from64 >= cut.total) {
      part.own(Owned{wg, 0, 0, 0, 0, 0, 0}, false, true, 0, 0, 0);
      return;
    }
    const int from = int(from64);
    left = min(cut.per, cut.total - from);
    for (int seen = 0;;) {
      const int cost = sb.head * a.n_kv, upto = seen + lanes_upto(cost);
      const unsigned long long hit = __ballot(upto - cost <= from && from < upto);
      if (hit) {
        const int src = __ffsll(hit) - 1;
        b += src;
        k0 = from - __builtin_amdgcn_readlane(upto - cost, src);
        sb.start = __builtin_amdgcn_readlane(sb.start, src);
        sb.q_len = __builtin_amdgcn_readlane(sb.q_len, src);
        sb.kv_len = __builtin_amdgcn_readlane(sb.kv_len, src);
        sb.head = __builtin_amdgcn_readlane(sb.head, src);
        break;
      }
      b += 64;
      if (b >= a.n_seq) return;  // (not reached: from < total)
      seen = __builtin_amdgcn_readlane(upto, 63);
      sb = seq_blocks<KT>(a, b + lane);
    }
    h = __builtin_amdgcn_readfirstlane(int(uint32_t(k0) / uint32_t(sb.head)));
    k0 -= h * sb.head;
    tw = tile_work<KT>(a, sb.q_len, sb.kv_len, 0);
    while (k0 >= tw.blocks) {
      k0 -= tw.blocks;
      tw = tile_work<KT>(a, sb.q_len, sb.kv_len, ++tile);
    }
  }

  for (bool first = true;; first = false) {
    b = uniform(b), h = uniform(h), tile = uniform(tile), k0 = uniform(k0), left = uniform(left);
    sb = {uniform(sb.start), uniform(sb.q_len), uniform(sb.kv_len), sb.head};
    tw = {uniform(tw.span), uniform(tw.n), uniform(tw.blocks)};
    const int k1 = left < tw.blocks - k0 ? k0 + left : tw.blocks;
    const bool whole = k0 == 0 && k1 == tw.blocks;
    const int start = sb.start, q_len = sb.q_len, kv_len = sb.kv_len, r0 = tile * kManyRows, n = tw.n;
    const Span sp = tw.span;
    const int k_lo = (sp.lo & ~15) + k0 * KT;
    const int k_hi = min(sp.hi, (sp.lo & ~15) + k1 * KT);
    if (threadIdx.x == 0) flagged = 0;

    // this wave's rows and this lane's
    const int w0 = my_rows * 32, wn = min(32, n - w0);  // wn <= 0: a wave that only helps to load
    const Span ws = uniform(wn > 0 ? span_of(a, q_len, kv_len, r0 + w0, r0 + w0 + wn - 1) : Span{0, 0, 0, 0});
    const int row = r0 + min(w0 + c, n - 1);
    const bool live = w0 + c < n;
    const int token = row / a.group, hq = h * a.group + row % a.group;
    const int p_row = live ? kv_len - q_len + token : -1;
    const int lo_row = a.window > 0 && p_row >= a.window ? int(p_row - a.window + 1) : 0;
    const uint32_t row_wide = max(min(p_row + 1, k_hi) - lo_row, 0);
    // The sign of the scale goes into Q, so that the largest product is the
    // largest score; a scale of zero makes Q zero.
    float qs = a.scale * kLog2e * (F8 && a.k_scale ? a.k_scale[h] : 1.0f);
    const uint32_t flip = qs < 0.0f ? 0x80008000u : 0u, keep = qs == 0.0f ? 0u : ~0u;
    qs = qs == 0.0f ? 1.0f : fabsf(qs);
    constexpr int QR = DW / 16 - G::QL;
    uint32_t qf[QR][4];
    uint4* q_lds = reinterpret_cast<uint4*>(tiles + 4 * G::kTileBytes) + wave * (G::QL * 64) + lane;
    {
      const uint16_t* q_row = a.q + (size_t(start + token) * a.n_q + hq) * D + my_part * DW + 8 * half;
#pragma unroll
      for (int s = 0; s < DW / 16; ++s) {
        const uint4 v = *reinterpret_cast<const uint4*>(q_row + 16 * s);
        const uint4 w = make_uint4((v.x ^ flip) & keep, (v.y ^ flip) & keep, (v.z ^ flip) & keep, (v.w ^ flip) & keep);
        if (s < QR)
          qf[s < QR ? s : 0][0] = w.x, qf[s < QR ? s : 0][1] = w.y, qf[s < QR ? s : 0][2] = w.z, qf[s < QR ? s : 0][3] = w.w;
        else
          q_lds[(s - QR) * 64] = w;  // (this lane alone reads it again)
      }
    }

    const int32_t* table = a.page_table + b * a.table_stride;
    const int page_mask = (1 << a.page_shift) - 1;
    const size_t page_bytes = (size_t(a.n_kv) << a.page_shift) * (D * ES);
    const size_t head_bytes = (size_t(h) << a.page_shift) * (D * ES);
    // Piece i of this thread: row first_row(i) + lane / CH of the tile, and
    // which 16 bytes of the source it takes (8 of an e4m3 row).
    auto first_row = [&](int i) { return (i * NW + wave) * 64 / CH; };
    auto group_of = [&](int i) { return i * (NW * 64 / CH) / 16 + (D == 64 ? wave >> 1 : 0); };
    auto source_at = [&](int i, int pg, int kb) {
      const int r = first_row(i);
      return size_t(max(pg, 0)) * page_bytes + head_bytes +
             size_t((pg < 0 ? r & 15 : (kb + r) & page_mask)) * (D * ES);
    };
    // (the empty asm statements here and below keep addresses that are cheap
    // to form from being kept in registers, which there are none of to spare)
    auto lane_anew = [&]() {
      uint32_t zero = 0;
      asm("" : "+v"(zero));
      return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
    };
    auto lane_at = [&]() {
      const uint32_t l = lane_anew();
      return l / CH * (D * ES) + ((l % CH) ^ G::swizzle(first_row(0) + l / CH)) * (8 * ES);
    };
    // pieces i and i + 1 are 8, 16 or 32 rows apart: 8 flip a bit of the swizzle
    auto lane_flip = [&](int i) { return NW * 64 / CH == 8 && (i & 1) ? 16 * ES : 0; };
    static_assert(NW * 64 / CH == 8 ? D > 64 : NW * 64 / CH % 16 == 0, "the swizzle goes by the row within 16");
    // bf16: straight into LDS. e4m3: into registers, put() converts them
    // (LDS piece i * THREADS + wave * 64 + lane either way).
    uint2 hold_k[F8 ? NL : 1], hold_v[F8 ? NL : 1];
    Pages pages;
    auto fetch = [&](int group, int kb, int buf) {  // group: the first, in `pages`
      uint8_t* to = tiles + buf * (2 * G::kTileBytes);
      const uint32_t lane0 = lane_at();
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const size_t at = source_at(i, pages.at(group + group_of(i)), kb);
        const uint32_t mine = lane0 ^ lane_flip(i);
        if constexpr (F8) {
          hold_k[i] = *reinterpret_cast<const uint2*>(a.k_cache + at + mine);
          hold_v[i] = *reinterpret_cast<const uint2*>(a.v_cache + at + mine);
        } else {
          uint8_t* dst = to + (i * NW + wave) * 1024;
          load_to_lds(a.k_cache + at, a.v_cache + at, mine, dst, dst + G::kTileBytes);
        }
      }
    };
    auto put = [&](int buf) {
      if constexpr (F8) {
        uint8_t* to = tiles + buf * (2 * G::kTileBytes) + (wave * 64 + lane) * 16;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          *reinterpret_cast<uint4*>(to + i * NW * 1024) =
              make_uint4(e4m3_pair<false>(hold_k[i].x), e4m3_pair<true>(hold_k[i].x), e4m3_pair<false>(hold_k[i].y),
                         e4m3_pair<true>(hold_k[i].y));
          *reinterpret_cast<uint4*>(to + i * NW * 1024 + G::kTileBytes) =
              make_uint4(e4m3_pair<false>(hold_v[i].x), e4m3_pair<true>(hold_v[i].x), e4m3_pair<false>(hold_v[i].y),
                         e4m3_pair<true>(hold_v[i].y));
        }
      }
    };

    // LDS addresses of this lane's operands: K piece 2s + half of row c at
    // k_base ^ 32 s; V: the 16-lane group reads rows 4 half + lane % 16 / 4
    // (+ 8 for the second read, + 16 s), columns 16 (lane / 16 % 2) .. + 15 of 32.
    const int k_base = c * (CH * 16) + ((half ^ G::swizzle(c)) << 4) + my_part * (DW * 2);
    // (8 rows more flip bit 1 of the swizzle, 16 leave it as it is.)
    const int vr = 4 * half + (lane & 15) / 4, piece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int v_base = vr * (CH * 16) + ((piece ^ G::swizzle(vr)) << 4) + (lane & 1) * 8 + my_part * (DW * 2);

    f32x16 o[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    auto compute = [&](uint8_t* kt, const uint8_t* vt, bool on, bool open, uint32_t pages_ok, int kb, bool more,
                       int next_buf) {
      // Operands are read from LDS a few matrix instructions ahead; K's fewer
      // where e4m3 pieces wait in registers beside 256 columns, or operands of Q
      // would be in scratch (four 512-token chunks over up to 8000 keys 78 us
      // with 2, 86 with 3, 89 with 4; bf16 has the registers).
      constexpr int PK = F8 && DW == 256 ? 2 : 4, PV = 4, MK = NK * (DW / 16), MV = 2 * NK * NB;
      bf16x8 kr[PK], vq[PV];
      int kx = k_base, vx = v_base;
      asm volatile("" : "+v"(kx), "+v"(vx));
      auto read_k = [&](int x) {
        const int t = x / (DW / 16), i = x % (DW / 16);
        return *reinterpret_cast<const bf16x8*>(kt + t * 32 * (CH * 16) + (kx ^ (32 * (i & 7))) + 256 * (i >> 3));
      };
      auto read_v = [&](int x) {
        typedef __attribute__((address_space(3))) bf16x4 lds4;
        const int t = x / NB, i = x % NB, at = t * 16 * (CH * 16) + 256 * (i >> 2), flip4 = 64 * (i & 3);
        const bf16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(vt + (vx ^ flip4) + at));
        const bf16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(vt + (vx ^ (flip4 ^ 32)) + 8 * (CH * 16) + at));
        return bf16x8(__builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
      };
      bf16x8 ql[G::QL > 0 ? G::QL : 1];
      const uint4* qx = q_lds;
      auto read_q = [&](int i) { return *reinterpret_cast<const bf16x8*>(qx + i * 64); };
      f32x16 s[NK];
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) s[t][j] = 0.0f;
      // With two waves on a SIMD one's softmax is meant to run beside the
      // other's products, which go first (no priorities: 1 to 7% slower; the
      // softmax first: slower still).
      __builtin_amdgcn_s_setprio(1);
      if (on) {
#pragma unroll
        for (int x = 0; x < PK; ++x) kr[x] = read_k(x);
#pragma unroll
        for (int x = 0; x < MK; ++x) {
          const int t = x / (DW / 16), i = x % (DW / 16);
          const bf16x8 q8 = i < QR ? __builtin_bit_cast(bf16x8, qf[i < QR ? i : 0]) : ql[i < QR ? 0 : i - QR];
          s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kr[x % PK], q8, s[t], 0, 0, 0);
          if (x + PK < MK) kr[x % PK] = read_k(x + PK);
          if (x + PK >= QR && x + PK < QR + G::QL) ql[x + PK - QR < G::QL ? x + PK - QR : 0] = read_q(x + PK - QR);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (more) put(next_buf);
      if constexpr (G::PARTS > 1) {
        // the halves of the scores, through the keys' place: no wave reads them any more
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        f32x4* mine = reinterpret_cast<f32x4*>(kt) + wave * 256 + lane;
        const f32x4* other = reinterpret_cast<const f32x4*>(kt) + (wave ^ 4) * 256 + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) mine[64 * j] = f32x4{s[0][4 * j], s[0][4 * j + 1], s[0][4 * j + 2], s[0][4 * j + 3]};
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 x = other[64 * j];
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][4 * j + e] += x[e];
        }
      }
      if (!on) return;
      __builtin_amdgcn_s_setprio(0);
#pragma unroll
      for (int x = 0; x < PV; ++x) vq[x] = read_v(x);
      if (!open) {
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int g = 2 * t + j / 8;  // the 16 keys it belongs to
            const uint32_t at = uint32_t(kb + 32 * t + 8 * (j / 4) + 4 * half + j % 4 - lo_row);
            s[t][j] = at < (pages_ok >> g & 1 ? row_wide : 0u) ? s[t][j] : -INFINITY;
          }
      }
      float mx = s[0][0];
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) mx = fmaxf(mx, s[t][j]);  // (leaves a NaN score out; its p is NaN)
      mx = swap_max(mx) * qs;
      // (a row's first score: -infinity + kLazy is -infinity)
      if (__ballot(mx > m + kLazy)) {
        mx = fmaxf(m, mx);
        const float f = __builtin_amdgcn_exp2f(m - (mx == -INFINITY ? 0.0f : mx));
        l *= f;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[i][j] *= f;
        m = mx;
      }
      const float base = m == -INFINITY ? 0.0f : -m;
      uint32_t p[NK][8];
#pragma unroll
      for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float p0 = __builtin_amdgcn_exp2f(fmaf(s[t][j], qs, base));
          const float p1 = __builtin_amdgcn_exp2f(fmaf(s[t][j + 1], qs, base));
          l += p0 + p1;
          // One rounding to bf16 (2^-8 of a probability; l takes them unrounded):
          // a second part, as for few rows, would be half as many matrix
          // instructions again in a kernel that they bound. Against 64 bits the
          // result is off by 0.0020 to 0.0022, its own last rounding by 0.0017.
          p[t][j / 2] = pack_bf16(p0, p1);
        }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int x = 0; x < MV; ++x) {
        const int t = x / NB, i = x % NB;  // 16 keys each
        const uint32_t pb[4] = {p[t / 2][4 * (t & 1)], p[t / 2][4 * (t & 1) + 1], p[t / 2][4 * (t & 1) + 2],
                                p[t / 2][4 * (t & 1) + 3]};
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vq[x % PV], __builtin_bit_cast(bf16x8, pb), o[i], 0, 0, 0);
        if (x + PV < MV) vq[x % PV] = read_v(x + PV);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    if (k_hi > k_lo) {
      // `pages` holds 64 groups from k_lo or a multiple of 64 further on; the
      // bits say which groups of a step's tiles are there
      constexpr int kStep = HALVES * KT;
      constexpr uint32_t kAll = (1u << (HALVES * NG)) - 1;
      auto key_of = [&](int kb) { return kb + 16 * lane; };
      auto bits_at = [&](int group) { return uint32_t(__ballot(pages.now >= 0) >> group) & kAll; };
      pages.now = Pages::checked(a, Pages::read(a, table, key_of(k_lo), k_hi), key_of(k_lo), k_hi);
      uint32_t ok = bits_at(0), next_ok = 0;
      if (k_lo + keys * KT < k_hi) {
        fetch(keys * NG, k_lo + keys * KT, 0);
        put(0);
      }
      pages.raw = Pages::read(a, table, key_of(k_lo + 1024), k_hi);
      int buf = 0;
      for (int step = k_lo; step < k_hi; step += kStep, buf ^= 1) {
        const int kb = step + keys * KT;
        const bool more = kb + kStep < k_hi;
        // this wave's loads of the tile are done, then everyone's; no wave
        // still reads the other buffer
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (step + kStep < k_hi) {
          const int j = (step + kStep - k_lo) / 16 & 63;
          if (j == 0) {
            pages.now = Pages::checked(a, pages.raw, key_of(step + kStep), k_hi);
            pages.raw = Pages::read(a, table, key_of(step + kStep + 1024), k_hi);
          }
          next_ok = bits_at(j);
          if (more) fetch(j + keys * NG, kb + kStep, buf ^ 1);
        }
        uint8_t* kt = tiles + buf * (2 * G::kTileBytes);
        uint8_t* vt = tiles + buf * (2 * G::kTileBytes) + G::kTileBytes;
        const uint32_t mine = ok >> (keys * NG) & ((1u << NG) - 1);
        if (ok != kAll || step < sp.lo_max || step + kStep > min(sp.hi_min, k_hi)) {
          // 0 * NaN is NaN: values at keys that no row sees become zero, and at
          // keys that only some see those that are not finite, added at the end
#pragma unroll
          for (int i = 0; i < NL; ++i) {
            const uint32_t l = lane_anew();
            const int r = first_row(i) + l / CH, key = kb + r;
            const bool any = (mine >> (r / 16) & 1) & (key >= sp.lo) & (key < k_hi);
            const bool all = (key >= sp.lo_max) & (key < sp.hi_min);
            uint4* at = reinterpret_cast<uint4*>(vt + (i * NW + wave) * 1024 + l * 16);
            const uint32_t there = any ? ~0u : 0u, some = all ? 0u : ~0u;
            uint4 v = *at;
            uint32_t out = 0;
            auto mend = [&](uint32_t x) {  // (selects, no branch of some lanes)
              x &= there;
              const uint32_t odd = nonfinite<false>(x) & some;
              out |= odd;
              return x & ~spread<false>(odd);
            };
            v = make_uint4(mend(v.x), mend(v.y), mend(v.z), mend(v.w));
            *at = v;
            if (__ballot(out != 0)) flagged = 1;
          }
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        compute(kt, vt, kb < min(ws.hi, k_hi) && kb + KT > ws.lo,
                mine == (1u << NG) - 1 && kb >= ws.lo_max && kb + KT <= min(ws.hi_min, k_hi), mine, kb, more, buf ^ 1);
        ok = next_ok;
      }
    }
    l = swap_sum(l);
    __syncthreads();
    if constexpr (HALVES > 1) {
      // sums relative to the larger of the two maxima, through the tiles' place
      f32x4* other = reinterpret_cast<f32x4*>(room) + my_rows * (D / 8 * 64) + lane;
      float2* other_ml = reinterpret_cast<float2*>(room + 4 * D / 8 * 1024) + my_rows * 64 + lane;
      static_assert(4 * D / 8 * 1024 + 4 * 64 * sizeof(float2) <= HALVES * G::kLds, "room for one half's sums");
      if (keys == 1) {
        *other_ml = make_float2(m, l);
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            other[(4 * i + j) * 64] = f32x4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
      }
      __syncthreads();
      if (keys == 0) {
        const float2 ml = *other_ml;
        const float mx = fmaxf(m, ml.x), base = mx == -INFINITY ? 0.0f : mx;
        const float f = __builtin_amdgcn_exp2f(m - base), f1 = __builtin_amdgcn_exp2f(ml.x - base);
        m = mx;
        l = l * f + ml.y * f1;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 x = other[(4 * i + j) * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][4 * j + e] = o[i][4 * j + e] * f + x[e] * f1;
          }
      }
    }
    if (wn > 0 && keys == 0) {
      const bool blank = (m == -INFINITY) & (l == 0.0f) & reaches(lo_row, row_wide, k_lo);
      if (__ballot(blank))
        l = (blank & sees_some(a, table, lo_row, row_wide, k_lo, k_hi)) ? (whole ? NAN : kBlank) : l;
      if (!whole) {
        const size_t at = block_at(part, size_t(wg) * 2 + (first ? 0 : 1), my_rows);
        if (half == 0 && my_part == 0) part.ml[at * 32 + c] = make_float2(m, l);
        f32x4* to = reinterpret_cast<f32x4*>(part.o) + (at * (D / 8) + my_part * (DW / 8)) * 64 + lane;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            to[(4 * i + j) * 64] = f32x4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
      } else if (live) {
        const float inv = l == 0.0f ? 0.0f : (F8 && a.v_scale ? a.v_scale[h] : 1.0f) / l;
        uint16_t* to = a.out + (size_t(start + token) * a.n_q + hq) * D + my_part * DW + 4 * half;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint2*>(to + 32 * i + 8 * j) = make_uint2(
                pack_bf16(o[i][4 * j] * inv, o[i][4 * j + 1] * inv), pack_bf16(o[i][4 * j + 2] * inv, o[i][4 * j + 3] * inv));
      }
      float spoilt = 0.0f;  // NaN if one of the sums is
      if constexpr (!F8) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < 16; j += 4) spoilt = fmaf(o[i][j] + o[i][j + 1] + (o[i][j + 2] + o[i][j + 3]), 0.0f, spoilt);
        if (l != l) spoilt = 0.0f;  // (all of the row is NaN)
      }
      if (k_hi > k_lo && (flagged | (__ballot(spoilt != spoilt) != 0)))
        put_nonfinite<D, F8, DW>(  // (a row that is all NaN stays so)
            a, table, h, my_part * DW, wn, lo_row, l != l ? 0u : row_wide, k_hi - k_lo, k_hi, [&](int i) { return k_lo + i; },
            [&](int row, int d, float x, bool anew) {
              if (whole) {
                const int t = (r0 + w0 + row) / a.group, q = h * a.group + (r0 + w0 + row) % a.group;
                uint16_t* at = a.out + (size_t(start + t) * a.n_q + q) * D + my_part * DW + d;
                *at = f32_to_bf16_rne(anew ? 0.0f : bf16_to_f32(*at) + x);
              } else {
                const size_t at = block_at(part, size_t(wg) * 2 + (first ? 0 : 1), my_rows) * (D / 8) + my_part * (DW / 8);
                float* to = part.o + ((at + d / 8) * 64 + d % 8 / 4 * 32 + row) * 4 + d % 4;
                *to = anew ? 0.0f : *to + x;
              }
            });
    }

    left -= k1 - k0;
    part.own(Owned{wg, pieces_of(k0 == 0, k1, tw.blocks, cut.per), first ? 0 : 1, start, h, r0, n}, k0 == 0, left <= 0, b,
             a.n_kv, tile);
    if (left <= 0) return;
    k0 = 0;
    if (++tile == tiles_of(a, sb.q_len)) {
      tile = 0;
      if (++h == a.n_kv) {
        h = 0;
        do {
          ++b;
          if (!sequence_of(a, b, sb.start, sb.q_len, sb.kv_len)) sb.q_len = 0;
        } while (sb.q_len == 0);  // (left > 0: there is one)
      }
    }
    tw = tile_work<KT>(a, sb.q_len, sb.kv_len, tile);
    __syncthreads();  // LDS and the flag are free again
  }
}

// Joins the pieces of a unit, 32 rows and 8 columns a wave; TAKERS waves share
// them where the pieces are many.
template <int D, int TAKERS>
__global__ __launch_bounds__(kAttnThreads) void attn_join_many_kernel(AttnArgs a, Partials part) {
  constexpr int kWide = kAttnWaves / TAKERS;  // groups of 8 columns of a workgroup
  __shared__ f32x4 sum[kAttnWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 31, taker = wave % TAKERS;
  const int block = blockIdx.x / (D / 8 / kWide);
  const int piece = blockIdx.x % (D / 8 / kWide) * kWide + wave / TAKERS;  // columns 8 piece .. + 7
  const Owned u = part.find(a, blockIdx.y, kManyRows);
  if (block * 32 >= u.n || u.pieces == 0) return;
  const int n = u.pieces;
  auto at_of = [&](int i) { return block_at(part, size_t(u.wg + i) * 2 + (i == 0 ? u.slot : 0), block); };
  float m = -INFINITY, l = 0.0f;
#pragma unroll 8
  for (int i = 0; i < n; ++i) m = fmaxf(m, part.ml[at_of(i) * 32 + c].x);
  const float base = m == -INFINITY ? 0.0f : m;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  const f32x4* from = reinterpret_cast<const f32x4*>(part.o) + piece * 64 + lane;
#pragma unroll 8
  for (int i = taker; i < n; i += TAKERS) {
    const float2 v = part.ml[at_of(i) * 32 + c];
    const float f = __builtin_amdgcn_exp2f(v.x - base);
    l += v.y * f;
    x += from[at_of(i) * (D / 8 * 64)] * f;
  }
  if (__ballot(any_nan(x))) {
    x = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int i = taker; i < n; i += TAKERS)
      x += scaled(from[at_of(i) * (D / 8 * 64)], __builtin_amdgcn_exp2f(part.ml[at_of(i) * 32 + c].x - base));
  }
  if constexpr (TAKERS > 1) {
    __shared__ float sum_l[kAttnWaves][64];
    sum[wave][lane] = x;
    sum_l[wave][lane] = l;
    __syncthreads();
    if (taker != 0) return;
#pragma unroll
    for (int w = 1; w < TAKERS; ++w) {
      x += sum[wave + w][lane];
      l += sum_l[wave + w][lane];
    }
  }
  if (__ballot(m == -INFINITY)) {
    bool blank = false;
#pragma unroll 1
    for (int i = 0; i < n; ++i) blank |= part.ml[at_of(i) * 32 + c].y != 0.0f;
    l = ((m == -INFINITY) & blank) ? NAN : l;
  }
  if (block * 32 + c >= u.n) return;
  const float inv = l == 0.0f ? 0.0f : (a.v_scale ? a.v_scale[u.h] : 1.0f) / l;
  const int row = u.r0 + block * 32 + c, t = row / a.group, q = u.h * a.group + row % a.group;
  *reinterpret_cast<uint2*>(a.out + (size_t(u.start + t) * a.n_q + q) * D + 8 * piece + 4 * (lane >> 5)) =
      make_uint2(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv));
}

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
  if (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 512)
    return fail(Q4DEC_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128, 256 or 512 (got %lld)", name,
                (long long)head_dim);
  if (n_kv <= 0 || n_q <= 0 || n_q > kMaxHeads || n_q % n_kv)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_q must be a positive multiple of n_kv, at most 4096 (got %lld, %lld)", name,
                (long long)n_q, (long long)n_kv);
  if (n_q / n_kv > kMaxGroup)
    return fail(Q4DEC_ERR_UNSUPPORTED, "%s: more than %d query heads per key/value head (n_q %lld, n_kv %lld)", name,
                int(kMaxGroup), (long long)n_q, (long long)n_kv);
  if (n_tok < 0 || n_tok >= (int64_t(1) << 31) / n_q)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_tok must be in [0, 2^31 / n_q) (got %lld)", name, (long long)n_tok);
  if (n_seq < 0 || n_seq > 65535)
    return fail(Q4DEC_ERR_SHAPE, "%s: n_seq must be in [0, 65535] (got %lld)", name, (long long)n_seq);
  if (n_seq == 0 || n_tok == 0) return Q4DEC_OK;
  if (max_q_len <= 0 || max_q_len >= (int64_t(1) << 30) / n_q)
    return fail(Q4DEC_ERR_SHAPE, "%s: max_q_len must be in [1, 2^30 / n_q) (got %lld)", name, (long long)max_q_len);
  if (window < 0) return fail(Q4DEC_ERR_SHAPE, "%s: window must not be negative (got %lld)", name, (long long)window);
  if (!isfinite(scale)) return fail(Q4DEC_ERR_SHAPE, "%s: scale must be finite", name);
  if (!q) return fail(Q4DEC_ERR_NULL, "%s: q is NULL", name);
  if (!out) return fail(Q4DEC_ERR_NULL, "%s: out is NULL", name);
  if (!page_table) return fail(Q4DEC_ERR_NULL, "%s: page_table is NULL", name);
  if (!q_starts) return fail(Q4DEC_ERR_NULL, "%s: q_starts is NULL", name);
  if (!kv_lens) return fail(Q4DEC_ERR_NULL, "%s: kv_lens is NULL", name);
  int page_shift = 0;
  const int rc = check_cache(name, k_cache, v_cache, kv_type, n_pages, page_size, k_scale, v_scale, &page_shift);
  if (rc != Q4DEC_OK) return rc;
  if (table_stride <= 0 || table_stride >= (int64_t(1) << 31))
    return fail(Q4DEC_ERR_SHAPE, "%s: table_stride must be in [1, 2^31) (got %lld)", name, (long long)table_stride);
  if (max_kv_len < 0 || max_kv_len > (int64_t(1) << 30) || (max_kv_len + page_size - 1) / page_size > table_stride)
    return fail(Q4DEC_ERR_SHAPE, "%s: max_kv_len must be in [0, table_stride * page_size], at most 2^30 (got %lld)", name,
                (long long)max_kv_len);
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(Q4DEC_ERR_ALIGN, "%s: q and out must be 16-byte aligned", name);
  if (!aligned(page_table, 4) || !aligned(q_starts, 4) || !aligned(kv_lens, 4))
    return fail(Q4DEC_ERR_ALIGN, "%s: page_table, q_starts and kv_lens must be 4-byte aligned", name);
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
