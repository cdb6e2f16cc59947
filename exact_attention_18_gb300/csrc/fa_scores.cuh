// Modified scores: a tanh cap and a bias that falls with distance, applied to
// the products q_i . k_j between the score MMA and the softmax (and, with the
// cap's derivative, in the backward).  In the base-2 domain of the softmax,
//
//   y = c tanh(scale x / cap) - s_h |i - j|,   c = cap log2 e, s_h = slopes[h] log2 e,
//
// or scale log2 e x in the first term's place without a cap.  Only the scores'
// registers change: what follows sees scores of another scale, the call's unit
// (ScoreParams in fa_internal.cuh).
//
// tanh.  The unit that has exp2 gives 32 of them a clock and SM, but 16 of
// tanh.approx (whose 2^-11 would show in the weights: 0.02 of a score at a cap of
// 50).  tanh(v) = 1 - 2 / (1 + e^(2v)) takes an exp2 and a reciprocal.  The FMA
// units, which the softmax leaves idle, do better on a polynomial as long as
// |v| <= 1.25 (0.49 for caps of 400 scales or more), the common case: a cap is set well
// above most scores.  Such a score gets the polynomial's value, another the exact form's, and a warp whose scores of a block
// are all small skips the latter.
#pragma once

#include "fa_kernel_common.cuh"
#include "fa_softmax.cuh"

namespace fa {

// tanh(scale x / cap) of small x: x times a polynomial in x^2, the minimax
// approximation of tanh(v) / v on |v| <= 1.25 (degree 6 in v^2: relative error 8.4e-7
// with fp32's roundings) with scale / cap folded into the coefficients on the host
// (tanh_poly in fa_api.cu).
__device__ __forceinline__ float2 tanh_small(float2 x, const ScoreParams& sc) {
  const float2 w = __fmul2_rn(x, x);
  float2 t = make_float2(sc.poly[kTanhTerms - 1], sc.poly[kTanhTerms - 1]);
#pragma unroll
  for (int k = kTanhTerms - 2; k >= 0; --k) t = __ffma2_rn(t, w, make_float2(sc.poly[k], sc.poly[k]));
  return __fmul2_rn(t, x);
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(v) = 1 - 2 / (1 + e^(2v)), v = scale x / cap.  A reciprocal each: one of the
// product of both denominators would let a hidden neighbour's NaN through.
__device__ __forceinline__ float2 tanh_exact(float2 x, const ScoreParams& sc) {
  const float2 z = __fmul2_rn(x, make_float2(sc.in2, sc.in2));
  const float2 a = __fadd2_rn(make_float2(ptx::ex2(z.x), ptx::ex2(z.y)), make_float2(1.f, 1.f));
  return __ffma2_rn(make_float2(rcp(a.x), rcp(a.y)), make_float2(-2.f, -2.f), make_float2(1.f, 1.f));
}

// Largest |x| of N scores (N a multiple of 8); NaN does not count.
template <int N>
__device__ __forceinline__ float abs_max(const uint32_t* sr) {
  constexpr int kChains = N >= 64 ? 4 : 2;
  float m[kChains];
#pragma unroll
  for (int k = 0; k < kChains; ++k) {
    const uint32_t* v = sr + k * (N / kChains);
    m[k] = 0.f;
#pragma unroll
    for (int c = 0; c < N / kChains; c += 2)
      asm("max.abs.f32 %0, %1, %2, %3;"
          : "=f"(m[k])
          : "f"(m[k]), "f"(__uint_as_float(v[c])), "f"(__uint_as_float(v[c + 1])));
  }
#pragma unroll
  for (int k = 1; k < kChains; ++k) m[0] = fmaxf(m[0], m[k]);
  return m[0];
}

// tanh of two products by the rule of both forms.  kCapAny looks at each; kCapSmall
// is for warps whose products are all small: the same bits.
enum CapForm { kNoCap = 0, kCapSmall = 1, kCapAny = 2 };
template <CapForm F>
__device__ __forceinline__ float2 tanh2(float2 x, const ScoreParams& sc) {
  float2 t = tanh_small(x, sc);
  if constexpr (F == kCapAny) {
    const float2 u = tanh_exact(x, sc);
    t.x = fabsf(x.x) <= sc.small ? t.x : u.x;
    t.y = fabsf(x.y) <= sc.small ? t.y : u.y;
  }
  return t;
}

// A row against the keys of a block, column c at distance d0 + c (key - row).  Its
// bias is s c + s d0 with s = s_h for keys at or before the row, -s_h for those
// behind: in a block on one side of all of its tile's rows, s d0 is a constant of
// the row (`fixed`), which joins minus the maximum.  (Causal calls: what lies behind
// the row is hidden, and a block counts as one at or before it.)
// The two parts are larger than their sum by up to a block's width of slopes, and so is
// their rounding: under 2^-15 in all for slopes up to 1, about the product's own.
// Blocks on both sides take each key's distance by itself, and so do blocks of drafted
// keys that do not stand at their slots, and steep rows: exact for the keys next to such a
// row, which are all that it weighs.  A steep row's scores are in base 2: a steep slope
// over a small unit leaves fp32's range, and a maximum as large as its biases (it sees far
// keys alone, or the slope is negative) is off by its product with the unit's rounding,
// which the exponentials would take for a score.
constexpr float kSteep = 1.5f;  // base 2: a slope of 1.04
struct RowBias {
  float slope;  // s_h (0: no bias), in the row's unit
  float s;      // the same with its sign, of a one-sided block; 0 where `both`
  float fixed;  // s d0, base 2
  float unit;   // of the row's scores, base 2: the call's, or 1 of a steep row
  int d0;
  bool both, steep;
};
// What a row keeps of its slope: the slope in the row's unit, and that unit.  slope2: s_h,
// base 2; steep: is_steep of it, or of any row of the warp.  A vote leaves unit and flag
// in uniform registers (causal B4 H16 S4096 D64 with a bias, a thread's own / the vote's:
// 189 / 183 us; 16 trees of 64 tokens 88.5 / 87.8); at D = 128 it spills (capped B2 H32/4
// S4096: 350 / 375).
struct RowSlope {
  float slope, unit;
  bool steep;
};
__device__ __forceinline__ bool is_steep(float slope2) { return fabsf(slope2) > kSteep; }
__device__ __forceinline__ RowSlope row_slope(const ScoreParams& sc, float slope2, bool steep) {
  return RowSlope{steep ? slope2 : slope2 * sc.per_unit, steep ? 1.f : sc.unit, steep};
}
__device__ __forceinline__ RowBias row_bias(const RowSlope& row, int d0, bool left, bool right) {
  const bool both = (!left && !right) || row.steep;
  const float s = both ? 0.f : (left ? row.slope : -row.slope);
  return RowBias{row.slope, s, s * static_cast<float>(d0) * row.unit, row.unit, d0, both, row.steep};
}

// Columns [lo, hi) of 32 as bits.
__device__ __forceinline__ unsigned bit_range(int lo, int hi) {
  const unsigned from = lo <= 0 ? ~0u : (lo >= 32 ? 0u : ~0u << lo);
  const unsigned to = hi >= 32 ? ~0u : (hi <= 0 ? 0u : ~(~0u << hi));
  return from & to;
}

// Which columns of a block a row sees: lo .. lim.  off: where column c's key stands,
// less the block's first key (group: what it needs to know of 16 columns).
struct PlainCols {
  int lo, lim;
  static constexpr bool kOff = false;
  __device__ __forceinline__ unsigned word(int c0) const { return bit_range(lo - c0, lim + 1 - c0); }
  __device__ __forceinline__ int group(int) const { return 0; }
  __device__ __forceinline__ int off(int, int c) const { return c; }
};

// The scores of a block in the row's unit, less the row's constant, in two forms that
// agree to the bit where both apply.  In registers, for warps whose block is one-sided
// and (under a cap) all small, and a sensible scale:
template <int N>
__device__ __forceinline__ void scores_fast(uint32_t* sr, const ScoreParams& sc, float s) {
  // (The bias of a column takes its number as an immediate: one scalar FMA.  Packed, the
  // pair of numbers is two moves on top.)
  auto each = [&](auto form, bool biased) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      float2 y = form(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])));
      if (biased) y = make_float2(fmaf(s, static_cast<float>(c), y.x), fmaf(s, static_cast<float>(c + 1), y.y));
      sr[c] = __float_as_uint(y.x);
      sr[c + 1] = __float_as_uint(y.y);
    }
  };
  auto capped = [&](float2 x) { return tanh2<kCapSmall>(x, sc); };
  // (Which form stands first is felt: a capped block without a bias is 2 % faster here
  // than behind the others, a biased one without a cap 1 to 4 % slower.)
  if (sc.slopes == nullptr) {
    if (sc.cap != 0.f) each(capped, false);
  } else {
    if (sc.cap != 0.f) each(capped, true);
    else each([](float2 x) { return x; }, true);
  }
}
// And for any block: from TMEM (column t_s on) and back to it, 16 columns at a time in
// a rolled loop.  Blocks that need it are few, and their code must be short: unrolled
// over a block's columns, beside the fast form, it made the warps wait for
// instructions most of the time (causal B2 H16/4 S4096 D128, capped: 1410 us).
template <int N, typename Cols>
__device__ __forceinline__ void scores_slow(uint32_t t_s, const ScoreParams& sc, const RowBias& r,
                                            const Cols& cols, float back, bool large) {
#pragma unroll 1
  for (int k0 = 0; k0 < N; k0 += 16) {
    uint32_t x16[16];
    ptx::tmem_ld16(t_s + k0, x16);
    const int grp = cols.group(k0);
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      float2 y = make_float2(__uint_as_float(x16[c]), __uint_as_float(x16[c + 1]));
      if (sc.cap != 0.f) y = Cols::kOff && !large ? tanh2<kCapSmall>(y, sc) : tanh2<kCapAny>(y, sc);
      else if (sc.premul) y = __fmul2_rn(y, make_float2(sc.pre, sc.pre));
      if (sc.slopes != nullptr) {
        if (r.steep) y = __fmul2_rn(y, make_float2(sc.unit, sc.unit));
        auto biased = [&](float v, int e) {
          if (r.both) return fmaf(-r.slope, fabsf(static_cast<float>(r.d0 + e)), v);
          if (Cols::kOff && r.d0 + e > 0) return fmaf(-r.slope, static_cast<float>(e), v) - back;
          return fmaf(r.s, static_cast<float>(e), v);
        };
        y = make_float2(biased(y.x, cols.off(grp, k0 + c)), biased(y.y, cols.off(grp, k0 + c + 1)));
      }
      x16[c] = __float_as_uint(y.x);
      x16[c + 1] = __float_as_uint(y.y);
    }
    ptx::tmem_st16(t_s + k0, x16);
  }
  ptx::tmem_st_wait();
}

// A block's scores in place of the products that sr holds, loaded from column t_s on;
// -inf where `cut` and the row does not see the key.
template <int N, typename Cols>
__device__ __forceinline__ void block_scores(uint32_t* sr, uint32_t t_s, const ScoreParams& sc,
                                             const RowBias& r, bool cut, const Cols& cols) {
  static_assert(N == 64 || N == 128, "block width");
  const bool large = sc.cap != 0.f && __any_sync(0xffffffffu, !(abs_max<N>(sr) <= sc.small));
  const bool slow =
      large || sc.premul || (sc.slopes != nullptr && (Cols::kOff || __any_sync(0xffffffffu, r.both)));
  if (slow) {
    // (a drafted key behind its row: -s d, less the constant s d0 that is added later)
    scores_slow<N>(t_s, sc, r, cols, 2.f * r.fixed * sc.per_unit, large);
    if constexpr (N == 128) ptx::tmem_ld128(t_s, sr);
    else ptx::tmem_ld64(t_s, sr);
  } else {
    scores_fast<N>(sr, sc, r.s);
  }
  if (cut) {
#pragma unroll
    for (int c0 = 0; c0 < N; c0 += 32) {
      const unsigned seen = cols.word(c0);
#pragma unroll
      for (int c = 0; c < 32; ++c)
        sr[c0 + c] = seen >> c & 1u ? sr[c0 + c] : __float_as_uint(-INFINITY);
    }
  }
}

// Maximum of a block's scores, base 2, rounded upwards: the exponentials' multiply-add
// then gives no score above 0, however large a far key's bias and so their rounding.
template <int N>
__device__ __forceinline__ float block_top(const uint32_t* sr, float unit) {
  return __fmul_ru(block_max_scaled<N>(sr, false, 0, N, 1.f, false), unit);
}

// The order in which a forward CTA takes its key blocks [lo, ..).  A bias makes the
// keys next to a row its largest scores: from there outwards the running maximum
// hardly moves, while towards them it moves, and O is rescaled, at every block.  So
// the blocks up to `split` come first, downwards, then those behind, upwards.  All
// upwards / so (us, causal S4096): biased D = 128 (B1 H32/4) 158 / 141, D = 64 (B2 H16)
// 106 / 93; capped, where the blocks that a mask cuts then come while others still
// load, 178 / 167 and 136 / 134.
struct BlockOrder {
  int lo, split;
  __device__ __forceinline__ int at(int x) const { return x < split - lo ? split - 1 - x : lo + x; }
  __device__ __forceinline__ int index(int blk) const { return blk < split ? split - 1 - blk : blk - lo; }
  // The blocks [a, b) are the loaded ones [*beg, *end): those of a tile lie together
  // because either b <= split, or split = lo, or a = lo.
  __device__ __forceinline__ void span(int a, int b, int* beg, int* end) const {
    if (b <= split) {
      *beg = split - b;
      *end = split - a;
    } else {
      *beg = split > lo ? 0 : a - lo;
      *end = b - lo;
    }
  }
};
// Of blocks [lo, hi); `diag`: the block after that of the CTA's last row; `open`: the
// window has no left side, so every tile starts at lo.
__device__ __forceinline__ BlockOrder block_order(int lo, int hi, bool open, int diag) {
  return BlockOrder{lo, open ? max(lo, min(hi, diag)) : hi};
}

// Visible keys of a sample's rows under a prefix: its clamped length (0: none).
__device__ __forceinline__ int prefix_len(const ScoreParams& sc, int b, int S) {
  return sc.prefix == nullptr ? 0 : max(0, min(S, __ldg(sc.prefix + b)));
}

// Rows r0 .. rows - 1 of a tile that TMA wrote become zero, for the products that
// follow.  The whole warp calls it; the caller then signals the tile.
template <typename G>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int rows, int r0) {
  constexpr int kVecs = G::kRowBytes / 16;
  const int per = (rows - r0) * kVecs;
  for (int i = threadIdx.x & 31; i < per * G::kChunks; i += 32) {
    const int ch = i / per;
    *reinterpret_cast<uint4*>(tile + ch * G::kChunkBytes + r0 * G::kRowBytes + (i - ch * per) * 16) =
        make_uint4(0, 0, 0, 0);
  }
  ptx::fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace fa
