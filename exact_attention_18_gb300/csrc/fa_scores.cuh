// Modified scores: a tanh cap and a bias that falls with distance, applied to
// the products q_i . k_j between the score MMA and the softmax (and, with the
// cap's derivative, in the backward).  In the base-2 domain of the softmax,
//
//   y = c tanh(scale x / cap) - s_h |i - j|,   c = cap log2 e, s_h = slopes[h] log2 e,
//
// or scale log2 e x in the first term's place without a cap.  Only the scores'
// registers change: what follows sees them as scores of scale 1.
//
// tanh.  The unit that has exp2 gives 32 of them a clock and SM, but 16 of
// tanh.approx (whose 2^-11 would show in the weights: 0.02 of a score at a cap of
// 50).  tanh(v) = 1 - 2 / (1 + e^(2v)) takes an exp2 and a reciprocal.  The FMA
// units, which the softmax leaves idle, do better on a polynomial as long as
// |v| <= 1, the common case: a cap is set well above most scores.  A score with
// |v| <= 1 gets the polynomial's value, another the exact form's, and a warp whose
// scores of a block are all small skips the latter.
#pragma once

#include "fa_kernel_common.cuh"

namespace fa {

// The minimax polynomial of degree 5 in w = v^2 for tanh(v) / v on |v| <= 1 (by
// Remez exchange; relative error 6e-7, 7e-7 with the roundings below).
constexpr float kTanhMax = 1.0f;
__device__ __forceinline__ float2 tanh_small(float2 v) {
  const float2 w = __fmul2_rn(v, v);
  float2 t = make_float2(-0.00306706037f, -0.00306706037f);
  t = __ffma2_rn(t, w, make_float2(0.0167431142f, 0.0167431142f));
  t = __ffma2_rn(t, w, make_float2(-0.0516056754f, -0.0516056754f));
  t = __ffma2_rn(t, w, make_float2(0.132814333f, 0.132814333f));
  t = __ffma2_rn(t, w, make_float2(-0.333290428f, -0.333290428f));
  t = __ffma2_rn(t, w, make_float2(0.999999404f, 0.999999404f));
  return __fmul2_rn(t, v);
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(v) = 1 - 2 / (1 + e^(2v)) of two values x with v = in x.  A reciprocal each: one
// of the product of both denominators would let a hidden neighbour's NaN through.
__device__ __forceinline__ float2 tanh_exact(float2 x, float in2) {
  const float2 z = __fmul2_rn(x, make_float2(in2, in2));
  const float2 a = __fadd2_rn(make_float2(ptx::ex2(z.x), ptx::ex2(z.y)), make_float2(1.f, 1.f));
  return __ffma2_rn(make_float2(rcp(a.x), rcp(a.y)), make_float2(-2.f, -2.f), make_float2(1.f, 1.f));
}

// Largest |x| of N scores (N a multiple of 2); NaN does not count.
template <int N>
__device__ __forceinline__ float abs_max(const uint32_t* sr) {
  constexpr int kChains = N >= 64 ? 4 : (N >= 16 ? 2 : 1);
  float m[kChains];
#pragma unroll
  for (int k = 0; k < kChains; ++k) {
    const uint32_t* v = sr + k * (N / kChains);
    m[k] = fabsf(__uint_as_float(v[0]));
#pragma unroll
    for (int c = 1; c < N / kChains; ++c) m[k] = fmaxf(m[k], fabsf(__uint_as_float(v[c])));
  }
#pragma unroll
  for (int k = 1; k < kChains; ++k) m[0] = fmaxf(m[0], m[k]);
  return m[0];
}

// Where a row's keys lie, for the bias: all of the block at or before the row
// (and in causal calls wherever it counts), all behind it, or on both sides.
enum ScoreSide { kSideLeft = 0, kSideRight = 1, kSideBoth = 2 };

// tanh of two scores x (v = in x) by the rule of both forms: a score alone decides
// which one gives it, so that nothing else in the warp's registers has a say in its
// bits.  `all_small` (of the warp): no score needs the exact form.
__device__ __forceinline__ float2 tanh2(float2 x, const ScoreParams& sc, bool all_small) {
  const float2 v = __fmul2_rn(x, make_float2(sc.in, sc.in));
  float2 t = tanh_small(v);
  if (!all_small) {
    const float2 u = tanh_exact(x, sc.in2);
    t.x = fabsf(v.x) <= kTanhMax ? t.x : u.x;
    t.y = fabsf(v.y) <= kTanhMax ? t.y : u.y;
  }
  return t;
}

// N products x of one row become capped, scaled base-2 scores in place (without a
// cap: times scale_log2).  The whole warp calls it.
template <int N>
__device__ __forceinline__ void cap_row(uint32_t* sr, const ScoreParams& sc, float scale_log2) {
  if (sc.cap != 0.f) {
    auto capped = [&](bool all_small) {
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const float2 t = tanh2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sc, all_small);
        const float2 y = __fmul2_rn(t, make_float2(sc.cap, sc.cap));
        sr[c] = __float_as_uint(y.x);
        sr[c + 1] = __float_as_uint(y.y);
      }
    };
    if (__any_sync(0xffffffffu, abs_max<N>(sr) * fabsf(sc.in) > kTanhMax)) capped(false);
    else capped(true);
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) sr[c] = __float_as_uint(__uint_as_float(sr[c]) * scale_log2);
  }
}

// Their bias: column c stands d0 + c behind the row.  slope: s_h.
template <int N>
__device__ __forceinline__ void bias_row(uint32_t* sr, float slope, int d0, ScoreSide side) {
  if (side == kSideBoth) {
#pragma unroll
    for (int c = 0; c < N; ++c)
      sr[c] = __float_as_uint(fmaf(-slope, fabsf(static_cast<float>(d0 + c)), __uint_as_float(sr[c])));
    return;
  }
  // -s |d| with d = d0 + c of one sign.  The distance d0 + c is formed first (exact
  // below 2^24), so each score's bias is rounded once.
  const float s = side == kSideLeft ? slope : -slope;
  const float f0 = static_cast<float>(d0);
  const float2 s2 = make_float2(s, s);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 d = make_float2(f0 + static_cast<float>(c), f0 + static_cast<float>(c + 1));
    const float2 y = __ffma2_rn(s2, d, make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])));
    sr[c] = __float_as_uint(y.x);
    sr[c + 1] = __float_as_uint(y.y);
  }
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
