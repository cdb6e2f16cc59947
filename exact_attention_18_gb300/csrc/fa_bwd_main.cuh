// The backward's kernel for one tile a CTA, both passes (fa_bwd.cu has the
// mathematics and the roles of the warps), and its launch.  Included by fa_bwd.cu
// and, for modified scores, fa_bwd_scores.cu.
#pragma once

#include "fa_scores.cuh"

namespace fa {
using namespace ptx;

// Source of L = +inf for partner query rows past a sample's end (dK/dV pass,
// general instantiation).
static __device__ const float g_pos_inf = __builtin_huge_valf();

namespace {

constexpr int kPartnerRows = 64;  // rows of a streamed B tile
constexpr int kBwdGroups = 2;     // softmax-gradient groups of 8 warps; group g takes blocks i = g mod 2
constexpr int kProducerWarp = 8 * kBwdGroups;
constexpr int kMmaWarp = kProducerWarp + 1;  // issues the score products X, Y
constexpr int kAccWarp = kMmaWarp + 1;       // issues the accumulations
constexpr int kBwdThreads = (kAccWarp + 1) * 32;
constexpr int kDeltaWarp = kAccWarp + 1;  // persistent dQ pass: computes Delta
constexpr int kDqpThreads = kBwdThreads + 32;
// "P and dS of block i stored" barriers, block i on bar_pfull[i % 4] (8
// arrivals, one per warp of group i % 2).  With three X/Y buffers a warp of a
// group may finish block i and move on to the group's next block, i + 2,
// before another warp of the group has finished block i: X, Y(i + 2) wait only
// for the accumulation of block i - 1, the other group's.  With one barrier
// per group the fast warp's next arrival would count toward block i's phase,
// which could then complete before all of block i's P and dS are stored; with
// two per group it lands on the other barrier.  No warp gets two blocks ahead:
// X, Y(i + 4) wait for an accumulation issued after block i's, which waits
// for all eight arrivals of block i.
constexpr int kPFullBars = 2 * kBwdGroups;

template <int D>
struct BwdLayout {
  using GA = TileGeom<D, 128>;
  using GB = TileGeom<D, kPartnerRows>;
  // Partner blocks in flight: enough to cover the load latency where shared
  // memory allows (D <= 64); D = 128 tiles leave room for four.
  static constexpr int kStages = D <= 64 ? 8 : 4;
  static constexpr int kOffA1 = 0;
  static constexpr int kOffA2 = kOffA1 + GA::kTileBytes;
  static constexpr int kOffB1 = kOffA2 + GA::kTileBytes;             // [kStages] tiles
  static constexpr int kOffB2 = kOffB1 + kStages * GB::kTileBytes;   // [kStages] tiles
  static constexpr int kOffVec = kOffB2 + kStages * GB::kTileBytes;  // [kStages][L, Delta][64] fp32
  static constexpr int kOffBar = kOffVec + kStages * 2 * kPartnerRows * 4;
  // X/Y buffers in TMEM (128 columns each): three when the accumulators
  // leave room (D <= 64), so the MMA warp can compute X, Y two blocks ahead.
  static constexpr int kXYBufs = D <= 64 ? 3 : 2;
  // a_full, b_full[S], empty[S], xy_full[buffers], acc_issued[buffers], p_full[4], acc_final, drain[2],
  // then (persistent kernels only) a_empty, acc_free, delta_full[2], delta_free[2], stage_full.
  static constexpr int kNumBars = 1 + 2 * kStages + 2 * kXYBufs + kPFullBars + 1 + 2 + 7;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemUsed = kOffMisc + 16;
  static constexpr int kSmemBytes = (kSmemUsed + 1024) > 116 * 1024 ? (kSmemUsed + 1024) : 116 * 1024;
  static constexpr uint32_t kTmemCols = 512;
  // Group g's buffer: X at column 128 g, Y at 128 g + 64 (64 fp32 columns each).
  static constexpr uint32_t kColAcc1 = 128 * kXYBufs;      // dV (dK/dV pass) or dQ
  static constexpr uint32_t kColAcc2 = 128 * kXYBufs + D;  // dK (dK/dV pass)
  static_assert(kColAcc2 + D <= kTmemCols, "TMEM layout");
  // dQ pass: the resident tiles A1 = Q, A2 = dO are copied into TMEM (D/2
  // columns each, after dQ; at D = 128 they take the columns dK would use in
  // the dK/dV pass) and the score products read A from there instead of
  // shared memory (32 instead of 48 cycles per M128 N64 K16 MMA).
  static constexpr bool kTmemA = true;
  static constexpr uint32_t kColA1 = kColAcc1 + D;
  static constexpr uint32_t kColA2 = kColA1 + D / 2;
  static_assert(!kTmemA || kColA2 + D / 2 <= kTmemCols, "TMEM layout");
};

// TMEM column (relative to a buffer's X or Y) of MMA K-step kk of the 16-bit
// P or dS block: warp half h wrote partner columns 32h..32h+31 packed into
// columns 32h..32h+15 of its own 32-column region.
__device__ __forceinline__ uint32_t packed_col(int kk) { return kk < 2 ? kk * 8 : 32 + (kk - 2) * 8; }


// One warp's 32 partner columns of a block: from the scores X and the
// gradient products Y (fp32, TMEM) form P = exp2(c X - L log2 e) and
// dS = P o (Y - Delta) and write them back as 16-bit pairs over the columns
// of X (P, dK/dV pass only) and Y (dS) already read.  In the dK/dV pass each
// column is a partner query whose L and Delta come from lv, dv; in the dQ
// pass they are the thread's own row's.  With DIAG the causal mask zeroes
// partner column c where c < lim (dK/dV pass) or c > lim (dQ pass); with WIN
// (a window band, dQ pass) also where c < lo.
template <bool BF16, bool KV_OUTER, bool DIAG, bool WIN = false>
__device__ __forceinline__ void grad_block(uint32_t tX, uint32_t tY, const float* lv, const float* dv, float2 c2,
                                           float my_l2, float my_delta, int lim, int lo = 0) {
  constexpr float kLog2e = 1.4426950408889634f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t xs[16], ys[16];
    tmem_ld16x2(tX + 16 * h, xs, tY + 16 * h, ys);
    uint32_t pk[8], dk[8];
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      const int cc = 16 * h + c;
      float2 nl2, dl;
      if constexpr (KV_OUTER) {
        nl2 = __fmul2_rn(make_float2(lv[cc], lv[cc + 1]), make_float2(-kLog2e, -kLog2e));
        dl = make_float2(dv[cc], dv[cc + 1]);
      } else {
        nl2 = make_float2(-my_l2, -my_l2);
        dl = make_float2(my_delta, my_delta);
      }
      const float2 y = __ffma2_rn(make_float2(__uint_as_float(xs[c]), __uint_as_float(xs[c + 1])), c2, nl2);
      float2 pr = make_float2(ex2(y.x), ex2(y.y));
      if constexpr (DIAG) {
        if ((KV_OUTER ? cc < lim : cc > lim) || (WIN && cc < lo)) pr.x = 0.f;
        if ((KV_OUTER ? cc + 1 < lim : cc + 1 > lim) || (WIN && cc + 1 < lo)) pr.y = 0.f;
      }
      const float2 gr = __fadd2_rn(make_float2(__uint_as_float(ys[c]), __uint_as_float(ys[c + 1])),
                                   make_float2(-dl.x, -dl.y));
      const float2 ds = __fmul2_rn(pr, gr);
      pk[c / 2] = pack2<BF16>(pr.x, pr.y);
      dk[c / 2] = pack2<BF16>(ds.x, ds.y);
    }
    // 16-bit P (dK/dV pass only) and dS of these 16 columns go to columns
    // 8h..8h+7 of this warp's region of X and Y, already read.
    if constexpr (KV_OUTER) tmem_st8(tX + 8 * h, pk);
    tmem_st8(tY + 8 * h, dk);
  }
}


// The dK/dV pass's version of grad_block, where the partner columns are
// queries with their own L and Delta.  The 32x32b layout would give every
// thread all 32 of the warp's columns and so all 32 (L, Delta) pairs from
// shared memory; with 16x256b loads a thread holds 2 adjacent columns of each
// of 4 column groups for 4 of the warp's rows (lanes t/4 + 8k), i.e. 8
// columns, a quarter of the shared-memory reads.  The packed 16-bit results
// of such a column pair go back with 16x128b stores to packed column
// (8i + 2(t%4)) / 2 = 4i + t%4, the layout the accumulation MMAs read.
// lim0: key index of the warp's first row minus its first partner column.
// With WIN (a window band) the mask keeps, for key row j, the partner
// queries j - wr .. j + wl: columns lim - wr .. lim + wl.
template <bool BF16, bool DIAG, bool WIN = false>
__device__ __forceinline__ void grad_block_kv(uint32_t tX, uint32_t tY, const float* lv, const float* dv, float2 c2,
                                              int lim0, int wr = 0, int wl = 0) {
  constexpr float kLog2e = 1.4426950408889634f;
  const int lane = threadIdx.x & 31;
  const int u = lane & 3;   // column pair within each group of 8
  const int r = lane >> 2;  // first of the thread's rows within 16
  float2 nl2[4], dl[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 l2 = *reinterpret_cast<const float2*>(lv + 8 * i + 2 * u);
    nl2[i] = __fmul2_rn(l2, make_float2(-kLog2e, -kLog2e));
    const float2 d2 = *reinterpret_cast<const float2*>(dv + 8 * i + 2 * u);
    dl[i] = make_float2(-d2.x, -d2.y);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t lane_off = static_cast<uint32_t>(16 * half) << 16;
    uint32_t xs[16], ys[16];
    tmem_ld16x256b_x4(tX + lane_off, xs);
    tmem_ld16x256b_x4(tY + lane_off, ys);
    tmem_ld_wait();
    uint32_t pk[8], dk[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = 4 * i + 2 * k;
        const float2 y = __ffma2_rn(make_float2(__uint_as_float(xs[e]), __uint_as_float(xs[e + 1])), c2, nl2[i]);
        float2 pr = make_float2(ex2(y.x), ex2(y.y));
        if constexpr (DIAG) {
          const int lim = lim0 + 16 * half + r + 8 * k;  // zero partner columns c < lim (query before key)
          const int cc = 8 * i + 2 * u;
          if constexpr (WIN) {
            if (cc < lim - wr || cc > lim + wl) pr.x = 0.f;
            if (cc + 1 < lim - wr || cc + 1 > lim + wl) pr.y = 0.f;
          } else {
            if (cc < lim) pr.x = 0.f;
            if (cc + 1 < lim) pr.y = 0.f;
          }
        }
        const float2 gr = __fadd2_rn(make_float2(__uint_as_float(ys[e]), __uint_as_float(ys[e + 1])), dl[i]);
        const float2 ds = __fmul2_rn(pr, gr);
        pk[2 * i + k] = pack2<BF16>(pr.x, pr.y);
        dk[2 * i + k] = pack2<BF16>(ds.x, ds.y);
      }
    }
    tmem_st16x128b_x4(tX + lane_off, pk);
    tmem_st16x128b_x4(tY + lane_off, dk);
  }
}

// Modified scores.  Of two products x: y = their base-2 scores plus `add` (minus L
// log2 e and the bias), and under a cap f = 1 - tanh^2.
template <CapForm F>
__device__ __forceinline__ float2 grad_score(float2 x, float2 add, const ScoreParams& sc, float2 c2, float2* f) {
  if constexpr (F == kNoCap) return __ffma2_rn(x, c2, add);
  const float2 t = tanh2<F>(x, sc);
  *f = __ffma2_rn(make_float2(-t.x, -t.y), t, make_float2(1.f, 1.f));
  return __ffma2_rn(t, make_float2(sc.cap, sc.cap), add);
}
template <int N>
__device__ __forceinline__ bool all_small(const uint32_t* xs, const ScoreParams& sc) {
  return __all_sync(0xffffffffu, abs_max<N>(xs) <= sc.small);
}

// What a thread of either pass knows of a block beside the products.
struct ScoreBlock {
  float slope;   // s_h
  int side;      // keys at or before their queries (-1), behind them (1), on both sides or steep (0)
  int d0;        // distance key - query at the thread's first row and column
  bool edge;     // a mask cuts the block: the limits count
  int lo, hi;    // dQ pass: visible columns; dK/dV pass: see below
  int wl, pfx;   // dK/dV pass
};

// grad_block (dQ pass) with modified scores: 16 columns whose products xs, ys are in
// registers.  FAST: blocks that no mask cuts, on one side of their queries, whose
// scores are all small (F = kCapSmall); the others have the same arithmetic.
// Beside dS it gives P o f, and adds P o dP to `sum` (see the kernel).
template <bool BF16, bool FAST, CapForm F, bool BIAS>
__device__ __forceinline__ void grad16_scored(const uint32_t* xs, const uint32_t* ys, uint32_t* pk, uint32_t* dk,
                                              int h, const ScoreParams& sc, float2 c2, float my_l2, float my_delta,
                                              const ScoreBlock& sb, float2& sum) {
  // Column cc's bias is s cc + s d0; the latter joins -L.
  const float s = sb.side > 0 ? -sb.slope : sb.slope;
  const float nb = BIAS ? fmaf(s, static_cast<float>(sb.d0 + 16 * h), -my_l2) : -my_l2;
#pragma unroll
  for (int c = 0; c < 16; c += 2) {
    float2 add = make_float2(nb, nb);
    if constexpr (BIAS) add = make_float2(fmaf(s, static_cast<float>(c), nb), fmaf(s, static_cast<float>(c + 1), nb));
    const int cc = 16 * h + c;
    if (BIAS && !FAST && sb.side == 0)
      add = make_float2(fmaf(-sb.slope, fabsf(static_cast<float>(sb.d0 + cc)), -my_l2),
                        fmaf(-sb.slope, fabsf(static_cast<float>(sb.d0 + cc + 1)), -my_l2));
    const float2 x = make_float2(__uint_as_float(xs[c]), __uint_as_float(xs[c + 1]));
    float2 f;
    const float2 y = grad_score<F>(x, add, sc, c2, &f);
    float2 pr = make_float2(ex2(y.x), ex2(y.y));
    if (!FAST && sb.edge) {
      if (cc < sb.lo || cc > sb.hi) pr.x = 0.f;
      if (cc + 1 < sb.lo || cc + 1 > sb.hi) pr.y = 0.f;
    }
    const float2 dp = make_float2(__uint_as_float(ys[c]), __uint_as_float(ys[c + 1]));
    const float2 gr = __fadd2_rn(dp, make_float2(-my_delta, -my_delta));
    sum = __ffma2_rn(pr, dp, sum);
    if constexpr (F != kNoCap) pr = __fmul2_rn(pr, f);
    const float2 ds = __fmul2_rn(pr, gr);
    pk[c / 2] = pack2<BF16>(pr.x, pr.y);
    dk[c / 2] = pack2<BF16>(ds.x, ds.y);
  }
}

template <bool BF16>
__device__ __forceinline__ void grad_block_scored(uint32_t tX, uint32_t tY, const ScoreParams& sc, float2 c2,
                                                  float my_l2, float my_delta, const ScoreBlock& sb, float2& sum) {
  const bool capped = sc.cap != 0.f, biased = sc.slopes != nullptr;
  // The whole of X first: which form the block takes, and the products of both halves.
  uint32_t xs[32], ys[16], pk[8], dk[8];
  const bool fast = !sb.edge && (sb.side != 0 || !biased);
  tmem_ld32(tX, xs);
  if (fast && (!capped || all_small<32>(xs, sc))) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      tmem_ld16(tY + 16 * h, ys);
      const uint32_t* x = xs + 16 * h;
      if (!capped) grad16_scored<BF16, true, kNoCap, true>(x, ys, pk, dk, h, sc, c2, my_l2, my_delta, sb, sum);
      else if (biased) grad16_scored<BF16, true, kCapSmall, true>(x, ys, pk, dk, h, sc, c2, my_l2, my_delta, sb, sum);
      else grad16_scored<BF16, true, kCapSmall, false>(x, ys, pk, dk, h, sc, c2, my_l2, my_delta, sb, sum);
      tmem_st8(tX + 8 * h, pk);
      tmem_st8(tY + 8 * h, dk);
    }
    return;
  }
  // (a rolled loop: the rare form's code is to be short, as in the forward)
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    tmem_ld16x2(tX + 16 * h, xs, tY + 16 * h, ys);
    if (capped) grad16_scored<BF16, false, kCapAny, true>(xs, ys, pk, dk, h, sc, c2, my_l2, my_delta, sb, sum);
    else grad16_scored<BF16, false, kNoCap, true>(xs, ys, pk, dk, h, sc, c2, my_l2, my_delta, sb, sum);
    tmem_st8(tX + 8 * h, pk);
    tmem_st8(tY + 8 * h, dk);
  }
}

// grad_block_kv with modified scores, in the same two forms.  A key row at distance
// d0 + its row sees (from its own mask) the partner queries hi + row .. lo + row of
// columns, all up to the latter where its key lies before the prefix (pfx).
template <bool BF16, bool FAST, CapForm F, bool BIAS>
__device__ __forceinline__ void grad16_kv_scored(const uint32_t* xs, const uint32_t* ys, uint32_t* pk, uint32_t* dk,
                                                 int half, const float2* nl2, const float2* dl, const ScoreParams& sc,
                                                 float2 c2, const ScoreBlock& sb) {
  const int lane = threadIdx.x & 31;
  const int u = lane & 3, r = lane >> 2;
  const float s = sb.side > 0 ? -sb.slope : sb.slope;
  // s (row - first column of the thread), of its two rows of this half
  float row[2] = {0.f, 0.f};
  if constexpr (BIAS) {
    row[0] = s * static_cast<float>(sb.d0 + 16 * half + r - 2 * u);
    row[1] = s * static_cast<float>(sb.d0 + 16 * half + r + 8 - 2 * u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 nb = nl2[i];
    if constexpr (BIAS)
      nb = make_float2(fmaf(s, -8.f * static_cast<float>(i), nb.x), fmaf(s, -8.f * static_cast<float>(i) - 1.f, nb.y));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int e = 4 * i + 2 * k;
      const int line = 16 * half + r + 8 * k, cc = 8 * i + 2 * u;
      float2 add = nb;
      if constexpr (BIAS) add = __fadd2_rn(nb, make_float2(row[k], row[k]));
      if (BIAS && !FAST && sb.side == 0)
        add = make_float2(fmaf(-sb.slope, fabsf(static_cast<float>(sb.d0 + line - cc)), nl2[i].x),
                          fmaf(-sb.slope, fabsf(static_cast<float>(sb.d0 + line - cc - 1)), nl2[i].y));
      const float2 x = make_float2(__uint_as_float(xs[e]), __uint_as_float(xs[e + 1]));
      float2 f;
      const float2 y = grad_score<F>(x, add, sc, c2, &f);
      float2 pr = make_float2(ex2(y.x), ex2(y.y));
      if (!FAST && sb.edge) {
        const int lim = sb.d0 + line;
        const int from = lim < sb.pfx ? -kNoWindow : lim - sb.hi;
        if (cc < from || cc > lim + sb.wl) pr.x = 0.f;
        if (cc + 1 < from || cc + 1 > lim + sb.wl) pr.y = 0.f;
      }
      const float2 gr = __fadd2_rn(make_float2(__uint_as_float(ys[e]), __uint_as_float(ys[e + 1])), dl[i]);
      float2 ds = __fmul2_rn(pr, gr);
      if constexpr (F != kNoCap) ds = __fmul2_rn(ds, f);
      pk[2 * i + k] = pack2<BF16>(pr.x, pr.y);
      dk[2 * i + k] = pack2<BF16>(ds.x, ds.y);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void grad_block_kv_scored(uint32_t tX, uint32_t tY, const float* lv, const float* dv,
                                                     const ScoreParams& sc, float2 c2, const ScoreBlock& sb) {
  constexpr float kLog2e = 1.4426950408889634f;
  const int u = threadIdx.x & 3;
  float2 nl2[4], dl[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 l2 = *reinterpret_cast<const float2*>(lv + 8 * i + 2 * u);
    nl2[i] = __fmul2_rn(l2, make_float2(-kLog2e, -kLog2e));
    const float2 d2 = *reinterpret_cast<const float2*>(dv + 8 * i + 2 * u);
    dl[i] = make_float2(-d2.x, -d2.y);
  }
  const bool capped = sc.cap != 0.f, biased = sc.slopes != nullptr;
  constexpr uint32_t kHalfLanes = 16u << 16;
  uint32_t xs[32], ys[16], pk[8], dk[8];
  auto store = [&](uint32_t off) {
    tmem_st16x128b_x4(tX + off, pk);
    tmem_st16x128b_x4(tY + off, dk);
  };
  const bool fast = !sb.edge && (sb.side != 0 || !biased);
  tmem_ld16x256b_x4(tX, xs);
  tmem_ld16x256b_x4(tX + kHalfLanes, xs + 16);
  tmem_ld_wait();
  if (fast && (!capped || all_small<32>(xs, sc))) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      tmem_ld16x256b_x4(tY + h * kHalfLanes, ys);
      tmem_ld_wait();
      if (!capped) grad16_kv_scored<BF16, true, kNoCap, true>(xs + 16 * h, ys, pk, dk, h, nl2, dl, sc, c2, sb);
      else if (biased) grad16_kv_scored<BF16, true, kCapSmall, true>(xs + 16 * h, ys, pk, dk, h, nl2, dl, sc, c2, sb);
      else grad16_kv_scored<BF16, true, kCapSmall, false>(xs + 16 * h, ys, pk, dk, h, nl2, dl, sc, c2, sb);
      store(h * kHalfLanes);
    }
    return;
  }
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    tmem_ld16x256b_x4(tX + h * kHalfLanes, xs);
    tmem_ld16x256b_x4(tY + h * kHalfLanes, ys);
    tmem_ld_wait();
    if (capped) grad16_kv_scored<BF16, false, kCapAny, true>(xs, ys, pk, dk, h, nl2, dl, sc, c2, sb);
    else grad16_kv_scored<BF16, false, kNoCap, true>(xs, ys, pk, dk, h, nl2, dl, sc, c2, sb);
    store(h * kHalfLanes);
  }
}

}  // namespace

// GENERAL = true is the instantiation for packed variable-length batches and
// window bands (the layouts of BwdParams; "Inside FlashAttention" §6.1):
// the CTA finds its sample from cu_seqlens, streams only the partner blocks
// that meet its tile's band, and masks blocks crossing either band edge.
// SCORED: modified scores and a prefix, in the general instantiation's rows and
// blocks.
template <int D, bool BF16, bool KV_OUTER, bool GENERAL, bool SCORED>
__global__ void __launch_bounds__(kBwdThreads, 1)
    fa_bwd_main_kernel(const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_a2,
                       const __grid_constant__ CUtensorMap tm_b1, const __grid_constant__ CUtensorMap tm_b2,
                       const ScoredParams<BwdParams, SCORED> p) {
  static_assert(GENERAL || !SCORED, "modified scores take the general instantiation");
  using L = BwdLayout<D>;
  using GA = typename L::GA;
  using GB = typename L::GB;
  using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int kPN = kPartnerRows;
  constexpr float kLog2e = 1.4426950408889634f;
  // Barrier tests before a wait blocks (mbar_wait): measured per pass at
  // causal B4 H16 S4096 D64 and B2 H32 S8192 D128 (a blocking try returns
  // some hundred cycles after the phase completes when the SM is busy): the
  // MMA warps gain in both passes except the D = 128 dQ pass, the other
  // waits only in the D <= 64 dK/dV pass; the dK/dV pass runs its tests
  // unrolled, the dQ pass eight per loop iteration.
  constexpr int kSpinMma = (D <= 64 || KV_OUTER) ? 64 : 0;
  constexpr int kSpinOther = (D <= 64 && KV_OUTER) ? 64 : 0;
  constexpr int kUnrollMma = (kSpinMma > 0 && KV_OUTER) ? kSpinMma : (kSpinMma > 0 ? 8 : 1);
  constexpr int kUnrollOther = kSpinOther > 0 ? kSpinOther : 1;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* bar_afull = bars;
  uint64_t* bar_bfull = bars + 1;
  uint64_t* bar_empty = bar_bfull + L::kStages;
  uint64_t* bar_xyfull = bar_empty + L::kStages;  // [buffers]
  uint64_t* bar_accissued = bar_xyfull + L::kXYBufs;  // [buffers] accumulation reading it issued
  uint64_t* bar_pfull = bar_accissued + L::kXYBufs;     // [4] block i's P, dS stored: bar_pfull[i % 4]
  uint64_t* bar_accfinal = bar_pfull + kPFullBars;
  uint64_t* bar_drain = bar_accfinal + 1;               // [2] one per MMA warp
  uint64_t* bar_btmp = bar_drain + 2;  // SCORED: a block whose rows past a packed sample are still to be cleared
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  float* vecs = reinterpret_cast<float*>(smem + L::kOffVec);

  const int warp = warp_index();
  const int lane = threadIdx.x & 31;
  // Head of the CTA's own tiles: a K/V head in the dK/dV pass, a query head in
  // the dQ pass.  K/V head h serves query heads h*group .. h*group+group-1; in
  // the dK/dV pass kv_splits CTAs share a K/V head, CTA `kv_part` taking the
  // group's heads kv_part*hpc .. kv_part*hpc+hpc-1.
  int cx, cy;
  cta_coords(!p.causal, &cx, &cy);
  const int bh = KV_OUTER ? cx / p.kv_splits : cx;
  const int kv_part = KV_OUTER ? cx - bh * p.kv_splits : 0;
  const int hpc = KV_OUTER ? p.group / p.kv_splits : 1;
  // General instantiation: the sample of a packed batch.  Head indices are
  // global (b*H + h) in the fixed-length layout and within a token when
  // packed: own_h for the CTA's own tiles, pz0 for the first partner head.
  const int heads_own = KV_OUTER ? p.heads / p.group : p.heads;  // per batch entry
  int S_ = p.S, tok0 = 0, own_h = bh;
  int pz0 = KV_OUTER ? bh * p.group + kv_part * hpc : bh / p.group;
  bool packed = false;
  if constexpr (GENERAL) {
    packed = p.cu_seqlens != nullptr;
    if (packed) {
      const int b = bh / heads_own;
      // (A CTA that leaves here or below still waits for the kernel before it: were all of
      // a grid's CTAs to leave at once, what follows on the stream could start beside it.)
      if (!packed_sample(p.cu_seqlens, b, p.S, p.total, p.err, &tok0, &S_)) {
        griddep_wait();
        return;
      }
      own_h = bh - b * heads_own;
      pz0 = KV_OUTER ? own_h * p.group + kv_part * hpc : own_h / p.group;
    }
  }
  const int S = S_;
  const int nt = p.n_tiles;
  const int np = (S + kPN - 1) / kPN;
  const int64_t rowbase = static_cast<int64_t>(bh) * S;
  // Row r of head h: L and Delta at h * lstride + loff + r (general instantiation).
  const int lstride = (GENERAL && packed) ? p.total : S;
  const int loff = tok0;
  // Own tile; heavy tiles first under the causal mask (key tile 0 and query
  // tile nt-1 see the most partners).
  const int own = KV_OUTER ? cy : (p.causal ? nt - 1 - cy : cy);
  const int own0 = own * 128;
  if constexpr (GENERAL) {
    if (own0 >= S) {  // packed batch: this CTA lies past its sample
      griddep_wait();
      return;
    }
  }
  // Window (general instantiation): key j is visible to query i iff i - wl <= j <= i + wr.
  const int wl = GENERAL ? p.win_left : 0;
  const int wr = GENERAL ? p.win_right : 0;
  // Partner blocks [first, last_excl): queries j - wr .. j + wl of the tile's
  // keys (dK/dV pass) or keys i - wl .. i + wr of its queries (dQ pass).
  int first, last_excl;
  int pfx = 0;  // keys before it are visible to every row
  if constexpr (SCORED) pfx = prefix_len(p.sc, bh / heads_own, S);
  if constexpr (GENERAL) {
    const int below = KV_OUTER ? wr : wl, above = KV_OUTER ? wl : wr;
    first = max(0, own0 - below) / kPN;
    last_excl = min(np, min(S - 1, own0 + 127 + above) / kPN + 1);
    if constexpr (SCORED) {
      if (KV_OUTER && own0 < pfx) first = 0;
      if (!KV_OUTER) last_excl = min(np, max(min(S - 1, own0 + 127 + wr), pfx - 1) / kPN + 1);
    }
  } else {
    first = (KV_OUTER && p.causal) ? own0 / kPN : 0;
    last_excl = (!KV_OUTER && p.causal) ? min(np, (own0 + 127) / kPN + 1) : np;
  }
  // Partner blocks per partner head; the dK/dV pass streams them for each of
  // the group's query heads in turn and sums over all of them.
  const int nper = last_excl - first;
  const int niter = KV_OUTER ? hpc * nper : nper;

  if (threadIdx.x == 0) {
    mbar_init(bar_afull, 1);
    for (int s = 0; s < L::kStages; ++s) {
      // dK/dV pass: the producer's TMA arrival plus one cp.async arrival per
      // producer lane for the block's L and Delta vectors.
      mbar_init(&bar_bfull[s], KV_OUTER ? 33 : 1);
      mbar_init(&bar_empty[s], 1);
    }
    for (int b = 0; b < L::kXYBufs; ++b) {
      mbar_init(&bar_xyfull[b], 1);
      mbar_init(&bar_accissued[b], 1);
    }
    for (int b = 0; b < kPFullBars; ++b) {
      mbar_init(&bar_pfull[b], 8);  // one arrival per warp of the block's group
    }
    mbar_init(bar_accfinal, 1);
    mbar_init(&bar_drain[0], 1);
    mbar_init(&bar_drain[1], 1);
    if constexpr (SCORED) mbar_init(bar_btmp, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sA1 = smem_u32(smem + L::kOffA1);
  const uint32_t sA2 = smem_u32(smem + L::kOffA2);
  const uint32_t sB1 = smem_u32(smem + L::kOffB1);
  const uint32_t sB2 = smem_u32(smem + L::kOffB2);
  // The dQ pass after the dK/dV pass may start its CTAs as this grid's last
  // ones run; it reads nothing this pass writes before its griddep_wait.
  // (SCORED: the other way round; the dK/dV pass reads the dQ pass's Delta.)
  if constexpr (KV_OUTER || SCORED) griddep_launch_dependents();

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    // Lane 0 issues the TMA copies; in the dK/dV pass every lane also copies
    // two entries of the block's L and Delta vectors (queries past S read 0:
    // their Q and dO rows are zero-filled, so P dO and dS vanish there).
    if (lane == 0) {
      prefetch_tmap(&tm_a1);
      prefetch_tmap(&tm_a2);
      prefetch_tmap(&tm_b1);
      prefetch_tmap(&tm_b2);
      mbar_arrive_expect_tx(bar_afull, 2 * GA::kTileBytes);
#pragma unroll
      for (int ch = 0; ch < GA::kChunks; ++ch) {
        tma_load_3d(smem + L::kOffA1 + ch * GA::kChunkBytes, &tm_a1, bar_afull, ch * (GA::kRowBytes / 2),
                    (GENERAL && packed) ? own_h : own0, (GENERAL && packed) ? tok0 + own0 : own_h);
        tma_load_3d(smem + L::kOffA2 + ch * GA::kChunkBytes, &tm_a2, bar_afull, ch * (GA::kRowBytes / 2),
                    (GENERAL && packed) ? own_h : own0, (GENERAL && packed) ? tok0 + own0 : own_h);
      }
    }
    int it = 0;
    int n_cleared = 0;
    // Partner head and block of iteration `it`, stepped along without divisions.
    int pz = pz0;
    int pblk = first;
    for (; it < niter; ++it, ++pblk) {
      if (KV_OUTER && pblk == last_excl) {
        pblk = first;
        ++pz;
      }
      const int st = it % L::kStages;
      const int use = it / L::kStages;
      if (use > 0 && !warp_wait<kSpinOther, kUnrollOther>(&bar_empty[st], (use - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutLoad)) break;
      const int r0 = pblk * kPN;
      // Partner rows past a packed sample's end belong to the next sample or to none
      // and may hold NaN: they are set to zero (0 * NaN is not 0).
      const bool clear = SCORED && packed && r0 + kPN > S;
      uint64_t* bbar = SCORED && clear ? bar_btmp : &bar_bfull[st];
      if (lane == 0) {
        mbar_arrive_expect_tx(bbar, 2 * GB::kTileBytes);
#pragma unroll
        for (int ch = 0; ch < GB::kChunks; ++ch) {
          tma_load_3d(smem + L::kOffB1 + st * GB::kTileBytes + ch * GB::kChunkBytes, &tm_b1, bbar,
                      ch * (GB::kRowBytes / 2), (GENERAL && packed) ? pz : r0, (GENERAL && packed) ? tok0 + r0 : pz);
          tma_load_3d(smem + L::kOffB2 + st * GB::kTileBytes + ch * GB::kChunkBytes, &tm_b2, bbar,
                      ch * (GB::kRowBytes / 2), (GENERAL && packed) ? pz : r0, (GENERAL && packed) ? tok0 + r0 : pz);
        }
      }
      if (SCORED && clear) {
        drain_wait(bar_btmp, n_cleared & 1, p.err);
        ++n_cleared;
        clear_rows<GB>(smem + L::kOffB1 + st * GB::kTileBytes, kPN, S - r0);
        clear_rows<GB>(smem + L::kOffB2 + st * GB::kTileBytes, kPN, S - r0);
        if (lane == 0) mbar_arrive(&bar_bfull[st]);
      }
      if constexpr (KV_OUTER) {
        // Delta may come from the kernel just before this one (a programmatic
        // dependent launch after the persistent dQ pass): wait for it before the
        // first read.  Nothing read earlier is written by that kernel.
        if (it == 0) griddep_wait();
        float* v = vecs + st * 2 * kPN;
#pragma unroll
        for (int h = 0; h < kPN; h += 32) {
          const int q = r0 + h + lane;
          if constexpr (GENERAL) {
            // Partner queries past the sample read L = +inf and Delta = 0, so
            // their P and dS are exactly 0 (when packed, their Q and dO rows
            // are the next sample's).
            const int64_t src = static_cast<int64_t>(pz) * lstride + loff + (q < S ? q : S - 1);
            cp_async_4(v + h + lane, q < S ? p.lse + src : &g_pos_inf, true);
            cp_async_4(v + kPN + h + lane, p.delta + src, q < S);
          } else {
            const int64_t src = static_cast<int64_t>(pz) * S + (q < S ? q : S - 1);
            cp_async_4(v + h + lane, p.lse + src, q < S);
            cp_async_4(v + kPN + h + lane, p.delta + src, q < S);
          }
        }
        cp_async_mbar_arrive(&bar_bfull[st]);
      }
    }
    // A CTA with no partner block (a key tile past a short sample's end) still
    // waits for the kernel before it, so that this grid never completes before
    // that one, whatever follows on the stream.
    if constexpr (KV_OUTER) {
      if (it == 0) griddep_wait();
    }
    // Teardown: every copy issued must land before the CTA exits.
    if (lane == 0) drain_wait(bar_afull, 0, p.err);
    for (int x = (it > L::kStages ? it - L::kStages : 0); x < it; ++x)
      drain_wait(&bar_bfull[x % L::kStages], (x / L::kStages) & 1, p.err);
  } else if (warp == kMmaWarp || warp == kAccWarp) {
    // ------------------------------------------------------------ MMA issuers
    // Warp kMmaWarp issues the score products X, Y of every block, warp
    // kAccWarp the accumulations, so X, Y keep the tensor core busy while the
    // accumulation of a block waits for its P and dS.  Both run converged and
    // one elected lane issues each MMA.  X, Y(i) reuse buffer i % kXYBufs,
    // last read by the accumulation of block i - kXYBufs: kAccWarp signals
    // acc_issued after issuing it (tcgen05 fences order the two warps' MMAs,
    // which the tensor core then runs in issue order).
    constexpr uint32_t idesc_xy = make_idesc_f16(BF16, 128, kPN, false, false);
    constexpr uint32_t idesc_acc = make_idesc_f16(BF16, 128, D, false, true);
    const AccFlags accf = runtime_flags(S);
    bool ok = true;
    if (warp == kMmaWarp) {
      const uint64_t a1_desc = make_sdesc(sA1, 16, 8 * GA::kRowBytes, GA::kSwz);
      const uint64_t a2_desc = make_sdesc(sA2, 16, 8 * GA::kRowBytes, GA::kSwz);
      ok = warp_wait(bar_afull, 0, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
      constexpr bool kAFromTmem = !KV_OUTER && !SCORED && L::kTmemA;  // (SCORED: those columns are M's)
      if (kAFromTmem && ok) {
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          tmem_cp_128x256b_warp(tmem + L::kColA1 + 8 * kk, desc_plus(a1_desc, kmajor_step_bytes<D, 128>(kk)));
          tmem_cp_128x256b_warp(tmem + L::kColA2 + 8 * kk, desc_plus(a2_desc, kmajor_step_bytes<D, 128>(kk)));
        }
      }
      for (int i = 0; ok && i < niter; ++i) {
        const int st = i % L::kStages;
        const int b = i % L::kXYBufs;
        ok = warp_wait<kSpinMma, kUnrollMma>(&bar_bfull[st], (i / L::kStages) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
        if (ok && i >= L::kXYBufs)
          ok = warp_wait<kSpinMma, kUnrollMma>(&bar_accissued[b], ((i / L::kXYBufs) - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tb = tmem + 128u * b;
        const uint64_t b1 = make_sdesc(sB1 + st * GB::kTileBytes, 16, 8 * GB::kRowBytes, GB::kSwz);
        const uint64_t b2 = make_sdesc(sB2 + st * GB::kTileBytes, 16, 8 * GB::kRowBytes, GB::kSwz);
        if constexpr (kAFromTmem) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts_warp(tb, tmem + L::kColA1 + 8 * kk, desc_plus(b1, kmajor_step_bytes<D, kPN>(kk)), idesc_xy,
                        kk > 0 ? accf.on : accf.off);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ts_warp(tb + 64, tmem + L::kColA2 + 8 * kk, desc_plus(b2, kmajor_step_bytes<D, kPN>(kk)), idesc_xy,
                        kk > 0 ? accf.on : accf.off);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_warp(tb, desc_plus(a1_desc, kmajor_step_bytes<D, 128>(kk)),
                        desc_plus(b1, kmajor_step_bytes<D, kPN>(kk)), idesc_xy, kk > 0 ? accf.on : accf.off);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_warp(tb + 64, desc_plus(a2_desc, kmajor_step_bytes<D, 128>(kk)),
                        desc_plus(b2, kmajor_step_bytes<D, kPN>(kk)), idesc_xy, kk > 0 ? accf.on : accf.off);
        }
        mma_commit_warp(&bar_xyfull[b]);
      }
      mma_commit_warp(&bar_drain[0]);
      drain_wait(&bar_drain[0], 0, p.err);
    } else {
      for (int x = 0; ok && x < niter; ++x) {
        const int st = x % L::kStages;
        const int b = x % L::kXYBufs;
        ok = warp_wait<kSpinMma, kUnrollMma>(&bar_pfull[x % kPFullBars], (x / kPFullBars) & 1, abort_flag, p.err, p.wait_ns,
                                             kErrTimeoutMma);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tb = tmem + 128u * b;
        const uint64_t b1 = make_sdesc(sB1 + st * GB::kTileBytes, GB::kChunkBytes, 8 * GB::kRowBytes, GB::kSwz);
        const uint64_t b2 = make_sdesc(sB2 + st * GB::kTileBytes, GB::kChunkBytes, 8 * GB::kRowBytes, GB::kSwz);
        if constexpr (KV_OUTER) {
#pragma unroll
          for (int kk = 0; kk < kPN / 16; ++kk)  // dV += P^T dO_i
            mma_ts_warp(tmem + L::kColAcc1, tb + packed_col(kk), desc_plus(b2, mnmajor_step_bytes<D>(kk)), idesc_acc,
                        (x > 0 || kk > 0) ? accf.on : accf.off);
#pragma unroll
          for (int kk = 0; kk < kPN / 16; ++kk)  // dK += dS^T Q_i
            mma_ts_warp(tmem + L::kColAcc2, tb + 64 + packed_col(kk), desc_plus(b1, mnmajor_step_bytes<D>(kk)),
                        idesc_acc, (x > 0 || kk > 0) ? accf.on : accf.off);
        } else {
#pragma unroll
          for (int kk = 0; kk < kPN / 16; ++kk)  // dQ += dS K_j
            mma_ts_warp(tmem + L::kColAcc1, tb + 64 + packed_col(kk), desc_plus(b1, mnmajor_step_bytes<D>(kk)),
                        idesc_acc, (x > 0 || kk > 0) ? accf.on : accf.off);
          if constexpr (SCORED) {
#pragma unroll
            for (int kk = 0; kk < kPN / 16; ++kk)  // M += (P o f) K_j
              mma_ts_warp(tmem + L::kColAcc2, tb + packed_col(kk), desc_plus(b1, mnmajor_step_bytes<D>(kk)),
                          idesc_acc, (x > 0 || kk > 0) ? accf.on : accf.off);
          }
        }
        // The stage's tiles are free once this completes: X, Y(x) finished
        // before the group could form P and dS.
        mma_commit_warp(&bar_empty[st]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_accissued[b]);
      }
      if (ok) mma_commit_warp(bar_accfinal);
      mma_commit_warp(&bar_drain[1]);
      drain_wait(&bar_drain[1], 0, p.err);
    }
  } else {
    // ------------------------------------------------------------ softmax-gradient warps 0-15
    // Group g = warp / 8 turns blocks g, g + 2, ... into P and dS, so two
    // blocks are in this stage at once while the tensor core works on a
    // third.  In a group, warp w owns TMEM lanes 32 (w % 4).. and partner
    // columns 32 ((w / 4) % 2)...
    const int g = warp >> 3;
    const int q4 = warp & 3;
    const int hf = (warp >> 2) & 1;
    const int col0 = 32 * hf;
    const int my = own0 + q4 * 32 + lane;  // key index (dK/dV pass) or query index (dQ pass)
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    const float sl2 = p.scale_log2;
    const float2 c2 = make_float2(sl2, sl2);
    // dQ pass: this thread's query row owns its L2 = L * log2 e and Delta
    // (rows past S: L2 = +inf, so their probabilities are exactly 0).
    float my_l2 = INFINITY, my_delta = 0.f;
    // Delta comes from a kernel before this one, which may still be running
    // when this pass is a programmatic dependent launch.
    if (!KV_OUTER) griddep_wait();
    if (!KV_OUTER && my < S) {
      const int64_t li = GENERAL ? static_cast<int64_t>(own_h) * lstride + loff + my : rowbase + my;
      my_l2 = p.lse[li] * kLog2e;
      // (SCORED: from L2, since another CTA may write its rows of the same line)
      my_delta = SCORED ? __ldcg(p.delta + li) : p.delta[li];
    }
    ScoreBlock sb;
    sb.slope = 0.f;
    float2 p_dp = make_float2(0.f, 0.f);  // SCORED, dQ pass: the thread's share of its row's P . dP
    bool alive = true;
    int ph = pz0;  // SCORED, dK/dV pass: partner head of the block
    int pi = g;  // i modulo nper: the partner block within its head (dK/dV pass)
    if constexpr (KV_OUTER) {
      while (pi >= nper) {
        pi -= nper;
        ++ph;
      }
    }
    for (int i = g; i < niter; i += kBwdGroups) {
      const int st = i % L::kStages;
      const int partner0 = (first + (KV_OUTER ? pi : i)) * kPN;
      if constexpr (SCORED) {
        if (p.sc.slopes != nullptr)
          sb.slope = __ldg(p.sc.slopes + (KV_OUTER ? ph : bh) % p.heads) * kLog2e;
      }
      if constexpr (KV_OUTER) {
        pi += kBwdGroups;
        while (pi >= nper) {
          pi -= nper;
          ++ph;
        }
      }
      bool ok = true;
      if constexpr (KV_OUTER) ok = warp_wait<kSpinOther, kUnrollOther>(&bar_bfull[st], (i / L::kStages) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax);
      ok = ok && warp_wait<kSpinOther, kUnrollOther>(&bar_xyfull[i % L::kXYBufs], (i / L::kXYBufs) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax);
      if (!ok) {
        alive = false;
        break;
      }
      tc_fence_after();
      const uint32_t tX = tmem + lane_base + 128u * (i % L::kXYBufs) + col0;
      const uint32_t tY = tX + 64;
      const float* lv = vecs + st * 2 * kPN + col0;  // L of this warp's 32 partner queries (dK/dV pass)
      const float* dv = lv + kPN;                    // and their Delta
      // Diagonal blocks under the causal mask: the dK/dV pass zeroes partner
      // column c where query partner0 + col0 + c < key `my`, the dQ pass where
      // key partner0 + col0 + c > query `my`.  Rows and columns past S need no
      // mask: their zero-filled operands make their terms vanish (see above).
      // Off-diagonal blocks (all but one or two per tile) take the path with
      // no per-element compare or select.
      if constexpr (GENERAL) {
        // Window band: blocks crossing either edge are masked; the dQ pass
        // also masks a packed sample's ragged last key block (those rows are
        // the next sample's).  Partner queries past S have P = 0 from L = +inf.
        if constexpr (SCORED) {
          // (causal without a prefix: a key behind its query is hidden, whatever its bias)
          const int key0 = KV_OUTER ? own0 : partner0, key1 = key0 + (KV_OUTER ? 127 : kPN - 1);
          const int row0 = KV_OUTER ? partner0 : own0, row1 = row0 + (KV_OUTER ? kPN - 1 : 127);
          sb.side = key1 <= row0 || (p.causal && pfx == 0) ? -1 : key0 >= row1 ? 1 : 0;
          if (fabsf(sb.slope) > kSteep) sb.side = 0;  // each distance by itself, as in the forward
          if constexpr (KV_OUTER) {
            sb.edge = (partner0 < own0 + 127 - wr && pfx < own0 + 128) || partner0 + kPN - 1 > own0 + wl;
            sb.d0 = own0 + q4 * 32 - partner0 - col0;
            sb.hi = wr;
            sb.wl = wl;
            sb.pfx = pfx - partner0 - col0;
            grad_block_kv_scored<BF16>(tX, tY, lv, dv, p.sc, c2, sb);
          } else {
            // (A key past S is a row of zeros, but a bias that favours distance would give it
            // an infinite P.)
            sb.edge = partner0 + kPN - 1 > max(own0 + wr, pfx - 1) || partner0 < own0 + 127 - wl || partner0 + kPN > S;
            sb.hi = max(min(S - 1, my + wr), pfx - 1) - partner0 - col0;
            sb.lo = my - wl - partner0 - col0;
            sb.d0 = partner0 + col0 - my;
            grad_block_scored<BF16>(tX, tY, p.sc, c2, my_l2, my_delta, sb, p_dp);
          }
        } else if constexpr (KV_OUTER) {
          const bool edge = partner0 < own0 + 127 - wr || partner0 + kPN - 1 > own0 + wl;
          const int lim0 = own0 + q4 * 32 - partner0 - col0;
          if (edge)
            grad_block_kv<BF16, true, true>(tX, tY, lv, dv, c2, lim0, wr, wl);
          else
            grad_block_kv<BF16, false>(tX, tY, lv, dv, c2, lim0);
        } else {
          const bool edge = partner0 + kPN - 1 > own0 + wr || partner0 < own0 + 127 - wl ||
                            (packed && partner0 + kPN > S);
          const int hi = min(S - 1, my + wr) - partner0 - col0;
          const int lo = my - wl - partner0 - col0;
          if (edge)
            grad_block<BF16, KV_OUTER, true, true>(tX, tY, lv, dv, c2, my_l2, my_delta, hi, lo);
          else
            grad_block<BF16, KV_OUTER, false>(tX, tY, lv, dv, c2, my_l2, my_delta, hi);
        }
      } else {
        const bool diag = p.causal && (KV_OUTER ? partner0 < own0 + 128 : partner0 + kPN - 1 > own0);
        const int lim = my - partner0 - col0;
        if constexpr (KV_OUTER) {
          const int lim0 = own0 + q4 * 32 - partner0 - col0;
          if (diag)
            grad_block_kv<BF16, true>(tX, tY, lv, dv, c2, lim0);
          else
            grad_block_kv<BF16, false>(tX, tY, lv, dv, c2, lim0);
        } else {
          if (diag)
            grad_block<BF16, KV_OUTER, true>(tX, tY, lv, dv, c2, my_l2, my_delta, lim);
          else
            grad_block<BF16, KV_OUTER, false>(tX, tY, lv, dv, c2, my_l2, my_delta, lim);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_pfull[i % kPFullBars]);
    }
    // ------------------------------------------------------------ epilogue
    // SCORED, dQ pass.  Delta of the stored O is off by half a 16-bit step of O, which
    // for rows whose weight lies on few keys is more than what is left of dP - Delta
    // there.  The row's P . dP, summed here in fp32, is the exact one: dQ formed with
    // the other is off by their difference times M = (P o f) K, and the dK/dV pass
    // after this one reads it in the other's place.
    float off_delta = 0.f;
    if constexpr (SCORED && !KV_OUTER) {
      float* part = vecs;  // [4][128]: group and column half, row
      part[(2 * g + hf) * 128 + q4 * 32 + lane] = p_dp.x + p_dp.y;
      named_sync(1, 32 * kProducerWarp);  // (the warps whose wait ran out come here too)
      const float* mine = part + q4 * 32 + lane;
      const float exact = (mine[0] + mine[128]) + (mine[256] + mine[384]);
      off_delta = exact - my_delta;
      if (warp < 4 && my < S) p.delta[static_cast<int64_t>(own_h) * lstride + loff + my] = exact;
    }
    const bool done = alive && mbar_wait<kSpinOther, kUnrollOther>(bar_accfinal, 0, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax);
    // The 16 warps split the accumulator columns of their 32 rows into up to
    // four parts of at least 16 columns.
    constexpr int kParts = D >= 64 ? 4 : D / 16;
    constexpr int kEpiCols = D / kParts;
    const int col_part = warp >> 2;
    if (__all_sync(0xffffffffu, done) && col_part < kParts) {
      tc_fence_after();
      const int c_begin = col_part * kEpiCols;
      const bool row_ok = my < S;
      // Output row: bh*S + my (fixed length) or (tok0 + my)*heads_own + own_h (packed).
      const int mr = row_ok ? my : 0;
      const int64_t orow = (GENERAL && packed) ? static_cast<int64_t>(tok0 + mr) * heads_own + own_h : rowbase + mr;
      const size_t off = static_cast<size_t>(orow) * D;
      const uint32_t t_acc = tmem + lane_base;
      if constexpr (KV_OUTER) {
        if (p.kv_splits == 1) {
          elem_t* dv_row = reinterpret_cast<elem_t*>(p.dv) + off;
          elem_t* dk_row = reinterpret_cast<elem_t*>(p.dk) + off;
#pragma unroll
          for (int c = c_begin; c < c_begin + kEpiCols; c += 16) {
            uint32_t v16[16];
            tmem_ld16(t_acc + L::kColAcc1 + c, v16);
            if (row_ok) store_row16<BF16>(dv_row + c, v16, 1.f);
            tmem_ld16(t_acc + L::kColAcc2 + c, v16);
            if (row_ok) store_row16<BF16>(dk_row + c, v16, p.scale);
          }
        } else {
          // This CTA's share of the group: fp32 rows [dV | scale * dK] of
          // partial `kv_part`, summed by the reduce kernel.
          const int64_t n_rows = (GENERAL && packed) ? static_cast<int64_t>(p.total) * heads_own
                                                     : static_cast<int64_t>(p.BH / p.group) * S;
          float* prow = p.dkv_part + ((static_cast<int64_t>(kv_part) * n_rows + orow) * (2 * D));
#pragma unroll
          for (int c = c_begin; c < c_begin + kEpiCols; c += 16) {
            uint32_t v16[16];
            tmem_ld16(t_acc + L::kColAcc1 + c, v16);
            if (row_ok) store_row16_f32(prow + c, v16, 1.f);
            tmem_ld16(t_acc + L::kColAcc2 + c, v16);
            if (row_ok) store_row16_f32(prow + D + c, v16, p.scale);
          }
        }
      } else {
        elem_t* dq_row = reinterpret_cast<elem_t*>(p.dq) + off;
#pragma unroll
        for (int c = c_begin; c < c_begin + kEpiCols; c += 16) {
          uint32_t v16[16];
          tmem_ld16(t_acc + L::kColAcc1 + c, v16);
          if constexpr (SCORED) {
            uint32_t m16[16];
            tmem_ld16(t_acc + L::kColAcc2 + c, m16);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              v16[e] = __float_as_uint(fmaf(-off_delta, __uint_as_float(m16[e]), __uint_as_float(v16[e])));
          }
          if (row_ok) store_row16<BF16>(dq_row + c, v16, p.scale);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

namespace {

// Launches `kern`; with `dependent`, as a programmatic dependent launch of the
// kernel before it on `stream`: its CTAs may start while that kernel's last
// CTAs still run, and it waits (griddep_wait) before reading that kernel's output.
template <typename... Params, typename... Args>
cudaError_t launch_kernel(void (*kern)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                          bool dependent, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = dependent ? attr : nullptr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, bool BF16, bool KV_OUTER, bool GENERAL, bool SCORED = false>
cudaError_t launch_main_t(const CUtensorMap& a1, const CUtensorMap& a2, const CUtensorMap& b1,
                          const CUtensorMap& b2, const ScoredParams<BwdParams, SCORED>& p, cudaStream_t stream,
                          bool dependent = false) {
  using L = BwdLayout<D>;
  auto kern = fa_bwd_main_kernel<D, BF16, KV_OUTER, GENERAL, SCORED>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
  if (e != cudaSuccess) return e;
  // dK/dV pass: kv_splits CTAs per (K/V head, key tile); dQ pass: one per (query head, query tile).
  dim3 grid(KV_OUTER ? p.BH / p.group * p.kv_splits : p.BH, p.n_tiles);
  return launch_kernel(kern, grid, kBwdThreads, L::kSmemBytes, stream, dependent, a1, a2, b1, b2, p);
}

}  // namespace

}  // namespace fa
