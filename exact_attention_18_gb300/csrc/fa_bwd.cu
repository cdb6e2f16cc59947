// Backward kernels: recompute backward of exact attention.
//
// With P = exp(S - L) rebuilt from the forward's logsumexp ("从零训练语言模型
// （第二部分）" §使用 LSE 连接正向和反向传播) and the row vector
// Delta_i = rowsum(dO o O) (CS336 Assignment 2 write-up, "4. Problem
// (flash_backward)", the vector D):
//   dV = P^T dO,   dP = dO V^T,   dS = P o (dP - Delta),
//   dQ = scale * dS K,   dK = scale * dS^T Q          ("第二部分" §反向传播).
//
// Three launches (the two-kernel split of the CS336 write-up, "6.
// FlashAttention-2 Leaderboard", which avoids atomics):
//   1. bwd_preprocess: Delta for every row (memory-bound, one pass over O, dO);
//   2. bwd_main<KV_OUTER = true>:  one CTA per (b*h, 128-key tile), looping
//      over 64-row blocks of the queries that see it; dV and dK stay in TMEM;
//   3. bwd_main<KV_OUTER = false>: one CTA per (b*h, 128-query tile), looping
//      over 64-row blocks of its visible keys; dQ stays in TMEM.
// Causal: a key tile starts at its diagonal query block, a query tile stops at
// its diagonal key block (CS336 write-up, causal tile skipping); the mask is
// applied element-wise only on diagonal blocks and on ragged tails.
//
// bwd_main is written once for both passes.  Per partner block i it computes
// two score-shaped products with the CTA's resident 128-row tiles A1, A2 as
// the MMA A operands and the streamed 64-row tiles B1, B2 as B operands:
//   X = A1 B1^T,  Y = A2 B2^T
//     dK/dV pass: A1 = K, A2 = V, B1 = Q_i, B2 = dO_i -> X = S^T, Y = dP^T
//     dQ pass:    A1 = Q, A2 = dO, B1 = K_j, B2 = V_j -> X = S,   Y = dP
// so TMEM lane = the CTA's own row (key or query).  Sixteen softmax-gradient
// warps in two groups of eight turn X, Y into P and dS (16-bit, written back
// into TMEM over X and Y); group g takes the blocks i with i mod 2 = g, and in
// a group warp w owns TMEM lanes 32(w%4).. and partner columns 32((w/4)%2)...
// The MMA warp then accumulates, with A read from TMEM:
//     dK/dV pass: dV += P^T dO_i,  dK += dS^T Q_i    (B = B2, B1 read MN-major)
//     dQ pass:    dQ += dS K_j                       (B = B1 read MN-major)
// X and Y of block i live in TMEM buffer i mod kXYBufs (128 columns; three
// buffers for D <= 64, two for D = 128).  One warp issues X, Y of every block
// as soon as its tiles and buffer are free, another the accumulations, so a
// group that finishes block i usually finds block i + 2 already computed, and
// both groups work while the tensor core runs the products around them.  In the dK/dV pass the producer warp also copies the
// block's L and Delta (one value per partner query) into the stage with
// cp.async, completing on the same barrier as the block's tiles.
#include "fa_bwd_main.cuh"

namespace fa {

// ------------------------------------------------------------------ preprocess
// Delta_i = sum_d dO_id * O_id in fp32.  D/8 lanes share a row, each reading
// 16 bytes of O and of dO; a shuffle tree sums the group.  The whole warp
// calls it (the shuffles need all 32 lanes); `valid` says whether this lane's
// row exists.  Every lane of the group gets the row's sum.
// This lane's part of the row's dot product: 8 elements of O (a) and of dO (b).
template <bool BF16>
__device__ __forceinline__ float chunk_dot(const uint4 a, const uint4 b) {
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
  const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
  float acc = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 fa2, fb2;
    if constexpr (BF16) {
      fa2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&aw[i]));
      fb2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&bw[i]));
    } else {
      fa2 = __half22float2(*reinterpret_cast<const __half2*>(&aw[i]));
      fb2 = __half22float2(*reinterpret_cast<const __half2*>(&bw[i]));
    }
    acc = fmaf(fa2.x, fb2.x, acc);
    acc = fmaf(fa2.y, fb2.y, acc);
  }
  return acc;
}

// Sum over the row's D/8 lanes.
template <int D>
__device__ __forceinline__ float row_sum(float acc) {
#pragma unroll
  for (int off = D / 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  return acc;
}

template <int D, bool BF16>
__device__ __forceinline__ float row_delta(const void* o, const void* dout, int64_t row, bool valid) {
  float acc = 0.f;
  if (valid) {
    const int64_t off = (row * D + ((threadIdx.x & 31) % (D / 8)) * 8) * 2;  // this lane's 8 elements
    acc = chunk_dot<BF16>(*reinterpret_cast<const uint4*>(static_cast<const char*>(o) + off),
                          *reinterpret_cast<const uint4*>(static_cast<const char*>(dout) + off));
  }
  return row_sum<D>(acc);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) fa_bwd_preprocess_kernel(const BwdParams p, int64_t rows) {
  // The dK/dV pass after it may start its CTAs; it waits for this grid before reading Delta.
  griddep_launch_dependents();
  constexpr int kTpr = D / 8;           // threads per row
  constexpr int kRowsPerWarp = 32 / kTpr;
  const int lane = threadIdx.x & 31;
  const int sub = lane % kTpr;
  const int64_t warp_id = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t n_warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  // Whole warps iterate together so the shuffles always see 32 lanes.
  for (int64_t r0 = warp_id * kRowsPerWarp; r0 < rows; r0 += n_warps * kRowsPerWarp) {
    const int64_t row = r0 + lane / kTpr;
    const float acc = row_delta<D, BF16>(p.o, p.dout, row, row < rows);
    // Row `row` of [B*H*S, D] (fixed length) or of [T*H, D] (packed: token
    // row / H, head row % H, whose Delta lives at [head, token]).
    if (row < rows && sub == 0)
      p.delta[p.cu_seqlens ? (row % p.heads) * p.total + row / p.heads : row] = acc;
  }
}

// ------------------------------------------------------------------ dK/dV partial sums
// dV, dK = sum over the kv_splits partials (fixed order, fp32), rounded once.
// One thread per 8 consecutive columns of a [dV | scale*dK] row.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) fa_bwd_dkv_reduce_kernel(const BwdParams p, int64_t rows) {
  constexpr int kG = 2 * D / 8;  // 8-column groups per row
  const int64_t n = rows * kG;
  const int64_t part_stride = rows * 2 * D;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < n;
       e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = e / kG;
    const int cg = static_cast<int>(e - row * kG);
    const float* src = p.dkv_part + row * 2 * D + cg * 8;
    float4 a = reinterpret_cast<const float4*>(src)[0];
    float4 b = reinterpret_cast<const float4*>(src)[1];
    for (int sp = 1; sp < p.kv_splits; ++sp) {
      const float4 a2 = reinterpret_cast<const float4*>(src + sp * part_stride)[0];
      const float4 b2 = reinterpret_cast<const float4*>(src + sp * part_stride)[1];
      a.x += a2.x; a.y += a2.y; a.z += a2.z; a.w += a2.w;
      b.x += b2.x; b.y += b2.y; b.z += b2.z; b.w += b2.w;
    }
    const uint4 w = make_uint4(pack2<BF16>(a.x, a.y), pack2<BF16>(a.z, a.w), pack2<BF16>(b.x, b.y),
                               pack2<BF16>(b.z, b.w));
    const bool is_dv = cg < D / 8;
    void* out = is_dv ? p.dv : p.dk;
    const int col = (is_dv ? cg : cg - D / 8) * 8;
    reinterpret_cast<uint4*>(static_cast<char*>(out) + (row * D + col) * 2)[0] = w;
  }
}

// Persistent version of the dQ pass for fixed-length calls at D <= 64: a grid
// of at most one CTA per SM, each running the pipeline of fa_bwd_main_kernel
// (roles, TMEM layout, barriers; Q and dO copied into TMEM) over a sequence of
// the non-persistent grid's query tiles ("work items", in that grid's launch
// order: heaviest first under the causal mask), dealt to the CTAs in a snake
// (round r gives item r*P + c to CTA c when r is even and r*P + P-1-c when it
// is odd, P CTAs).  Between items nothing drains: the producer loads the next
// item's first key blocks, then its Q and dO tiles as soon as the current
// item's copies of them into TMEM are done (a_empty); the score-product warp
// computes the next item's first X, Y while the softmax-gradient warps store
// the current item's dQ; the accumulation warp starts the next item's dQ once
// those stores have read it out of TMEM (acc_free).  Barrier phases run on
// across items: key stages, X/Y buffers and the "P stored" barriers by a
// running block count, the tile and accumulator barriers by item.
// One more warp computes Delta = rowsum(dO o O) of each item's rows (the
// preprocess kernel's arithmetic, from O and dO rows staged in shared memory
// one item ahead), writes it to the workspace for the dK/dV pass, which then
// runs after this one, and hands it to the softmax-gradient warps through
// shared memory (delta_full), so the backward needs no separate Delta kernel.
template <int D>
struct DqpLayout {
  static constexpr int kOffStage = (BwdLayout<D>::kSmemUsed + 127) / 128 * 128;
  static constexpr int kStageBytes = 128 * D * 2;  // one item's rows of one tensor
  static constexpr int kSmemBytes = kOffStage + 2 * kStageBytes + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "persistent dQ pass: shared memory");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kDqpThreads, 1)
    fa_bwd_dqp_kernel(const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_a2,
                      const __grid_constant__ CUtensorMap tm_b1, const __grid_constant__ CUtensorMap tm_b2,
                      const BwdParams p, int n_items) {
  using L = BwdLayout<D>;
  using DL = DqpLayout<D>;
  static_assert(D <= 64 && L::kTmemA, "persistent dQ pass: D <= 64, Q and dO in TMEM");
  using GA = typename L::GA;
  using GB = typename L::GB;
  using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int kPN = kPartnerRows;
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr int kS = L::kStages;
  constexpr int kB = L::kXYBufs;
  // Barrier tests before blocking as in fa_bwd_main_kernel's dQ pass at D <= 64.
  constexpr int kSpinMma = 64;
  constexpr int kUnrollMma = 8;
  constexpr int kPreBlocks = 4;  // key blocks of the next item loaded before its Q, dO tiles

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* bar_afull = bars;
  uint64_t* bar_bfull = bars + 1;
  uint64_t* bar_empty = bar_bfull + kS;
  uint64_t* bar_xyfull = bar_empty + kS;         // [buffers]
  uint64_t* bar_accissued = bar_xyfull + kB;     // [buffers] accumulation reading it issued
  uint64_t* bar_pfull = bar_accissued + kB;      // [4] block i's dS stored: bar_pfull[i % 4]
  uint64_t* bar_accfinal = bar_pfull + kPFullBars;
  uint64_t* bar_drain = bar_accfinal + 1;        // [2] one per MMA warp
  uint64_t* bar_aempty = bar_drain + 2;          // the item's Q, dO copies into TMEM done
  uint64_t* bar_accfree = bar_aempty + 1;        // the item's dQ read out by all 16 warps
  uint64_t* bar_deltafull = bar_accfree + 1;     // [2] item n's Delta in buffer n % 2
  uint64_t* bar_deltafree = bar_deltafull + 2;   // [2] buffer n % 2 read by all 16 warps
  uint64_t* bar_stage = bar_deltafree + 2;       // an item's O, dO rows in the staging buffer
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  // Two 128-row Delta buffers (item n in buffer n % 2), in the stage vectors'
  // space, which the dQ pass does not use.
  float* delta_buf = reinterpret_cast<float*>(smem + L::kOffVec);
  static_assert(L::kStages * 2 * kPartnerRows >= 2 * 128, "Delta buffers");

  const int warp = warp_index();
  const int lane = threadIdx.x & 31;
  const int S = p.S;
  const int nt = p.n_tiles;
  const int np = (S + kPN - 1) / kPN;
  const int gx = p.BH;
  const int P = static_cast<int>(gridDim.x);
  const int c = static_cast<int>(blockIdx.x);
  auto item_at = [&](int r) -> int {
    const int k = r * P + ((r & 1) ? (P - 1 - c) : c);
    return k < n_items ? k : -1;
  };
  // One work item: query head bh, its 128-row tile at own0, key blocks 0 .. nb-1.
  struct Item {
    int bh, kvh, own0, nb;
  };
  auto decode = [&](int k) -> Item {
    int cx, cy;
    if (p.causal) {  // x fastest: every head's heaviest tile first
      cy = k / gx;
      cx = k - cy * gx;
    } else {         // y fastest: one head's tiles in a row
      cx = k / nt;
      cy = k - cx * nt;
    }
    Item it;
    it.bh = cx;
    it.kvh = cx / p.group;
    it.own0 = (p.causal ? nt - 1 - cy : cy) * 128;
    it.nb = p.causal ? min(np, (it.own0 + 127) / kPN + 1) : np;
    return it;
  };

  if (threadIdx.x == 0) {
    mbar_init(bar_afull, 1);
    for (int s = 0; s < kS; ++s) {
      mbar_init(&bar_bfull[s], 1);
      mbar_init(&bar_empty[s], 1);
    }
    for (int b = 0; b < kB; ++b) {
      mbar_init(&bar_xyfull[b], 1);
      mbar_init(&bar_accissued[b], 1);
    }
    for (int b = 0; b < kPFullBars; ++b) mbar_init(&bar_pfull[b], 8);
    mbar_init(bar_accfinal, 1);
    mbar_init(&bar_drain[0], 1);
    mbar_init(&bar_drain[1], 1);
    mbar_init(bar_aempty, 1);
    mbar_init(bar_accfree, 16);  // one arrival per softmax-gradient warp
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bar_deltafull[b], 1);
      mbar_init(&bar_deltafree[b], 16);  // one arrival per softmax-gradient warp
    }
    mbar_init(bar_stage, 1);
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
  // The dK/dV pass that follows may start its CTAs as this grid's CTAs exit
  // (it cannot share an SM with one: registers); it waits for this grid to
  // complete before it reads Delta.
  griddep_launch_dependents();

  if (warp == kDeltaWarp) {
    // ------------------------------------------------------------ Delta warp
    // Lane 0 copies an item's O and dO rows into the staging buffer (one bulk
    // copy each: a fixed-length head's rows are contiguous), one item ahead of
    // the sums; D/8 lanes per row then sum dO o O from shared memory.
    constexpr int kTpr = D / 8;
    constexpr int kRowsPerStep = 32 / kTpr;
    uint8_t* stage_o = smem + DL::kOffStage;
    uint8_t* stage_do = stage_o + DL::kStageBytes;
    auto issue = [&](const Item& w) {
      const uint32_t bytes = static_cast<uint32_t>(min(128, S - w.own0)) * D * 2;
      const int64_t off = (static_cast<int64_t>(w.bh) * S + w.own0) * D * 2;
      mbar_arrive_expect_tx(bar_stage, 2 * bytes);
      // Evict-first: these lines are not read again soon (the item's dO tile
      // comes in through its own TMA load), and K, V blocks keep their L2 place.
      const uint64_t pol = l2_policy_evict_first();
      bulk_load(stage_o, static_cast<const char*>(p.o) + off, bytes, bar_stage, pol);
      bulk_load(stage_do, static_cast<const char*>(p.dout) + off, bytes, bar_stage, pol);
    };
    bool ok = true;
    int k = item_at(0);
    if (k >= 0 && lane == 0) issue(decode(k));
    int n = 0;  // item n's copy is the one in flight
    for (int r = 0; ok && k >= 0; ++r, ++n) {
      const Item w = decode(k);
      const int64_t rowbase = static_cast<int64_t>(w.bh) * S;
      // Buffer n % 2 was last read at the start of item n - 2.
      if (n >= 2)
        ok = warp_wait(&bar_deltafree[n & 1], ((n >> 1) - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax);
      if (ok) ok = warp_wait(bar_stage, n & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax);
      if (!ok) break;
      float* buf = delta_buf + (n & 1) * 128;
      const int sub16 = (lane % kTpr) * 16;
#pragma unroll 4
      for (int r0 = 0; r0 < 128; r0 += kRowsPerStep) {
        const int rr = r0 + lane / kTpr;
        const int row = w.own0 + rr;
        float acc = 0.f;
        if (row < S)
          acc = chunk_dot<BF16>(*reinterpret_cast<const uint4*>(stage_o + rr * D * 2 + sub16),
                                *reinterpret_cast<const uint4*>(stage_do + rr * D * 2 + sub16));
        const float d = row_sum<D>(acc);
        if (lane % kTpr == 0) {
          buf[rr] = d;
          if (row < S) p.delta[rowbase + row] = d;
        }
      }
      k = item_at(r + 1);
      __syncwarp();
      if (lane == 0) {
        if (k >= 0) {  // the staging buffer is free again: the next item's rows
          fence_proxy_async_smem();
          issue(decode(k));
        }
        mbar_arrive(&bar_deltafull[n & 1]);  // release: the buffer's writes reach its waiters
      }
    }
    // Given up: the copy in flight lands before the CTA exits.
    if (!ok && lane == 0) drain_wait(bar_stage, n & 1, p.err);
  } else if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer (lane 0)
    if (lane == 0) {
      prefetch_tmap(&tm_a1);
      prefetch_tmap(&tm_a2);
      prefetch_tmap(&tm_b1);
      prefetch_tmap(&tm_b2);
      bool ok = true;
      int it = 0;  // key blocks loaded so far
      int n = 0;   // items whose Q, dO tiles were loaded
      for (int r = 0; ok; ++r) {
        const int k = item_at(r);
        if (k < 0) break;
        const Item w = decode(k);
        auto load_block = [&](int x) -> bool {
          const int st = it % kS;
          const int use = it / kS;
          if (use > 0 && !mbar_wait(&bar_empty[st], (use - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutLoad))
            return false;
          mbar_arrive_expect_tx(&bar_bfull[st], 2 * GB::kTileBytes);
#pragma unroll
          for (int ch = 0; ch < GB::kChunks; ++ch) {
            tma_load_3d(smem + L::kOffB1 + st * GB::kTileBytes + ch * GB::kChunkBytes, &tm_b1, &bar_bfull[st],
                        ch * (GB::kRowBytes / 2), x * kPN, w.kvh);
            tma_load_3d(smem + L::kOffB2 + st * GB::kTileBytes + ch * GB::kChunkBytes, &tm_b2, &bar_bfull[st],
                        ch * (GB::kRowBytes / 2), x * kPN, w.kvh);
          }
          ++it;
          return true;
        };
        const int pre = min(w.nb, kPreBlocks);
        for (int x = 0; ok && x < pre; ++x) ok = load_block(x);
        // Q and dO, once the previous item's copies of them into TMEM are done.
        if (ok && n > 0) ok = mbar_wait(bar_aempty, (n - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutLoad);
        if (!ok) break;
        mbar_arrive_expect_tx(bar_afull, 2 * GA::kTileBytes);
#pragma unroll
        for (int ch = 0; ch < GA::kChunks; ++ch) {
          tma_load_3d(smem + L::kOffA1 + ch * GA::kChunkBytes, &tm_a1, bar_afull, ch * (GA::kRowBytes / 2), w.own0,
                      w.bh);
          tma_load_3d(smem + L::kOffA2 + ch * GA::kChunkBytes, &tm_a2, bar_afull, ch * (GA::kRowBytes / 2), w.own0,
                      w.bh);
        }
        ++n;
        for (int x = pre; ok && x < w.nb; ++x) ok = load_block(x);
      }
      // Teardown: every copy issued must land before the CTA exits.
      if (n > 0) drain_wait(bar_afull, (n - 1) & 1, p.err);
      for (int x = (it > kS ? it - kS : 0); x < it; ++x) drain_wait(&bar_bfull[x % kS], (x / kS) & 1, p.err);
    }
  } else if (warp == kMmaWarp || warp == kAccWarp) {
    // ------------------------------------------------------------ MMA issuers
    constexpr uint32_t idesc_xy = make_idesc_f16(BF16, 128, kPN, false, false);
    constexpr uint32_t idesc_acc = make_idesc_f16(BF16, 128, D, false, true);
    const AccFlags accf = runtime_flags(S);
    bool ok = true;
    int i0 = 0;  // key blocks of the earlier items
    int n = 0;   // items
    if (warp == kMmaWarp) {
      const uint64_t a1_desc = make_sdesc(sA1, 16, 8 * GA::kRowBytes, GA::kSwz);
      const uint64_t a2_desc = make_sdesc(sA2, 16, 8 * GA::kRowBytes, GA::kSwz);
      for (int r = 0; ok; ++r) {
        const int k = item_at(r);
        if (k < 0) break;
        const Item w = decode(k);
        ok = warp_wait(bar_afull, n & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
        if (!ok) break;
        // Q and dO into TMEM (after the previous item's score products, which
        // read the columns they overwrite: the tensor core runs them in order).
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          tmem_cp_128x256b_warp(tmem + L::kColA1 + 8 * kk, desc_plus(a1_desc, kmajor_step_bytes<D, 128>(kk)));
          tmem_cp_128x256b_warp(tmem + L::kColA2 + 8 * kk, desc_plus(a2_desc, kmajor_step_bytes<D, 128>(kk)));
        }
        mma_commit_warp(bar_aempty);  // the shared-memory Q, dO are free once the copies land
        for (int x = 0; ok && x < w.nb; ++x) {
          const int i = i0 + x;
          const int st = i % kS;
          const int b = i % kB;
          ok = warp_wait<kSpinMma, kUnrollMma>(&bar_bfull[st], (i / kS) & 1, abort_flag, p.err, p.wait_ns,
                                               kErrTimeoutMma);
          if (ok && i >= kB)
            ok = warp_wait<kSpinMma, kUnrollMma>(&bar_accissued[b], ((i / kB) - 1) & 1, abort_flag, p.err,
                                                 p.wait_ns, kErrTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tb = tmem + 128u * b;
          const uint64_t b1 = make_sdesc(sB1 + st * GB::kTileBytes, 16, 8 * GB::kRowBytes, GB::kSwz);
          const uint64_t b2 = make_sdesc(sB2 + st * GB::kTileBytes, 16, 8 * GB::kRowBytes, GB::kSwz);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)  // X = S = Q K_j^T
            mma_ts_warp(tb, tmem + L::kColA1 + 8 * kk, desc_plus(b1, kmajor_step_bytes<D, kPN>(kk)), idesc_xy,
                        kk > 0 ? accf.on : accf.off);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)  // Y = dP = dO V_j^T
            mma_ts_warp(tb + 64, tmem + L::kColA2 + 8 * kk, desc_plus(b2, kmajor_step_bytes<D, kPN>(kk)), idesc_xy,
                        kk > 0 ? accf.on : accf.off);
          mma_commit_warp(&bar_xyfull[b]);
        }
        i0 += w.nb;
        ++n;
      }
      mma_commit_warp(&bar_drain[0]);
      drain_wait(&bar_drain[0], 0, p.err);
    } else {
      for (int r = 0; ok; ++r) {
        const int k = item_at(r);
        if (k < 0) break;
        const Item w = decode(k);
        for (int x = 0; ok && x < w.nb; ++x) {
          const int i = i0 + x;
          const int st = i % kS;
          const int b = i % kB;
          ok = warp_wait<kSpinMma, kUnrollMma>(&bar_pfull[i % kPFullBars], (i / kPFullBars) & 1, abort_flag, p.err,
                                               p.wait_ns, kErrTimeoutMma);
          // The item's first accumulation overwrites dQ: the previous item's
          // must have been read out.
          if (ok && x == 0 && n > 0)
            ok = warp_wait(bar_accfree, (n - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tb = tmem + 128u * b;
          const uint64_t b1 = make_sdesc(sB1 + st * GB::kTileBytes, GB::kChunkBytes, 8 * GB::kRowBytes, GB::kSwz);
#pragma unroll
          for (int kk = 0; kk < kPN / 16; ++kk)  // dQ += dS K_j
            mma_ts_warp(tmem + L::kColAcc1, tb + 64 + packed_col(kk), desc_plus(b1, mnmajor_step_bytes<D>(kk)),
                        idesc_acc, (x > 0 || kk > 0) ? accf.on : accf.off);
          mma_commit_warp(&bar_empty[st]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_accissued[b]);
        }
        if (!ok) break;
        mma_commit_warp(bar_accfinal);  // the item's dQ is complete once this lands
        i0 += w.nb;
        ++n;
      }
      mma_commit_warp(&bar_drain[1]);
      drain_wait(&bar_drain[1], 0, p.err);
    }
  } else {
    // ------------------------------------------------------------ softmax-gradient warps 0-15
    const int g = warp >> 3;
    const int q4 = warp & 3;
    const int hf = (warp >> 2) & 1;
    const int col0 = 32 * hf;
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    const float sl2 = p.scale_log2;
    const float2 c2 = make_float2(sl2, sl2);
    constexpr int kParts = D >= 64 ? 4 : D / 16;
    constexpr int kEpiCols = D / kParts;
    const int col_part = warp >> 2;
    bool alive = true;
    int i0 = 0;
    int n = 0;
    for (int r = 0; alive; ++r) {
      const int k = item_at(r);
      if (k < 0) break;
      const Item w = decode(k);
      const int my = w.own0 + q4 * 32 + lane;  // this thread's query
      const int64_t rowbase = static_cast<int64_t>(w.bh) * S;
      // This row's L2 = L * log2 e (rows past S: L2 = +inf, so P = 0 exactly)
      // and its Delta, from the Delta warp.
      const float my_l2 = my < S ? p.lse[rowbase + my] * kLog2e : INFINITY;
      if (!warp_wait(&bar_deltafull[n & 1], (n >> 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax)) {
        alive = false;
        break;
      }
      const float my_delta = delta_buf[(n & 1) * 128 + q4 * 32 + lane];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_deltafree[n & 1]);
      // This group's blocks of the item: global block indices i0 + x with (i0 + x) % 2 == g.
      for (int x = (g - i0) & 1; x < w.nb; x += kBwdGroups) {
        const int i = i0 + x;
        const int partner0 = x * kPN;
        if (!warp_wait(&bar_xyfull[i % kB], (i / kB) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax)) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t tX = tmem + lane_base + 128u * (i % kB) + col0;
        const uint32_t tY = tX + 64;
        const int lim = my - partner0 - col0;
        if (p.causal && partner0 + kPN - 1 > w.own0)  // the diagonal blocks: keys after the query masked
          grad_block<BF16, false, true>(tX, tY, nullptr, nullptr, c2, my_l2, my_delta, lim);
        else
          grad_block<BF16, false, false>(tX, tY, nullptr, nullptr, c2, my_l2, my_delta, lim);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_pfull[i % kPFullBars]);
      }
      if (!alive) break;
      // ---------------------------------------------------------- epilogue of the item
      if (!warp_wait(bar_accfinal, n & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax)) {
        alive = false;
        break;
      }
      tc_fence_after();
      if (col_part < kParts) {
        const int c_begin = col_part * kEpiCols;
        const bool row_ok = my < S;
        const size_t off = static_cast<size_t>(rowbase + (row_ok ? my : 0)) * D;
        const uint32_t t_acc = tmem + lane_base;
        elem_t* dq_row = reinterpret_cast<elem_t*>(p.dq) + off;
#pragma unroll
        for (int cc = c_begin; cc < c_begin + kEpiCols; cc += 16) {
          uint32_t v16[16];
          tmem_ld16(t_acc + L::kColAcc1 + cc, v16);
          if (row_ok) store_row16<BF16>(dq_row + cc, v16, p.scale);
        }
      }
      // dQ is read: the next item's accumulation may overwrite it.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_accfree);
      i0 += w.nb;
      ++n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Persistent version of the dK/dV pass for fixed-length calls at D <= 64 with
// at most 32 partner blocks per work item on average (launch_dkdv_t decides):
// a grid of at most one CTA per SM, each running the pipeline of
// fa_bwd_main_kernel over a sequence of the per-tile grid's key tiles (work
// items, in that grid's launch order, dealt in a snake as in the persistent
// dQ pass).  Between items: the producer loads the next item's first partner
// blocks, then its K and V tiles as soon as the current item's last score
// products have read them (a_empty); the accumulation warp starts the next
// item's dV, dK once all 16 softmax-gradient warps have read the current ones
// out of TMEM (acc_free).  The per-block steps run slower inside this
// kernel's item loops than in the per-tile kernel, so it pays only while the
// per-item overlap outweighs that: measured (whole backward, causal fp16 D64)
// B8 H16 S1024 111 -> 101 us, B4 H16 S2048 147 -> 139 us, B4 H16 S4096 417 ->
// 411 us, but B2 H16 S8192 703 -> 724 us and grouped K/V heads at S4096
// (hpc 2 or 4 query heads per item) 5-7 % slower.
template <int D, bool BF16>
__global__ void __launch_bounds__(kBwdThreads, 1)
    fa_bwd_dkdvp_kernel(const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_a2,
                        const __grid_constant__ CUtensorMap tm_b1, const __grid_constant__ CUtensorMap tm_b2,
                        const BwdParams p, int gx, int n_items) {
  using L = BwdLayout<D>;
  static_assert(D <= 64, "persistent dK/dV pass: D <= 64");
  using GA = typename L::GA;
  using GB = typename L::GB;
  using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int kPN = kPartnerRows;
  constexpr int kS = L::kStages;
  constexpr int kB = L::kXYBufs;
  // Barrier tests before blocking as in fa_bwd_main_kernel's dK/dV pass, but
  // not unrolled: this kernel's longer code ran faster with the small loops
  // (c2 242 -> 234 us).
  constexpr int kSpinMma = 64;
  constexpr int kSpinOther = 64;
  constexpr int kUnrollMma = 1;
  constexpr int kUnrollOther = 1;
  constexpr int kPreBlocks = 4;  // partner blocks of the next item loaded before its resident tiles

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* bar_afull = bars;
  uint64_t* bar_bfull = bars + 1;
  uint64_t* bar_empty = bar_bfull + kS;
  uint64_t* bar_xyfull = bar_empty + kS;         // [buffers]
  uint64_t* bar_accissued = bar_xyfull + kB;     // [buffers] accumulation reading it issued
  uint64_t* bar_pfull = bar_accissued + kB;      // [4] block i's P, dS stored: bar_pfull[i % 4]
  uint64_t* bar_accfinal = bar_pfull + kPFullBars;
  uint64_t* bar_drain = bar_accfinal + 1;        // [2] one per MMA warp
  uint64_t* bar_aempty = bar_drain + 2;          // the item's last score products (last reads of A1, A2) done
  uint64_t* bar_accfree = bar_aempty + 1;        // the item's accumulators read out by all 16 warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  float* vecs = reinterpret_cast<float*>(smem + L::kOffVec);

  const int warp = warp_index();
  const int lane = threadIdx.x & 31;
  const int S = p.S;
  const int nt = p.n_tiles;
  const int np = (S + kPN - 1) / kPN;
  const int hpc = p.group / p.kv_splits;  // query heads per CTA share of a K/V head
  const int gy = nt;
  const int P = static_cast<int>(gridDim.x);
  const int c = static_cast<int>(blockIdx.x);
  auto item_at = [&](int r) -> int {
    const int k = r * P + ((r & 1) ? (P - 1 - c) : c);
    return k < n_items ? k : -1;
  };
  // One work item: the tile the non-persistent grid's CTA number k took.
  struct Item {
    int bh, kv_part, pz0, own0, first, nper, niter;
  };
  auto decode = [&](int k) -> Item {
    int cx, cy;
    if (p.causal) {  // x fastest: every head's heaviest tile first
      cy = k / gx;
      cx = k - cy * gx;
    } else {         // y fastest: one head's tiles in a row
      cx = k / gy;
      cy = k - cx * gy;
    }
    Item it;
    it.bh = cx / p.kv_splits;  // K/V head
    it.kv_part = cx - it.bh * p.kv_splits;
    it.pz0 = it.bh * p.group + it.kv_part * hpc;  // first partner (query) head
    it.own0 = cy * 128;
    it.first = p.causal ? it.own0 / kPN : 0;
    it.nper = np - it.first;
    it.niter = hpc * it.nper;
    return it;
  };

  if (threadIdx.x == 0) {
    mbar_init(bar_afull, 1);
    for (int s = 0; s < kS; ++s) {
      mbar_init(&bar_bfull[s], 33);  // the TMA arrival + one cp.async arrival per producer lane
      mbar_init(&bar_empty[s], 1);
    }
    for (int b = 0; b < kB; ++b) {
      mbar_init(&bar_xyfull[b], 1);
      mbar_init(&bar_accissued[b], 1);
    }
    for (int b = 0; b < kPFullBars; ++b) mbar_init(&bar_pfull[b], 8);
    mbar_init(bar_accfinal, 1);
    mbar_init(&bar_drain[0], 1);
    mbar_init(&bar_drain[1], 1);
    mbar_init(bar_aempty, 1);
    mbar_init(bar_accfree, 16);  // one arrival per softmax-gradient warp
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

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tm_a1);
      prefetch_tmap(&tm_a2);
      prefetch_tmap(&tm_b1);
      prefetch_tmap(&tm_b2);
    }
    bool ok = true;
    int it = 0;  // partner blocks loaded so far
    int n = 0;   // items whose resident tiles were loaded
    for (int r = 0; ok; ++r) {
      const int k = item_at(r);
      if (k < 0) break;
      const Item w = decode(k);
      // Partner head and block of the next block to load, stepped without divisions.
      int pz = w.pz0, pblk = w.first;
      auto load_block = [&](int) -> bool {
        const int st = it % kS;
        const int use = it / kS;
        if (use > 0 && !warp_wait<kSpinOther, kUnrollOther>(&bar_empty[st], (use - 1) & 1, abort_flag, p.err,
                                                             p.wait_ns, kErrTimeoutLoad))
          return false;
        const int r0 = pblk * kPN;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_bfull[st], 2 * GB::kTileBytes);
#pragma unroll
          for (int ch = 0; ch < GB::kChunks; ++ch) {
            tma_load_3d(smem + L::kOffB1 + st * GB::kTileBytes + ch * GB::kChunkBytes, &tm_b1, &bar_bfull[st],
                        ch * (GB::kRowBytes / 2), r0, pz);
            tma_load_3d(smem + L::kOffB2 + st * GB::kTileBytes + ch * GB::kChunkBytes, &tm_b2, &bar_bfull[st],
                        ch * (GB::kRowBytes / 2), r0, pz);
          }
        }
        // The block's L and Delta (partner queries past S read 0: their Q and
        // dO rows are zero-filled, so P dO and dS vanish there).  Delta may come
        // from the kernel just before this one (as in fa_bwd_main_kernel).
        if (it == 0) griddep_wait();
        float* v = vecs + st * 2 * kPN;
#pragma unroll
        for (int h = 0; h < kPN; h += 32) {
          const int q = r0 + h + lane;
          const int64_t src = static_cast<int64_t>(pz) * S + (q < S ? q : S - 1);
          cp_async_4(v + h + lane, p.lse + src, q < S);
          cp_async_4(v + kPN + h + lane, p.delta + src, q < S);
        }
        cp_async_mbar_arrive(&bar_bfull[st]);
        if (++pblk == w.first + w.nper) {
          pblk = w.first;
          ++pz;
        }
        ++it;
        return true;
      };
      const int pre = min(w.niter, kPreBlocks);
      for (int x = 0; ok && x < pre; ++x) ok = load_block(x);
      // The resident tiles, once the previous item's score products have read them.
      if (ok && n > 0)
        ok = warp_wait(bar_aempty, (n - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutLoad);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar_afull, 2 * GA::kTileBytes);
#pragma unroll
        for (int ch = 0; ch < GA::kChunks; ++ch) {
          tma_load_3d(smem + L::kOffA1 + ch * GA::kChunkBytes, &tm_a1, bar_afull, ch * (GA::kRowBytes / 2), w.own0,
                      w.bh);
          tma_load_3d(smem + L::kOffA2 + ch * GA::kChunkBytes, &tm_a2, bar_afull, ch * (GA::kRowBytes / 2), w.own0,
                      w.bh);
        }
      }
      ++n;
      for (int x = pre; ok && x < w.niter; ++x) ok = load_block(x);
    }
    // Teardown: every copy issued must land before the CTA exits.
    if (lane == 0 && n > 0) drain_wait(bar_afull, (n - 1) & 1, p.err);
    for (int x = (it > kS ? it - kS : 0); x < it; ++x) drain_wait(&bar_bfull[x % kS], (x / kS) & 1, p.err);
  } else if (warp == kMmaWarp || warp == kAccWarp) {
    // ------------------------------------------------------------ MMA issuers
    constexpr uint32_t idesc_xy = make_idesc_f16(BF16, 128, kPN, false, false);
    constexpr uint32_t idesc_acc = make_idesc_f16(BF16, 128, D, false, true);
    const AccFlags accf = runtime_flags(S);
    bool ok = true;
    int i0 = 0;  // partner blocks of the earlier items
    int n = 0;   // items
    if (warp == kMmaWarp) {
      const uint64_t a1_desc = make_sdesc(sA1, 16, 8 * GA::kRowBytes, GA::kSwz);
      const uint64_t a2_desc = make_sdesc(sA2, 16, 8 * GA::kRowBytes, GA::kSwz);
      for (int r = 0; ok; ++r) {
        const int k = item_at(r);
        if (k < 0) break;
        const Item w = decode(k);
        ok = warp_wait(bar_afull, n & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
        if (!ok) break;
        for (int x = 0; ok && x < w.niter; ++x) {
          const int i = i0 + x;
          const int st = i % kS;
          const int b = i % kB;
          ok = warp_wait<kSpinMma, kUnrollMma>(&bar_bfull[st], (i / kS) & 1, abort_flag, p.err, p.wait_ns,
                                               kErrTimeoutMma);
          if (ok && i >= kB)
            ok = warp_wait<kSpinMma, kUnrollMma>(&bar_accissued[b], ((i / kB) - 1) & 1, abort_flag, p.err,
                                                 p.wait_ns, kErrTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tb = tmem + 128u * b;
          const uint64_t b1 = make_sdesc(sB1 + st * GB::kTileBytes, 16, 8 * GB::kRowBytes, GB::kSwz);
          const uint64_t b2 = make_sdesc(sB2 + st * GB::kTileBytes, 16, 8 * GB::kRowBytes, GB::kSwz);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)  // X = S^T = K Q_i^T
            mma_ss_warp(tb, desc_plus(a1_desc, kmajor_step_bytes<D, 128>(kk)),
                        desc_plus(b1, kmajor_step_bytes<D, kPN>(kk)), idesc_xy, kk > 0 ? accf.on : accf.off);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)  // Y = dP^T = V dO_i^T
            mma_ss_warp(tb + 64, desc_plus(a2_desc, kmajor_step_bytes<D, 128>(kk)),
                        desc_plus(b2, kmajor_step_bytes<D, kPN>(kk)), idesc_xy, kk > 0 ? accf.on : accf.off);
          mma_commit_warp(&bar_xyfull[b]);
        }
        if (!ok) break;
        mma_commit_warp(bar_aempty);  // the item's last reads of A1, A2 are issued
        i0 += w.niter;
        ++n;
      }
      mma_commit_warp(&bar_drain[0]);
      drain_wait(&bar_drain[0], 0, p.err);
    } else {
      for (int r = 0; ok; ++r) {
        const int k = item_at(r);
        if (k < 0) break;
        const Item w = decode(k);
        for (int x = 0; ok && x < w.niter; ++x) {
          const int i = i0 + x;
          const int st = i % kS;
          const int b = i % kB;
          ok = warp_wait<kSpinMma, kUnrollMma>(&bar_pfull[i % kPFullBars], (i / kPFullBars) & 1, abort_flag, p.err,
                                               p.wait_ns, kErrTimeoutMma);
          // The item's first accumulation overwrites the accumulators: the
          // previous item's must have been read out.
          if (ok && x == 0 && n > 0)
            ok = warp_wait(bar_accfree, (n - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tb = tmem + 128u * b;
          const uint64_t b1 = make_sdesc(sB1 + st * GB::kTileBytes, GB::kChunkBytes, 8 * GB::kRowBytes, GB::kSwz);
          const uint64_t b2 = make_sdesc(sB2 + st * GB::kTileBytes, GB::kChunkBytes, 8 * GB::kRowBytes, GB::kSwz);
#pragma unroll
          for (int kk = 0; kk < kPN / 16; ++kk)  // dV += P^T dO_i
            mma_ts_warp(tmem + L::kColAcc1, tb + packed_col(kk), desc_plus(b2, mnmajor_step_bytes<D>(kk)), idesc_acc,
                        (x > 0 || kk > 0) ? accf.on : accf.off);
#pragma unroll
          for (int kk = 0; kk < kPN / 16; ++kk)  // dK += dS^T Q_i
            mma_ts_warp(tmem + L::kColAcc2, tb + 64 + packed_col(kk), desc_plus(b1, mnmajor_step_bytes<D>(kk)),
                        idesc_acc, (x > 0 || kk > 0) ? accf.on : accf.off);
          mma_commit_warp(&bar_empty[st]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_accissued[b]);
        }
        if (!ok) break;
        mma_commit_warp(bar_accfinal);  // the item's accumulators are complete once this lands
        i0 += w.niter;
        ++n;
      }
      mma_commit_warp(&bar_drain[1]);
      drain_wait(&bar_drain[1], 0, p.err);
    }
  } else {
    // ------------------------------------------------------------ softmax-gradient warps 0-15
    const int g = warp >> 3;
    const int q4 = warp & 3;
    const int hf = (warp >> 2) & 1;
    const int col0 = 32 * hf;
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    const float sl2 = p.scale_log2;
    const float2 c2 = make_float2(sl2, sl2);
    constexpr int kParts = D >= 64 ? 4 : D / 16;
    constexpr int kEpiCols = D / kParts;
    const int col_part = warp >> 2;
    bool alive = true;
    int i0 = 0;
    int n = 0;
    for (int r = 0; alive; ++r) {
      const int k = item_at(r);
      if (k < 0) break;
      const Item w = decode(k);
      const int my = w.own0 + q4 * 32 + lane;  // this thread's key
      const int64_t rowbase = static_cast<int64_t>(w.bh) * S;
      // This group's blocks of the item: global block indices i0 + x with (i0 + x) % 2 == g.
      const int x0 = (g - i0) & 1;
      int pi = x0;  // x modulo nper (the partner block within its head), stepped without divisions
      if (pi >= w.nper) pi -= w.nper;
      for (int x = x0; x < w.niter; x += kBwdGroups) {
        const int i = i0 + x;
        const int st = i % kS;
        const int partner0 = (w.first + pi) * kPN;
        pi += kBwdGroups;
        while (pi >= w.nper) pi -= w.nper;
        bool ok = warp_wait<kSpinOther, kUnrollOther>(&bar_bfull[st], (i / kS) & 1, abort_flag, p.err, p.wait_ns,
                                                      kErrTimeoutSoftmax);
        ok = ok && warp_wait<kSpinOther, kUnrollOther>(&bar_xyfull[i % kB], (i / kB) & 1, abort_flag, p.err,
                                                       p.wait_ns, kErrTimeoutSoftmax);
        if (!ok) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint32_t tX = tmem + lane_base + 128u * (i % kB) + col0;
        const uint32_t tY = tX + 64;
        const float* lv = vecs + st * 2 * kPN + col0;
        const float* dv = lv + kPN;
        // Diagonal blocks: partner queries before this key are masked.
        const int lim0 = w.own0 + q4 * 32 - partner0 - col0;
        if (p.causal && partner0 < w.own0 + 128)
          grad_block_kv<BF16, true>(tX, tY, lv, dv, c2, lim0);
        else
          grad_block_kv<BF16, false>(tX, tY, lv, dv, c2, lim0);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_pfull[i % kPFullBars]);
      }
      if (!alive) break;
      // ---------------------------------------------------------- epilogue of the item
      if (!warp_wait<kSpinOther, kUnrollOther>(bar_accfinal, n & 1, abort_flag, p.err, p.wait_ns,
                                               kErrTimeoutSoftmax)) {
        alive = false;
        break;
      }
      tc_fence_after();
      if (col_part < kParts) {
        const int c_begin = col_part * kEpiCols;
        const bool row_ok = my < S;
        const int64_t orow = rowbase + (row_ok ? my : 0);
        const size_t off = static_cast<size_t>(orow) * D;
        const uint32_t t_acc = tmem + lane_base;
        if (p.kv_splits == 1) {
          elem_t* dv_row = reinterpret_cast<elem_t*>(p.dv) + off;
          elem_t* dk_row = reinterpret_cast<elem_t*>(p.dk) + off;
#pragma unroll
          for (int cc = c_begin; cc < c_begin + kEpiCols; cc += 16) {
            uint32_t v16[16];
            tmem_ld16(t_acc + L::kColAcc1 + cc, v16);
            if (row_ok) store_row16<BF16>(dv_row + cc, v16, 1.f);
            tmem_ld16(t_acc + L::kColAcc2 + cc, v16);
            if (row_ok) store_row16<BF16>(dk_row + cc, v16, p.scale);
          }
        } else {
          // This CTA's share of the group: fp32 rows [dV | scale * dK] of partial kv_part.
          const int64_t n_rows = static_cast<int64_t>(p.BH / p.group) * S;
          float* prow = p.dkv_part + ((static_cast<int64_t>(w.kv_part) * n_rows + orow) * (2 * D));
#pragma unroll
          for (int cc = c_begin; cc < c_begin + kEpiCols; cc += 16) {
            uint32_t v16[16];
            tmem_ld16(t_acc + L::kColAcc1 + cc, v16);
            if (row_ok) store_row16_f32(prow + cc, v16, 1.f);
            tmem_ld16(t_acc + L::kColAcc2 + cc, v16);
            if (row_ok) store_row16_f32(prow + D + cc, v16, p.scale);
          }
        }
      }
      // The accumulators are read: the next item's accumulation may overwrite them.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_accfree);
      i0 += w.niter;
      ++n;
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

template <int D, bool BF16>
cudaError_t launch_pre_t(const BwdParams& p, int64_t rows, cudaStream_t stream) {
  const int64_t threads = rows * (D / 8);
  const int64_t blocks = (threads + 255) / 256;
  const int grid = static_cast<int>(blocks < 152 * 16 ? blocks : 152 * 16);
  fa_bwd_preprocess_kernel<D, BF16><<<grid, 256, 0, stream>>>(p, rows);
  return cudaGetLastError();
}

int bwd_sm_count() {
  static int n = 0;
  if (n == 0) {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
      n = v;
    if (n <= 0) n = 1;
  }
  return n;
}

template <int D, bool BF16>
cudaError_t launch_dq_persistent_t(const CUtensorMap& a1, const CUtensorMap& a2, const CUtensorMap& b1,
                                   const CUtensorMap& b2, const BwdParams& p, cudaStream_t stream) {
  constexpr int kSmem = DqpLayout<D>::kSmemBytes;
  auto kern = fa_bwd_dqp_kernel<D, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // Work items: the query tiles of the non-persistent grid (B*H x n_tiles).
  const int64_t n_items = static_cast<int64_t>(p.BH) * p.n_tiles;
  if (n_items <= 0) return cudaSuccess;
  if (n_items > (1LL << 30)) return cudaErrorInvalidValue;
  const int grid = static_cast<int>(n_items < bwd_sm_count() ? n_items : bwd_sm_count());
  kern<<<grid, kDqpThreads, kSmem, stream>>>(a1, a2, b1, b2, p, static_cast<int>(n_items));
  return cudaGetLastError();
}

// The dQ pass: the persistent kernel for fixed-length calls at D <= 64 (measured at causal
// B4 H16 S4096 D64 185 -> 165 us, B1 H16 S16384 D64 547 -> 538 us); at D = 128 the per-tile
// grid (the persistent kernel was as fast at B2 H32 S8192, 1.6 % slower at B1 H8 S32768).
template <int D, bool BF16>
cudaError_t launch_dq_t(bool general, const BwdMaps& m, const BwdParams& p, cudaStream_t stream, bool dependent) {
  if (general) return launch_main_t<D, BF16, false, true>(m.q128, m.do128, m.k64, m.v64, p, stream, dependent);
  if constexpr (D <= 64)  // the persistent kernel: bwd_dq_computes_delta(D, false)
    return launch_dq_persistent_t<D, BF16>(m.q128, m.do128, m.k64, m.v64, p, stream);
  else
    return launch_main_t<D, BF16, false, false>(m.q128, m.do128, m.k64, m.v64, p, stream, dependent);
}

template <int D, bool BF16>
cudaError_t launch_dkdv_persistent_t(const CUtensorMap& a1, const CUtensorMap& a2, const CUtensorMap& b1,
                                     const CUtensorMap& b2, const BwdParams& p, cudaStream_t stream,
                                     bool dependent) {
  using L = BwdLayout<D>;
  auto kern = fa_bwd_dkdvp_kernel<D, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
  if (e != cudaSuccess) return e;
  // Work items: the key tiles of the per-tile grid (K/V heads x kv_splits x n_tiles).
  const int gx = p.BH / p.group * p.kv_splits;
  const int64_t n_items = static_cast<int64_t>(gx) * p.n_tiles;
  if (n_items <= 0) return cudaSuccess;
  if (n_items > (1LL << 30)) return cudaErrorInvalidValue;
  const int grid = static_cast<int>(n_items < bwd_sm_count() ? n_items : bwd_sm_count());
  return launch_kernel(kern, dim3(grid), kBwdThreads, L::kSmemBytes, stream, dependent, a1, a2, b1, b2, p, gx,
                       static_cast<int>(n_items));
}

// The dK/dV pass: the persistent kernel for fixed-length calls at D <= 64 whose items average at
// most 32 partner blocks (query heads per item x 64-row query blocks, halved under the causal
// mask); the per-tile grid otherwise.
template <int D, bool BF16>
cudaError_t launch_dkdv_t(bool general, const BwdMaps& m, const BwdParams& p, cudaStream_t stream,
                          bool dependent) {
  if (general) return launch_main_t<D, BF16, true, true>(m.k128, m.v128, m.q64, m.do64, p, stream, dependent);
  if constexpr (D <= 64) {
    const int64_t blocks = static_cast<int64_t>(p.group / p.kv_splits) * ((p.S + kPartnerRows - 1) / kPartnerRows);
    if ((p.causal ? blocks / 2 : blocks) <= 32)
      return launch_dkdv_persistent_t<D, BF16>(m.k128, m.v128, m.q64, m.do64, p, stream, dependent);
  }
  return launch_main_t<D, BF16, true, false>(m.k128, m.v128, m.q64, m.do64, p, stream, dependent);
}

template <int D, bool BF16>
cudaError_t launch_reduce_t(const BwdParams& p, int64_t rows, cudaStream_t stream) {
  const int64_t threads = rows * (2 * D / 8);
  const int64_t blocks = (threads + 255) / 256;
  const int grid = static_cast<int>(blocks < 152 * 8 ? blocks : 152 * 8);
  fa_bwd_dkv_reduce_kernel<D, BF16><<<grid, 256, 0, stream>>>(p, rows);
  return cudaGetLastError();
}

}  // namespace

int bwd_kv_splits(int64_t BHkv, int64_t n_tiles, int group) {
  constexpr int64_t kWant = 2 * 152;
  if (group <= 1) return 1;
  for (int s = 1; s < group; ++s)
    if (group % s == 0 && BHkv * n_tiles * s >= kWant) return s;
  return group;
}

#define FA_BWD_DISPATCH(CALL)                                   \
  switch (D) {                                                  \
    case 16: return bf16 ? CALL(16, true) : CALL(16, false);    \
    case 32: return bf16 ? CALL(32, true) : CALL(32, false);    \
    case 64: return bf16 ? CALL(64, true) : CALL(64, false);    \
    case 128: return bf16 ? CALL(128, true) : CALL(128, false); \
    default: return cudaErrorInvalidValue;                      \
  }

cudaError_t launch_bwd_preprocess(int D, bool bf16, const BwdParams& p, int64_t rows, cudaStream_t stream) {
#define FA_PRE(DD, BB) launch_pre_t<DD, BB>(p, rows, stream)
  FA_BWD_DISPATCH(FA_PRE)
#undef FA_PRE
}

cudaError_t launch_bwd_dkdv(int D, bool bf16, bool general, const BwdMaps& m, const BwdParams& p,
                            cudaStream_t stream, bool dependent) {
#define FA_DKDV(DD, BB) launch_dkdv_t<DD, BB>(general, m, p, stream, dependent)
  FA_BWD_DISPATCH(FA_DKDV)
#undef FA_DKDV
}

cudaError_t launch_bwd_dkv_reduce(int D, bool bf16, const BwdParams& p, int64_t rows, cudaStream_t stream) {
#define FA_RED(DD, BB) launch_reduce_t<DD, BB>(p, rows, stream)
  FA_BWD_DISPATCH(FA_RED)
#undef FA_RED
}

cudaError_t launch_bwd_dq(int D, bool bf16, bool general, const BwdMaps& m, const BwdParams& p,
                          cudaStream_t stream, bool dependent) {
#define FA_DQ(DD, BB) launch_dq_t<DD, BB>(general, m, p, stream, dependent)
  FA_BWD_DISPATCH(FA_DQ)
#undef FA_DQ
}

#undef FA_BWD_DISPATCH

bool bwd_dq_computes_delta(int D, bool general) { return !general && D <= 64; }

}  // namespace fa
