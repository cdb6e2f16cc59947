// Attention of prompt chunks over a paged key/value cache: the query rows of
// a unit are the tensor core's rows.
//
// fa_paged_kernel.cuh puts keys on the rows, which wastes nothing when a K/V
// head has few query rows but sends P through shared memory.  Here a unit is
// kTiles tiles of 128 query rows of one K/V head (tokens x the group's heads,
// so a chunk of 64 tokens with 4 heads to a K/V head already fills two tiles);
// S = Q K^T and O += P V keep P in TMEM, and a softmax thread owns a row, as in
// the fixed-length forward kernels (same recurrence, same stale maximum).  The
// tiles share every K and V block.  D = 128: two tiles, 128-key blocks;
// D <= 64: four tiles, 64-key blocks (there the exponentials bound the kernel,
// and sixteen softmax warps hide more of each other's latency than eight).
//
// At D = 128 the tensor core bounds it: chunks of 2048 tokens over 16384 keys,
// 32 heads on 4, take 588 us with the join, 1.53 PFLOP/s, at the power cap (557
// before it bites).  At D = 64 the chain of products and exponentials does:
// ragged chunks of 16 heads take 85 us, the tensor pipes active a third of the
// time, DRAM a fifth.
//
// Units, blocks, runs and partials are fa_paged_kernel.cuh's: one persistent
// CTA per SM takes a run of blocks, equal to the others' in cost.  Within a unit
// each tile starts at the first block its own rows see and stops after the last.
//
// Per tile the MMA warp issues O += P(j) V(j), then S of the tile's next block,
// then one commit: "next S ready" also means "P(j) consumed, O updated", so the
// softmax waits once per block and may rescale O as soon as it sees that S.
#pragma once

#include "fa_paged_units.cuh"
#include "fa_softmax.cuh"

namespace fa {
using namespace ptx;

namespace {

template <int D>
struct PagedTileLayout {
  static constexpr int kTiles = D == 128 ? 2 : 4;
  static constexpr int kShift = D == 128 ? 7 : 6;
  static constexpr int kBlk = 1 << kShift;      // keys per block
  using GQ = TileGeom<D, 128>;
  using GK = TileGeom<D, kBlk>;
  static constexpr int kSoftWarps = 4 * kTiles;
  // Warps that issue MMAs, each for kTiles / kMmaWarps tiles.  Two tiles: one
  // warp, which issues a tile's P V and next S as a whole before the other's.
  // With a warp each the two tiles' products interleave whenever they meet, both
  // come late, and the tiles stay in step for hundreds of blocks (a block of two
  // tiles 2900 cycles, or up to 4000, instead of 2430).  Four tiles: two warps;
  // one cannot keep the tensor core fed.
  static constexpr int kMmaWarps = kTiles == 2 ? 1 : 2;
  static constexpr int kThreads = 32 * kSoftWarps + 128;  // and the producers of K and V, the MMA warps
  // Register split: every thread gets kLaunchRegs at launch, the last four
  // warps drop to kRegsLow and the softmax warps rise to kRegsHigh.
  static constexpr int kLaunchRegs = kTiles == 2 ? 168 : 96;
  static constexpr uint32_t kRegsHigh = kTiles == 2 ? 216 : 104;
  static constexpr uint32_t kRegsLow = kTiles == 2 ? 72 : 64;
  static_assert(32 * kSoftWarps * kRegsHigh + 128 * kRegsLow <= kThreads * kLaunchRegs, "register split");
  static constexpr int kSmallBytes = D == 128 ? 2048 : 5120;  // barriers, run, walks, row statistics
  static constexpr int kStatBytes = kTiles == 4 ? 3 * 128 * 8 : 32 * 8;
  // Two Q buffers where they fit beside the ring, so that the next unit's Q is
  // there when the last blocks of this one are done.
  static constexpr int kQBufs = D == 128 ? 1 : 2;
  static constexpr int kQBytes = kTiles * GQ::kTileBytes;
  static constexpr int kUnitsFit = (227 * 1024 - 1024 - kQBufs * kQBytes - kSmallBytes) / GK::kTileBytes;
  static constexpr int kUnits = kUnitsFit > 20 ? 20 : kUnitsFit;  // stages of both rings, one block each
  static_assert(kUnits >= 4, "rings");
  static constexpr int kUnitsK = (kUnits + 1) / 2, kUnitsV = kUnits / 2;
  static constexpr int kOffQ = kUnits * GK::kTileBytes;
  static constexpr int kOffSmall = kOffQ + kQBufs * kQBytes;
  // full[U], empty[U], qfull[2], qempty[2], sfull[T], pfull[T], ofinal[T], stat[T], freed[T], vtmp, drain[2]
  static constexpr int kNumBars = 2 * kUnits + 4 + 5 * kTiles + 3;
  static_assert(kNumBars * 8 + 16 + sizeof(RunStart) + kSoftWarps * (sizeof(SegWalk<kShift, true>) + 8) + kStatBytes <=
                    kSmallBytes, "barriers");
  static constexpr int kSmemUsed = kOffSmall + kSmallBytes + 1024;
  static constexpr int kSmemBytes = kSmemUsed > 116 * 1024 ? kSmemUsed : 116 * 1024;  // one CTA per SM
  static constexpr uint32_t kTileCols = 512 / kTiles;  // TMEM columns of a tile: S (P over it), then O
  static constexpr uint32_t kColO = kBlk;
  static_assert(kColO + D <= kTileCols, "TMEM layout");
};

// Tile t of the CTA in the current unit.  With four tiles (D <= 64) a unit of
// one or two row tiles would leave the others idle while a block's chain
// (products, exponentials, products) runs uncovered, so they take its blocks in
// turns, and their O are joined at the segment's end: 256 units of 8192 keys of
// one row tile 192 -> 125 us, of two 216 -> 171 (D = 64).  With two (D = 128) the
// chain is covered by the block's memory time: 203 us either way, so not there.
struct TileSpan {
  int tiles;       // row tiles of the unit
  int turns;       // tiles of the CTA that share each of them (a power of two)
  int row_tile, turn;  // this tile's; turn >= turns: it is idle
  int ta, n_tok;   // first token within the unit, tokens
  int pos0;        // cache position of its first token
  int beg, end;    // its blocks: beg, beg + turns, .. end - 1
};

template <int SHIFT, int TILES>
__device__ __forceinline__ TileSpan tile_span(const PagedParams& p, const SegWalk<SHIFT, true>& w, int t, int tile_tok,
                                              int n) {
  TileSpan s;
  s.tiles = (w.u.n_tok + tile_tok - 1) / tile_tok;
  s.turns = TILES < 4 || s.tiles > 2 ? 1 : 4 / s.tiles;
  s.turn = t / s.tiles;
  s.row_tile = t - s.turn * s.tiles;
  s.ta = s.row_tile * tile_tok;
  s.n_tok = min(tile_tok, w.u.n_tok - s.ta);
  s.pos0 = w.u.pos0 + s.ta;
  s.beg = s.end = 0;
  if (s.turn >= s.turns) return s;
  const int lo = max(0, s.pos0 - p.win_left), hi = min(w.u.kv_len, s.pos0 + s.n_tok + p.win_right);
  if (hi <= lo) return s;
  const int base = (w.u.lo >> SHIFT) + w.blk;  // the segment's first block
  const int beg = min(n, max(0, (lo >> SHIFT) - base));
  const int end = min(n, max(0, ((hi + (1 << SHIFT) - 1) >> SHIFT) - base));
  s.beg = beg + ((s.turn - beg) & (s.turns - 1));
  s.end = end - ((end - 1 - s.turn) & (s.turns - 1));
  if (s.end <= s.beg) s.beg = s.end = 0;
  return s;
}

}  // namespace

// tm_q: {D, H, T} map, box {row chunk, G, tile tokens}; tm_k, tm_v: {D, H_kv,
// page_size, pages} maps, box {row chunk, 1, min(page_size, block), 1}.
template <int D, bool BF16>
__global__ void __launch_bounds__(PagedTileLayout<D>::kThreads, 1)
    fa_paged_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using L = PagedTileLayout<D>;
  using GQ = typename L::GQ;
  using GK = typename L::GK;
  using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  using Walk = SegWalk<L::kShift, true>;
  constexpr int U = L::kUnits, T = L::kTiles, BN = L::kBlk;
  // The last four warps sit on one scheduler each; MMA issuers on the first
  // two (the other way round four full tiles at D = 64 take 309 us, not 301).
  constexpr int kMma0 = L::kSoftWarps, kProducer = L::kSoftWarps + 2, kProducerV = L::kSoftWarps + 3;
  constexpr int kMmaWarps = L::kMmaWarps, kTilesPerMma = T / kMmaWarps;
  constexpr float kSumLimit = 256.0f;  // largest block sum of P~ kept with a stale maximum

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + L::kOffSmall);  // [U] block landed
  uint64_t* bar_empty = bar_full + U;    // [U] every MMA warp is done with it
  uint64_t* bar_qfull = bar_empty + U;   // [2] segment's Q landed
  uint64_t* bar_qempty = bar_qfull + 2;  // [2] the segment's last score products are done
  uint64_t* bar_sfull = bar_qempty + 2;  // [T] S_t computed (and the P_t V before it done)
  uint64_t* bar_pfull = bar_sfull + T;   // [T] P_t stored, O_t rescaled
  uint64_t* bar_ofinal = bar_pfull + T;  // [T] the segment's last P_t V done
  uint64_t* bar_stat = bar_ofinal + T;   // [T] this tile's share of a split unit can be joined
  uint64_t* bar_freed = bar_stat + T;    // [T] this tile's share was joined
  uint64_t* bar_vtmp = bar_freed + T;    // a V block that still needs rows cleared has landed
  uint64_t* bar_drain = bar_vtmp + 1;    // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  RunStart* s_start = reinterpret_cast<RunStart*>(tmem_slot + 2);
  // Each softmax warp's walk, parked here while it works through a segment's
  // blocks: in registers it made the block loop spill.
  struct Parked {
    Walk w;
    unsigned phases;
  };
  Parked* s_walk = reinterpret_cast<Parked*>(s_start + 1);
  // Maximum and sum of the rows of tiles 1 .. T-1 where they share a unit.
  float2* s_stat = reinterpret_cast<float2*>(smem + L::kOffSmall + L::kSmallBytes - L::kStatBytes);
  long long* s_warp = reinterpret_cast<long long*>(s_stat);  // (before the first unit)

  const int warp = warp_index();
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < U; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], kMmaWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar_qfull[s], 1);
      mbar_init(&bar_qempty[s], kMmaWarps);
    }
    for (int t = 0; t < T; ++t) {
      mbar_init(&bar_sfull[t], 1);
      mbar_init(&bar_pfull[t], 4);
      mbar_init(&bar_ofinal[t], 1);
      mbar_init(&bar_stat[t], 4);
      mbar_init(&bar_freed[t], 4);
    }
    mbar_init(bar_vtmp, 1);
    mbar_init(&bar_drain[0], 1);
    mbar_init(&bar_drain[1], 1);
    *abort_flag = 0;
    s_start->left = 0;
    s_start->u.n_blk = 0;
    s_start->blk = 0;
    fence_mbar_init();
  }
  if (warp == kMma0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == kProducer && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // Up to here nothing of the caller's was touched.
  griddep_wait();
  if (threadIdx.x == 0) {
    if (p.go && blockIdx.x == 0) say_go(p);
    griddep_launch_dependents();
  }
  SeqLens own{0, 0, 0};
  {
    int per;
    const int x0 = paged_first_unit(p, L::kThreads, &per);
    if (x0 < p.batch * p.tiles) own = seq_lens(p, p.tiles == 1 ? x0 : x0 / p.tiles);
  }
  if (threadIdx.x == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  paged_find_run<L::kShift, true, L::kThreads>(p, own, s_warp, s_start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tile_tok = 128 / p.G;  // tokens of a 128-row tile

  if (warp >= L::kSoftWarps) {
    regs_decrease<L::kRegsLow>();
    Walk w;
    w.start(p, *s_start);
    if (warp == kProducer || warp == kProducerV) {
      // ------------------------------------------------------------ producers
      // One warp copies Q and the K blocks, one the V blocks, each through its
      // own ring.  The whole warp runs this; lane i copies page box i of a block.
      const int kv = warp == kProducer ? 0 : 1;
      const CUtensorMap* map = kv == 0 ? &tm_k : &tm_v;
      const int stages = kv == 0 ? L::kUnitsK : L::kUnitsV;
      uint64_t* full = bar_full + (kv == 0 ? 0 : L::kUnitsK);
      uint64_t* empty = bar_empty + (kv == 0 ? 0 : L::kUnitsK);
      uint8_t* ring = smem + (kv == 0 ? 0 : L::kUnitsK * GK::kTileBytes);
      const int frag = min(BN, 1 << p.page_shift);
      const int n_frag = BN / frag;
      int c = 0, seg = 0, n_cut = 0;  // blocks started, segments started, V blocks that had rows cleared
      int st = 0;         // ring stage of the next block
      unsigned pass = 0;  // passes over the ring
      bool ok = true;
      auto box_page = [&](int blk) -> int {  // page (or out of range) of this lane's box of the unit's block
        const int key = ((w.u.lo >> L::kShift) + blk) * BN + lane * frag;
        if (lane >= n_frag || key >= w.u.hi || key + frag <= w.u.lo) return p.num_pages;
        const int page = p.block_table[static_cast<int64_t>(w.b) * p.table_stride + (key >> p.page_shift)];
        if (page >= 0 && page < p.num_pages) return page;
        record_error(p.err, kErrBadPage);
        return p.num_pages;
      };
      for (int n; ok && (n = w.seg_len()) > 0; w.next(p, n), ++seg) {
        int page = box_page(w.blk);
        if (kv == 0) {
          const int qb = seg % L::kQBufs, qu = seg / L::kQBufs;
          if (qu > 0) ok = warp_wait(&bar_qempty[qb], (qu - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutLoad);
          if (!ok) break;
          if (lane == 0) {
            const int tiles = (w.u.n_tok + tile_tok - 1) / tile_tok;
            mbar_arrive_expect_tx(&bar_qfull[qb], tiles * GQ::kChunks * GQ::kRowBytes * p.G * tile_tok);
            for (int t = 0; t < tiles; ++t)
#pragma unroll
              for (int ch = 0; ch < GQ::kChunks; ++ch)
                tma_load_3d(smem + L::kOffQ + qb * L::kQBytes + t * GQ::kTileBytes + ch * GQ::kChunkBytes, &tm_q,
                            &bar_qfull[qb], ch * (GQ::kRowBytes / 2), w.kvh * p.G, w.u.tok0 + t * tile_tok);
          }
          __syncwarp();
        }
        for (int j = 0; ok && j < n; ++j) {
          const int page_next = j + 1 < n ? box_page(w.blk + j + 1) : 0;
          const int key0 = ((w.u.lo >> L::kShift) + w.blk + j) * BN;
          const int row = (key0 + lane * frag) & ((1 << p.page_shift) - 1);
          const bool clear = kv == 1 && (key0 < w.u.lo || key0 + BN > w.u.hi);
          if (pass > 0) {
            ok = warp_wait(&empty[st], (pass - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutLoad);
            if (!ok) break;
          }
          uint8_t* tile = ring + st * GK::kTileBytes;
          uint64_t* bar = clear ? bar_vtmp : &full[st];
          if (lane == 0) mbar_arrive_expect_tx(bar, GK::kTileBytes);
          __syncwarp();
          if (lane < n_frag) {
#pragma unroll
            for (int ch = 0; ch < GK::kChunks; ++ch)
              tma_load_4d(tile + ch * GK::kChunkBytes + lane * frag * GK::kRowBytes, map, bar,
                          ch * (GK::kRowBytes / 2), w.kvh, row, page);
          }
          ++c;
          if (clear) {
            // Clear the V rows no row of the unit sees (0 * NaN is not 0).
            drain_wait(bar_vtmp, n_cut & 1, p.err);
            ++n_cut;
            const int k0 = max(0, w.u.lo - key0), k1 = min(BN, w.u.hi - key0);  // visible rows [k0, k1)
            constexpr int kVecs = GK::kRowBytes / 16;
            for (int i = lane; i < BN * kVecs * GK::kChunks; i += 32) {
              const int r = (i / kVecs) % BN;
              if (r < k0 || r >= k1) *reinterpret_cast<uint4*>(tile + i * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
          }
          page = page_next;
          if (++st == stages) {
            st = 0;
            ++pass;
          }
        }
      }
      // Teardown: every copy this warp started lands before the CTA exits.
      for (int x = max(0, c - stages); x < c; ++x) drain_wait(&full[x % stages], (x / stages) & 1, p.err);
      if (kv == 0)
        for (int x = (seg > L::kQBufs ? seg - L::kQBufs : 0); x < seg; ++x)
          drain_wait(&bar_qfull[x % L::kQBufs], (x / L::kQBufs) & 1, p.err);
      __syncwarp();
    } else if (warp < kMma0 + kMmaWarps) {
      // ------------------------------------------------------------ MMA issuers
      const int m = warp - kMma0;  // tiles m * kTilesPerMma ..
      constexpr uint32_t idesc_qk = make_idesc_f16(BF16, 128, BN, false, false);
      constexpr uint32_t idesc_pv = make_idesc_f16(BF16, 128, D, false, true);
      const AccFlags acc = runtime_flags(p.batch);
      const uint32_t s_ring = smem_u32(smem), s_q = smem_u32(smem + L::kOffQ);
      int c = 0;                     // blocks before the segment
      int done[kTilesPerMma];        // blocks of each tile whose P V was issued
#pragma unroll
      for (int h = 0; h < kTilesPerMma; ++h) done[h] = 0;
      bool ok = true;
      int seg = 0;
      for (int n; ok && (n = w.seg_len()) > 0; w.next(p, n), ++seg) {
        int beg[kTilesPerMma], end[kTilesPerMma], turn[kTilesPerMma], row_tile[kTilesPerMma], turns;
#pragma unroll
        for (int h = 0; h < kTilesPerMma; ++h) {
          const TileSpan s = tile_span<L::kShift, T>(p, w, m * kTilesPerMma + h, tile_tok, n);
          beg[h] = s.beg;
          end[h] = s.end;
          turn[h] = s.turn;
          row_tile[h] = s.row_tile;
          turns = s.turns;
        }
        const int qb = seg % L::kQBufs;
        ok = warp_wait(&bar_qfull[qb], (seg / L::kQBufs) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
        for (int j = -turns; ok && j < n; ++j) {
          const int jk = j + turns;
          const int kc = c + jk, vc = c + j;
          const int ks = kc % L::kUnitsK, vs = vc % L::kUnitsV;  // ring stages of K(jk), V(j)
          if (j >= 0)
            ok = warp_wait(&bar_full[L::kUnitsK + vs], (vc / L::kUnitsV) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
          if (ok && jk < n)
            ok = warp_wait(&bar_full[ks], (kc / L::kUnitsK) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
          if (!ok) break;
#pragma unroll
          for (int h = 0; h < kTilesPerMma; ++h) {
            const int t = m * kTilesPerMma + h;
            const uint32_t t_s = tmem + t * L::kTileCols;
            if (turn[h] != (jk & (turns - 1))) continue;
            if (j >= beg[h] && j < end[h]) {
              if (!ok) break;
              ok = warp_wait(&bar_pfull[t], done[h] & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
              if (!ok) break;
              ++done[h];
              tc_fence_after();
              const uint64_t v_desc =
                  make_sdesc(s_ring + (L::kUnitsK + vs) * GK::kTileBytes, GK::kChunkBytes, 8 * GK::kRowBytes, GK::kSwz);
#pragma unroll
              for (int kk = 0; kk < BN / 16; ++kk)
                mma_ts_warp(t_s + L::kColO, t_s + kk * 8, desc_plus(v_desc, mnmajor_step_bytes<D>(kk)), idesc_pv,
                            (j > beg[h] || kk > 0) ? acc.on : acc.off);
              if (j == end[h] - 1) mma_commit_warp(&bar_ofinal[t]);
            }
            if (jk >= beg[h] && jk < end[h]) {
              tc_fence_after();
              const uint64_t q_desc = make_sdesc(
                  s_q + qb * L::kQBytes + row_tile[h] * GQ::kTileBytes, 16, 8 * GQ::kRowBytes, GQ::kSwz);
              const uint64_t k_desc = make_sdesc(s_ring + ks * GK::kTileBytes, 16, 8 * GK::kRowBytes, GK::kSwz);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ss_warp(t_s, desc_plus(q_desc, kmajor_step_bytes<D, 128>(kk)),
                            desc_plus(k_desc, kmajor_step_bytes<D, BN>(kk)), idesc_qk, kk > 0 ? acc.on : acc.off);
              mma_commit_warp(&bar_sfull[t]);
            }
          }
          if (!ok) break;
          if (j >= 0) mma_commit_warp(&bar_empty[L::kUnitsK + vs]);
          if (jk < n) mma_commit_warp(&bar_empty[ks]);
          if (jk == n - 1) mma_commit_warp(&bar_qempty[qb]);
        }
        c += n;
      }
      mma_commit_warp(&bar_drain[m]);
      drain_wait(&bar_drain[m], 0, p.err);
    }
  } else {
    regs_increase<L::kRegsHigh>();
    // -------------------------------------------------------------- softmax
    Walk w;
    w.start(p, *s_start);
    const int t = warp >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the tile == TMEM lane
    const int rt = r / p.G, rh = r - rt * p.G;  // its token within the tile, head within the group
    const uint32_t t_s = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + t * L::kTileCols;
    const uint32_t t_o = t_s + L::kColO;
    const float sl2 = p.scale_log2;
    // Blocks that a mask cuts.  D <= 64: the scores a row does not see become
    // -inf (+inf under a negative scale) in place, and one copy of the code
    // serves all blocks; a copy of its own for the few cut ones cost up to 5000
    // cycles of instruction fetch per unit (ragged chunks 129 -> 121 us).  At
    // D = 128 the selects between load and maximum cost more than that (chunks
    // of 2048: 668 us with a copy of its own, 723 in place).
    constexpr bool kMaskInPlace = D <= 64;
    constexpr bool kShare = T == 4;  // tiles may share a unit's row tile
    // In place, a scale of 0 is applied ahead of the mask (0 times a hidden key's
    // infinity would not be -inf); a NaN stays one.
    const bool zero_scale = kMaskInPlace && sl2 == 0.f;
    const float ce = zero_scale ? 1.f : sl2;
    const float2 c2 = make_float2(ce, ce);
    const bool neg_scale = sl2 < 0.f;
    const uint32_t hidden = __float_as_uint(neg_scale ? INFINITY : -INFINITY);
    int cnt = 0, fin = 0;  // blocks of this tile so far; segments in which it had blocks
    bool alive = true;
    if (lane == 0) s_walk[warp].phases = 0;
    for (int n; alive && (n = w.seg_len()) > 0; w.next(p, n)) {
      const TileSpan sp = tile_span<L::kShift, T>(p, w, t, tile_tok, n);
      const bool row_ok = rt < sp.n_tok && rt < tile_tok;
      // Relative to the segment's first key: this row's visible keys [lo0, lim0],
      // and the blocks [j_lo, j_hi) that every row of the tile sees whole.
      const int key_base = ((w.u.lo >> L::kShift) + w.blk) * BN;
      const int pos = sp.pos0 + rt;
      const int lim0 = min(w.u.kv_len - 1, pos + p.win_right) - key_base, lo0 = pos - p.win_left - key_base;
      const int j_lo = (sp.pos0 + sp.n_tok - 1 - p.win_left - key_base + BN - 1) >> L::kShift;
      const int j_hi = (min(w.u.kv_len, sp.pos0 + 1 + p.win_right) - key_base) >> L::kShift;
      const int beg = sp.beg, end = sp.end, step = kShare ? sp.turns : 1;
      if (lane == 0) s_walk[warp].w = w;
      __syncwarp();
      // (the span is worked out again after the blocks: its other members would
      // take registers from the block loop)
      float m = -INFINITY, l = 0.f;
      for (int j = beg; j < end; j += step, ++cnt) {
        if (!warp_wait(&bar_sfull[t], cnt & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax)) {
          alive = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[BN];
        if constexpr (BN == 128) tmem_ld128(t_s, sr);
        else tmem_ld64(t_s, sr);
        const int lim = lim0 - j * BN, lo = lo0 - j * BN;  // columns lo <= c <= lim are visible to this row
        const bool cut = j < j_lo || j >= j_hi;  // a mask cuts the block
        if constexpr (kMaskInPlace) {
          if (zero_scale) {
#pragma unroll
            for (int c = 0; c < BN; ++c) sr[c] = __float_as_uint(0.f * __uint_as_float(sr[c]));
          }
          if (cut) {
#pragma unroll
            for (int c = 0; c < BN; ++c) sr[c] = c < lo || c > lim ? hidden : sr[c];
          }
        }
        const bool masked = !kMaskInPlace && cut;
        auto block_max = [&]() {
          return block_max_scaled<BN, !kMaskInPlace>(sr, masked, lo, kMaskInPlace ? BN : lim, ce, neg_scale);
        };
        if (j == beg) m = block_max();
        float alpha = 1.f;
        auto exps = [&]() {
          const float m_use = m == -INFINITY ? 0.f : m;  // rows with no visible key so far
          const float2 negm = make_float2(-m_use, -m_use);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                           make_float2(0.f, 0.f)};
          if (masked) {
#pragma unroll
            for (int k0 = 0; k0 < BN; k0 += 16) {
              uint32_t pk[8];
              exp16<BF16, !kMaskInPlace, true>(sr, k0, c2, negm, lo, lim, acc, pk);
              tmem_st8(t_s + k0 / 2, pk);
            }
          } else {
#pragma unroll
            for (int k0 = 0; k0 < BN; k0 += 16) {
              uint32_t pk[8];
              exp16<BF16, false>(sr, k0, c2, negm, 0, BN, acc, pk);
              tmem_st8(t_s + k0 / 2, pk);
            }
          }
          const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
          return a.x + a.y;
        };
        float blk = exps();
        // A block whose sum breaks the bound (or a row's first visible key)
        // moves the maximum, rescales O and is done again.  Lanes past the
        // tile's rows hold anything and never ask for it.
        const bool need = row_ok && (!(blk <= kSumLimit) || m == -INFINITY);
        if (__any_sync(0xffffffffu, need)) {
          const float m_blk = block_max();
          const bool upd = need && m_blk > m;
          if (upd) {
            alpha = ex2(m - m_blk);
            m = m_blk;
          }
          if (__any_sync(0xffffffffu, upd)) {
            tmem_st_wait();  // the first pass's stores land before they are overwritten
            blk = exps();
            if (j > beg) {
#pragma unroll
              for (int c = 0; c < D; c += 16) {
                uint32_t o16[16];
                tmem_ld16(t_o + c, o16);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  const float2 v = __fmul2_rn(make_float2(__uint_as_float(o16[i]), __uint_as_float(o16[i + 1])),
                                              make_float2(alpha, alpha));
                  o16[i] = __float_as_uint(v.x);
                  o16[i + 1] = __float_as_uint(v.y);
                }
                tmem_st16(t_o + c, o16);
              }
            }
          }
        }
        l = l * alpha + blk;
        tmem_st_wait();
        warp_arrive(&bar_pfull[t]);
      }
      if (!alive) break;
      // ------------------------------------------------------------ segment's end
      w = s_walk[warp].w;
      __syncwarp();  // (a tile without blocks meets no other before lane 0 parks the next segment's)
      n = w.seg_len();
      const bool have = end > beg;
      if (have) {
        if (!warp_wait(&bar_ofinal[t], fin & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax)) {
          alive = false;
          break;
        }
        ++fin;
        tc_fence_after();
      }
      const TileSpan es = tile_span<L::kShift, T>(p, w, t, tile_tok, n);
      const int tiles = es.tiles, turn = es.turn, row_tile = es.row_tile, turns = kShare ? es.turns : 1;
      // (a sum of 0: no key was seen; NaN scores make it NaN, and the row with it)
      const bool mine = have && l != 0.f;
      // A unit's row tile whose blocks several tiles took in turns: the first
      // of them joins the others' O and statistics to its own.
      float w_own = 1.f, w_other[T - 1];
#pragma unroll
      for (int k = 1; k < T; ++k) w_other[k - 1] = 0.f;
      if (turns > 1) {
        // Tile t >= tiles gives its share on bar_stat[t] and goes on when its row
        // tile's joiner has released it on bar_freed[t].  A pair of its own each, so
        // that no tile skips a phase it later waits past: with one bar_freed a row
        // tile, a tile whose row tile changed from unit to unit took the phase
        // before last for the last (the same parity) and ran ahead.  The joiner of
        // bar_stat[3] is tile 0 or 1; its waits in this order (k = 1, 2, 3) keep the
        // one from passing the other's phase: tile 1 gives bar_stat[1] only after
        // it has seen bar_stat[3].
        const unsigned phases = s_walk[warp].phases;  // bit t: of bar_stat[t] and bar_freed[t]
        if (turn > 0) {
          s_stat[(t - 1) * 128 + r] = make_float2(m, mine ? l : 0.f);
          warp_arrive(&bar_stat[t]);
          alive = warp_wait(&bar_freed[t], (phases >> t) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax);
        } else {
          float2 st[T - 1];
          float top = mine ? m : -INFINITY;
#pragma unroll
          for (int k = 1; k < T; ++k) {
            st[k - 1] = make_float2(-INFINITY, 0.f);
            if (k < turns && alive) {
              const int tk = k * tiles + row_tile;
              alive = warp_wait(&bar_stat[tk], (phases >> tk) & 1, abort_flag, p.err, p.wait_ns,
                                kErrTimeoutSoftmax);
              st[k - 1] = s_stat[(tk - 1) * 128 + r];
              if (st[k - 1].y != 0.f) top = fmaxf(top, st[k - 1].x);
            }
          }
          w_own = mine ? ex2(m - top) : 0.f;
          l = mine ? l * w_own : 0.f;
#pragma unroll
          for (int k = 1; k < T; ++k) {
            if (st[k - 1].y != 0.f) w_other[k - 1] = ex2(st[k - 1].x - top);
            l += w_other[k - 1] * st[k - 1].y;
          }
          m = top;
        }
        if (!alive) break;
        tc_fence_after();
        __syncwarp();
        if (lane == 0) s_walk[warp].phases = phases ^ ((1u << T) - (1u << tiles));
        __syncwarp();
      }
      const bool whole = n == w.u.n_blk;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (w.blk == 0 ? 1 : 0);
      const bool seen = turns > 1 ? l != 0.f : mine;
      const float inv_l = seen ? 1.f / l : 0.f;
      const int ta = row_tile * tile_tok, tok = w.u.tok0 + ta + rt, head = w.kvh * p.G + rh;
      // Partials lie [slot][D / 4][part_rows][4]: neighbouring lanes (rows) write
      // neighbouring 16 bytes.
      const int prow = (ta + rt) * p.G + rh;
      float* part = p.o_part + static_cast<int64_t>(slot) * p.part_rows * D + prow * 4;
      elem_t* orow = static_cast<elem_t*>(p.o) + (static_cast<int64_t>(tok) * p.H + head) * D;
      if (turn == 0) {  // (warp-uniform)
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          uint32_t o16[16];
          if (have) tmem_ld16(t_o + c, o16);
#pragma unroll
          for (int i = 0; i < 16; ++i) o16[i] = mine ? o16[i] : 0u;
          if (turns > 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o16[i] = __float_as_uint(w_own * __uint_as_float(o16[i]));
#pragma unroll
            for (int k = 1; k < T; ++k) {
              const bool add = w_other[k - 1] != 0.f;
              if (!__any_sync(0xffffffffu, add)) continue;  // (a tile without blocks holds an earlier unit's O)
              uint32_t x16[16];
              tmem_ld16(t_o + k * tiles * L::kTileCols + c, x16);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (add)
                  o16[i] = __float_as_uint(__uint_as_float(o16[i]) + w_other[k - 1] * __uint_as_float(x16[i]));
            }
          }
          if (row_ok) {
            if (whole) store_row16<BF16>(orow + c, o16, inv_l);
            else
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(part + static_cast<int64_t>((c + i) / 4) * p.part_rows * 4) =
                    make_float4(__uint_as_float(o16[i]) * inv_l, __uint_as_float(o16[i + 1]) * inv_l,
                                __uint_as_float(o16[i + 2]) * inv_l, __uint_as_float(o16[i + 3]) * inv_l);
          }
        }
        if (row_ok) {
          const float l2 = seen ? m + log2f(l) : -INFINITY;
          if (whole) p.lse[static_cast<int64_t>(head) * p.total + tok] = l2 * 0.69314718055994530942f;
          else p.lse_part[static_cast<int64_t>(slot) * p.part_rows + prow] = l2;
        }
      }
      if (turns > 1 && turn == 0)
        for (int k = 1; k < turns; ++k) warp_arrive(&bar_freed[k * tiles + row_tile]);
      if (!whole && w.blk == 0 && threadIdx.x == 0) {
        const long long last = s_start->at + s_start->left - w.left + static_cast<long long>(w.u.n_blk - 1) * w.cost;
        p.desc[blockIdx.x] = make_int4(w.u.tok0, w.u.n_tok, w.kvh, static_cast<int>(last / s_start->share));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {

template <int D, bool BF16>
cudaError_t launch_paged_tile_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const PagedParams& p, int grid, cudaStream_t stream) {
  using L = PagedTileLayout<D>;
  auto kern = fa_paged_tile_kernel<D, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
  if (e != cudaSuccess) return e;
  // The register split assumes the launch gives exactly kLaunchRegs per
  // thread; with fewer, the softmax warps' increase could never be met.
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, kern);
  if (e != cudaSuccess) return e;
  if (attr.numRegs != L::kLaunchRegs) return cudaErrorInvalidConfiguration;
  return launch_dependent(kern, dim3(grid), L::kThreads, L::kSmemBytes, stream, tq, tk, tv, p);
}

}  // namespace

}  // namespace fa
