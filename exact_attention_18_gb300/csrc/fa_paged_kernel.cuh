// Attention of new tokens over a paged key/value cache: few query rows per K/V
// head (decoding, drafted tokens).
//
//   O_i = sum_j softmax_j(scale q_i . k_j) v_j,   L_i = ln sum_j exp(scale q_i . k_j)
//
// over the keys j of the sequence's cache that row i sees.
//
// Keys are the matrix rows.  With few query rows a product that puts queries
// on the tensor core's 128 rows would leave most of them empty, so both
// products are taken transposed: S^T = K Q^T (128 keys x N rows) and
// O^T += V^T P^T (D x N), N = 16, 32 or 64 query rows of one K/V head (tokens x
// the group's heads).  K and V come from shared memory exactly as TMA wrote
// them: K K-major, V MN-major.  A TMEM lane is a key, so a softmax thread
// holds one key's scores for all N rows: running sums stay per thread until
// the unit ends, and the running maximum is one value per row that all lanes
// share.  It is taken exactly on a unit's first block and kept, stale, while
// no score exceeds it by more than 2^8 (exact in real arithmetic, as in the
// other forward kernels); a block that breaks the bound, or one that a mask
// cuts, takes the block maximum across lanes.
//
// What bounds it: with few rows, reading the cache.  At D = 128 a 128-key
// block is 64 KB, 2800 cycles of an SM's share of the memory's rate; decoding 32
// sequences of up to 8192 keys keeps the tensor pipe active 4.5 % of the time
// and takes 58 - 59 us with the join, 83 - 85 % of the copy rate (4 contexts of up
// to 131072 keys: 150 - 157 us, 96 - 100 %).  32 sequences of up to 8192 keys in
// pages of 16 take 34 us at D = 64 (floor 25) and 24 at D = 16 (6): there a
// block's chain shows.  So the kernel is organised around keeping copies in flight: one or two persistent CTAs per
// SM, their shared memory given to a ring of K and V tiles, and work dealt in
// 128-key blocks: the blocks of all units, in order, are cut into equal runs,
// one per CTA, whatever the sequences' lengths (each CTA finds its run from
// the lengths on the device).  A unit cut between CTAs leaves fp32 partials
// (O / l and the base-2 logsumexp), which a second kernel, launched as a
// programmatic dependent, joins in CTA order: no atomics, the result depends
// only on the lengths.
//
// Warp roles: 4 to 16 softmax warps, two TMA producers (K, V), one MMA issuer.
// Order of the tensor core's work: S(0), then S(j+1), O(j) for each block j, so
// scores of the next block are computed during the softmax.
//
// Pages.  A 128-key tile arrives as 128 / min(page, 128) boxes of whole or
// part pages; boxes that hold no visible key are not read (an out-of-range
// page coordinate, which the copy engine fills with zeros without reading).
// Keys the unit cannot see inside a box (past the sequence's end, before the
// window) may hold anything: their scores are never used, and their V rows
// are set to zero in shared memory, since 0 * NaN in the second product would
// not be 0.
#pragma once

#include "fa_paged_units.cuh"
#include "fa_softmax.cuh"

namespace fa {
using namespace ptx;

namespace {

constexpr int kPShift = 7;               // 128 keys per block
constexpr int kPBlk = 1 << kPShift;
constexpr float kPagedTau = 8.0f;        // log2 of the largest P~ kept with a stale maximum

template <int D, int N>
struct PagedLayout {
  using GK = TileGeom<D, kPBlk>;   // K and V tiles
  using GQ = TileGeom<D, N>;       // Q tile, N rows
  using GP = TileGeom<N, kPBlk>;   // P^T tile: 128 keys x N rows
  // Softmax warpgroups, each over kCols rows.  More of them hide more of each
  // other's latency: 16 sequences of 8192 keys at D = 64, N = 64 with 32 / 16
  // rows a thread 38.7 / 36.4 us.
  static constexpr int kCols = 16;
  static constexpr int kWgs = N / kCols;
  static constexpr int kThreads = 128 * kWgs + 96;  // and the producers of K and V, the MMA issuer
  static constexpr int kQBytes = (GQ::kTileBytes + 1023) / 1024 * 1024;
  static constexpr int kSmallBytes = 5 * 1024;      // barriers and per-row arrays
  // CTAs per SM (paged_ctas).  A block's chain of waits, loads and exponentials
  // takes about 1100 cycles however narrow the heads; at D = 128 that hides
  // behind the block's 2800 cycles of memory, below it a second CTA fills it.
  static constexpr int kCtas = paged_ctas(D, N);
  static constexpr int kBudget = (kCtas == 2 ? 113 : 227) * 1024 - 1024;
  static constexpr int kUnitsFit =
      (kBudget - 2 * GP::kTileBytes - 2 * kQBytes - kSmallBytes) / GK::kTileBytes;
  // Ring stages, one K or V tile each.  An even number: K tiles have the even
  // stages, V tiles the odd ones, and each producer sees every phase of its
  // stages' barriers.  (On a stage that both used, a producer could take a
  // phase for the one before the last: they have the same parity.)
  static constexpr int kUnits = (kUnitsFit > 16 ? 16 : kUnitsFit) & ~1;
  static_assert(kUnits >= 4, "ring");
  static constexpr int kOffP = kUnits * GK::kTileBytes;
  static constexpr int kOffQ = kOffP + 2 * GP::kTileBytes;
  static constexpr int kOffSmall = kOffQ + 2 * kQBytes;
  // full[U], empty[U], qfull[2], qempty[2], sfull[2], pfull[2], pv[2], vtmp, drain
  static constexpr int kNumBars = 2 * kUnits + 10 + 2;
  static_assert(kNumBars * 8 + 24 + sizeof(RunStart) + 8 * N * 4 + 2 * N <= kSmallBytes, "small arrays");
  // The request is padded so that no more CTAs than meant share an SM, nor one
  // of these with a kernel that takes the whole tensor memory (those ask for
  // 116 KB at least).
  static constexpr int kSmemUsed = kOffSmall + kSmallBytes + 1024;
  static constexpr int kSmemLeast = (kCtas == 2 ? 112 : 116) * 1024;
  static constexpr int kSmemBytes = kSmemUsed > kSmemLeast ? kSmemUsed : kSmemLeast;
  static constexpr uint32_t kTmemCols = 4 * N;  // S twice, O, and up to a power of two
  // V^T is D rows; the MMA's 128 rows past D repeat tile rows 8 further on
  // (in bounds: the ring is followed by the P tiles) into TMEM lanes nobody reads.
  static constexpr uint32_t kVLbo = D == 128 ? GK::kChunkBytes : 8 * GK::kRowBytes;
};

// Sum or maximum over the warp's 32 lanes of each of 16 values a lane holds:
// lane l receives that of column l % 16.  Halving exchange: each step keeps the
// half of the columns the lane's bit selects.
template <bool MAX>
__device__ __forceinline__ float warp_reduce_cols16(const float* x) {
  const int lane = threadIdx.x & 31;
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = x[i];
#pragma unroll
  for (int h = 8; h >= 1; h /= 2) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float keep = up ? v[i + h] : v[i], give = up ? v[i] : v[i + h];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, h));
    }
  }
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

// Byte offset of 16-byte chunk c of row k in a swizzled tile with rows of ROW_BYTES.
template <int ROW_BYTES>
__device__ __forceinline__ uint32_t swizzled(int k, int c) {
  constexpr int kShift = ROW_BYTES == 128 ? 0 : (ROW_BYTES == 64 ? 1 : 2);
  constexpr int kMask = ROW_BYTES / 16 - 1;
  return static_cast<uint32_t>(k * ROW_BYTES + ((c ^ ((k >> kShift) & kMask)) << 4));
}

}  // namespace

// tm_q: {D, H, T} map, box {row chunk, G, tok_tile}; tm_k, tm_v: {D, H_kv,
// page_size, pages} maps, box {row chunk, 1, min(page_size, 128), 1}.
template <int D, int N, bool BF16>
__global__ void __launch_bounds__(PagedLayout<D, N>::kThreads, PagedLayout<D, N>::kCtas)
    fa_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using L = PagedLayout<D, N>;
  using GK = typename L::GK;
  using GQ = typename L::GQ;
  using GP = typename L::GP;
  using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int U = L::kUnits;
  constexpr int NC = L::kCols;
  constexpr int kSoftWarps = 4 * L::kWgs;
  constexpr int kProducer = kSoftWarps, kMma = kSoftWarps + 2;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + L::kOffSmall);  // [U] tile landed
  uint64_t* bar_empty = bar_full + U;      // [U] tile's MMAs done
  uint64_t* bar_qfull = bar_empty + U;     // [2] segment's Q landed
  uint64_t* bar_qempty = bar_qfull + 2;    // [2] segment's last score product done
  uint64_t* bar_sfull = bar_qempty + 2;    // [2] S(i) computed (and O(i-2) done)
  uint64_t* bar_pfull = bar_sfull + 2;     // [2] P(i) stored, O rescaled
  uint64_t* bar_pv = bar_pfull + 2;        // [2] O(i) done
  uint64_t* bar_vtmp = bar_pv + 2;         // a V tile that still needs rows cleared has landed
  uint64_t* bar_drain = bar_vtmp + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  RunStart* s_start = reinterpret_cast<RunStart*>(tmem_slot + 2);
  float* s_m = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bar_full) + L::kNumBars * 8 + 8 + sizeof(RunStart));
  s_m = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(s_m) + 15) & ~static_cast<uintptr_t>(15));
  float* s_negm = s_m + N;          // [N] -(maximum), 0 while no key was seen
  float* s_alpha = s_negm + N;      // [N] factor of the last change of maximum; at a segment's end 1 / l
  float* s_red = s_alpha + N;       // [N][4] per-warp partial of each row
  int* s_off = reinterpret_cast<int*>(s_red + 4 * N);     // [N] output row of row n after its unit's first
  short* s_tok = reinterpret_cast<short*>(s_off + N);     // [N] token of row n

  // Behind the tile kernel of the same call this grid's CTAs start as that
  // kernel's end, and work beside the last of them once they have its word that
  // the grids before the call are done (the two share no output).  Waiting for
  // the tile kernel itself, a chunk of 512 tokens beside 63 single ones takes 135
  // us for 125 at D = 128, 103 for 94 at D = 64.  Where no sequence is short
  // enough for this kernel, it leaves before any set-up.
  if (p.after_tile && !__syncthreads_or(threadIdx.x == 0 && heard_go(p))) griddep_wait();
  SeqLens own{0, 0, 0};
  const bool all_known = p.after_tile && p.batch <= L::kThreads;  // a thread each
  if (all_known) {
    if (static_cast<int>(threadIdx.x) < p.batch) own = seq_lens(p, threadIdx.x);
    const int n = own.e - own.a;
    if (!__syncthreads_or(n > 0 && n <= p.tok_hi)) {
      if (threadIdx.x == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
      griddep_launch_dependents();
      griddep_wait();
      return;
    }
  }

  const int warp = warp_index();
  const int lane = threadIdx.x & 31;
  if (warp == 0) {
    // Barriers lie in a row; only pfull counts more than one arrival.
    for (int i = lane; i < L::kNumBars; i += 32)
      mbar_init(bar_full + i, bar_full + i == bar_pfull || bar_full + i == bar_pfull + 1 ? kSoftWarps : 1);
    fence_mbar_init();
    if (lane == 0) {
      *abort_flag = 0;
      s_start->left = 0;
      s_start->u.n_blk = 0;
      s_start->blk = 0;
    }
  }
  if (warp == kMma) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kProducer && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // (Behind other kernels nothing of the caller's was touched up to here.)
  if (!p.after_tile) griddep_wait();
  griddep_launch_dependents();
  if (!all_known) {
    int per;
    const int x0 = paged_first_unit(p, L::kThreads, &per);
    if (x0 < p.batch * p.tiles) own = seq_lens(p, p.tiles == 1 ? x0 : x0 / p.tiles);
  }
  if (threadIdx.x == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  for (int n = threadIdx.x; n < N; n += L::kThreads) {
    s_tok[n] = static_cast<short>(n / p.G);
    s_off[n] = (n / p.G) * p.H + n % p.G;
  }
  // (the per-row arrays are free until the first segment)
  paged_find_run<kPShift, false, L::kThreads>(p, own, reinterpret_cast<long long*>(s_red), s_start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  SegWalk<kPShift, false> w;
  w.start(p, *s_start);

  if (warp == kProducer || warp == kProducer + 1) {
    // -------------------------------------------------------------- producers
    // One warp copies Q and the K tiles, one the V tiles (ring stages alternate).
    // The whole warp runs this; lane i copies page box i of each tile.  With one
    // warp for both, its 450-750 cycles per tile bounded the kernel at D <= 64.
    const int kv = warp - kProducer;  // 0: K, 1: V
    if (p.after_tile) fence_proxy_async_global();
    const CUtensorMap* map = kv == 0 ? &tm_k : &tm_v;
    const int frag = min(kPBlk, 1 << p.page_shift);
    const int n_frag = kPBlk / frag;
    int c = kv;   // ring stage of the next tile, counted through (K even, V odd)
    int seg = 0;  // segments started (Q tiles)
    int n_cut = 0;  // V tiles that had rows cleared
    bool ok = true;
    auto box_page = [&](int blk) -> int {  // page (or out of range) of this lane's box of the unit's block
      const int key = (w.u.lo / kPBlk + blk) * kPBlk + lane * frag;
      if (lane >= n_frag || key >= w.u.hi || key + frag <= w.u.lo) return p.num_pages;
      const int page = p.block_table[static_cast<int64_t>(w.b) * p.table_stride + (key >> p.page_shift)];
      if (page >= 0 && page < p.num_pages) return page;
      record_error(p.err, kErrBadPage);
      return p.num_pages;
    };
    for (int n; ok && (n = w.seg_len()) > 0; w.next(p, n), ++seg) {
      int page = box_page(w.blk);
      if (kv == 0) {
        const int qb = seg & 1, qu = seg >> 1;
        if (qu > 0) ok = warp_wait(&bar_qempty[qb], (qu - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutLoad);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar_qfull[qb], GQ::kChunks * GQ::kRowBytes * p.G * p.tok_tile);
#pragma unroll
          for (int ch = 0; ch < GQ::kChunks; ++ch)
            tma_load_3d(smem + L::kOffQ + qb * L::kQBytes + ch * GQ::kChunkBytes, &tm_q, &bar_qfull[qb],
                        ch * (GQ::kRowBytes / 2), w.kvh * p.G, w.u.tok0);
        }
        __syncwarp();
      }
      for (int j = 0; ok && j < n; ++j) {
        const int page_next = j + 1 < n ? box_page(w.blk + j + 1) : 0;
        const int key0 = (w.u.lo / kPBlk + w.blk + j) * kPBlk;
        const int row = (key0 + lane * frag) & ((1 << p.page_shift) - 1);
        const bool cut = key0 < w.u.lo || key0 + kPBlk > w.u.hi;
        const int st = c % U, use = c / U;
        if (use > 0) {
          ok = warp_wait(&bar_empty[st], (use - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutLoad);
          if (!ok) break;
        }
        uint8_t* tile = smem + st * GK::kTileBytes;
        uint64_t* bar = kv == 1 && cut ? bar_vtmp : &bar_full[st];
        if (lane == 0) mbar_arrive_expect_tx(bar, GK::kTileBytes);
        __syncwarp();
        if (lane < n_frag) {
#pragma unroll
          for (int ch = 0; ch < GK::kChunks; ++ch)
            tma_load_4d(tile + ch * GK::kChunkBytes + lane * frag * GK::kRowBytes, map, bar, ch * (GK::kRowBytes / 2),
                        w.kvh, row, page);
        }
        c += 2;
        if (kv == 1 && cut) {
          // Clear the V rows no row of the unit sees.
          drain_wait(bar_vtmp, n_cut & 1, p.err);
          ++n_cut;
          const int k0 = max(0, w.u.lo - key0), k1 = min(kPBlk, w.u.hi - key0);  // visible rows [k0, k1)
          constexpr int kVecs = GK::kRowBytes / 16;
          for (int i = lane; i < kPBlk * kVecs * GK::kChunks; i += 32) {
            const int r = (i / kVecs) % kPBlk;
            if (r < k0 || r >= k1) *reinterpret_cast<uint4*>(tile + i * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_full[st]);
        }
        page = page_next;
      }
    }
    // Teardown: every copy this warp started lands before the CTA exits (older
    // ones of a stage were consumed before it was used again).
    for (int x = c - 2; x >= 0 && x >= c - U; x -= 2)
      drain_wait(&bar_full[x % U], (x / U) & 1, p.err);
    if (kv == 0)
      for (int x = (seg > 2 ? seg - 2 : 0); x < seg; ++x) drain_wait(&bar_qfull[x & 1], (x >> 1) & 1, p.err);
    __syncwarp();
  } else if (warp == kMma) {
    // -------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_s = make_idesc_f16(BF16, 128, N, false, false);
    constexpr uint32_t idesc_o = make_idesc_f16(BF16, 128, N, true, true);
    const AccFlags acc = runtime_flags(p.batch);
    const uint32_t s_ring = smem_u32(smem), s_p = smem_u32(smem + L::kOffP), s_q = smem_u32(smem + L::kOffQ);
    const uint32_t t_o = tmem + 2 * N;
    int seg = 0;
    int seg_n = w.seg_len(), j = 0;  // the walk's block is block j of segment seg
    const int run = w.left;
    // S(i): the walk's current block.
    auto scores = [&](int i) -> bool {
      const int qb = seg & 1, qu = seg >> 1;
      if (j == 0 && !warp_wait(&bar_qfull[qb], qu & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma)) return false;
      const int c = 2 * i, st = c % U;
      if (!warp_wait(&bar_full[st], (c / U) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma)) return false;
      tc_fence_after();
      const uint64_t k_desc = make_sdesc(s_ring + st * GK::kTileBytes, 16, 8 * GK::kRowBytes, GK::kSwz);
      const uint64_t q_desc = make_sdesc(s_q + qb * L::kQBytes, 16, 8 * GQ::kRowBytes, GQ::kSwz);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss_warp(tmem + (i & 1) * N, desc_plus(k_desc, kmajor_step_bytes<D, kPBlk>(kk)),
                    desc_plus(q_desc, kmajor_step_bytes<D, N>(kk)), idesc_s, kk > 0 ? acc.on : acc.off);
      mma_commit_warp(&bar_sfull[i & 1]);
      mma_commit_warp(&bar_empty[st]);
      if (++j == seg_n) {  // the segment's last score product
        mma_commit_warp(&bar_qempty[qb]);
        w.next(p, seg_n);
        ++seg;
        seg_n = w.seg_len();
        j = 0;
      }
      return true;
    };
    bool ok = run > 0 && scores(0);
    bool first = true;  // block i is its segment's first
    for (int i = 0; ok && i < run; ++i) {
      const bool first_next = j == 0;  // the walk stands at block i + 1
      if (i + 1 < run && !(ok = scores(i + 1))) break;
      ok = warp_wait(&bar_pfull[i & 1], (i >> 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
      const int c = 2 * i + 1, st = c % U;
      ok = ok && warp_wait(&bar_full[st], (c / U) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutMma);
      if (!ok) break;
      tc_fence_after();
      const uint64_t v_desc = make_sdesc(s_ring + st * GK::kTileBytes, L::kVLbo, 8 * GK::kRowBytes, GK::kSwz);
      const uint64_t p_desc =
          make_sdesc(s_p + (i & 1) * GP::kTileBytes, GP::kChunkBytes, 8 * GP::kRowBytes, GP::kSwz);
#pragma unroll
      for (int kk = 0; kk < kPBlk / 16; ++kk)
        mma_ss_warp(t_o, desc_plus(v_desc, mnmajor_step_bytes<D>(kk)), desc_plus(p_desc, mnmajor_step_bytes<N>(kk)),
                    idesc_o, (!first || kk > 0) ? acc.on : acc.off);
      mma_commit_warp(&bar_empty[st]);
      mma_commit_warp(&bar_pv[i & 1]);
      first = first_next;
    }
    mma_commit_warp(bar_drain);
    drain_wait(bar_drain, 0, p.err);
  } else {
    // -------------------------------------------------------------- softmax
    const int g = warp >> 2;             // warpgroup: rows g NC .. g NC + NC - 1
    const int q4 = warp & 3;             // lane quarter
    const int key_lane = q4 * 32 + lane;  // key within the block; row of O^T
    const int wt = threadIdx.x & 127;    // thread within the warpgroup
    const int bar_id = 1 + g;
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t t_s = tmem + lane_base + g * NC;
    const uint32_t t_o = tmem + lane_base + 2 * N + g * NC;
    float* m_s = s_m + g * NC;
    float* negm_s = s_negm + g * NC;
    float* alpha_s = s_alpha + g * NC;
    float* red_s = s_red + g * NC * 4;
    const short* tok_s = s_tok + g * NC;
    const int* off_s = s_off + g * NC;
    const float c = p.scale_log2;
    const float2 c2 = make_float2(c, c);
    // This warpgroup's columns of the P^T tile.
    uint8_t* p_tile = smem + L::kOffP;
    const int p_chunk = g * NC / 8;  // first 16-byte chunk of this warpgroup's rows
    int i = 0;  // block within the CTA's run
    bool alive = true;
    float l[NC];
    long long at = s_start->at;  // blocks before the segment's first
    for (int n; alive && (n = w.seg_len()) > 0; w.next(p, n)) {
      const Unit& u = w.u;
      const int n_rows = u.n_tok * p.G;
      const int blk_first = u.lo / kPBlk + w.blk;
      // Blocks every row sees whole: keys in [full_lo, full_hi).
      const int full_lo = max(0, u.pos0 + u.n_tok - 1 - p.win_left);
      const int full_hi = min(u.kv_len, u.pos0 + 1 + p.win_right);
#pragma unroll
      for (int k = 0; k < NC; ++k) l[k] = 0.f;
      // Rows past the unit's hold other tokens' queries, or what shared memory held.
      // +inf for their maximum never moves, and its negative puts their scores
      // below every bound: they have no say in which blocks take the block maximum.
      if (wt < NC) m_s[wt] = g * NC + wt < n_rows ? -INFINITY : INFINITY;
      // The first block, a cut block, the one after it, and any block as long as
      // a row has seen no score above -inf take the block maximum.
      bool exact_max = true;
      for (int jb = 0; jb < n; ++jb, ++i) {
        bool ok = warp_wait(&bar_sfull[i & 1], (i >> 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax);
        // O(i-2) is done (S(i) was issued after it).  Waiting for it keeps this
        // warp one phase behind each of the two barriers, so that a wait for
        // O(i-1) below cannot take the phase before it for it.
        if (ok && i >= 2)
          ok = warp_wait(&bar_pv[i & 1], ((i >> 1) - 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax);
        const int key0 = (blk_first + jb) * kPBlk;
        const int key = key0 + key_lane;
        const bool cut = key0 < full_lo || key0 + kPBlk > full_hi;
        uint32_t sr[NC];
        if (ok) {
          tc_fence_after();
          tmem_ld16(t_s + (i & 1) * N, sr);
        }
        float2 cc = c2;
        if (cut && ok) {
          // The scaled scores in place of the scores (cc = 1 from here on),
          // -inf where the row does not see the key.
          cc = make_float2(1.f, 1.f);
#pragma unroll
          for (int k = 0; k < NC; ++k) {
            const int pos = u.pos0 + tok_s[k];
            const bool hidden = key >= u.kv_len || key > pos + p.win_right || key < pos - p.win_left;
            sr[k] = __float_as_uint(hidden ? -INFINITY : c * __uint_as_float(sr[k]));
          }
        }
        bool need = exact_max || cut;
        exact_max = cut;
        if (!need) {
          float mx = -INFINITY;
#pragma unroll
          for (int k = 0; k < NC; k += 2) {
            const float2 nm = *reinterpret_cast<const float2*>(negm_s + k);
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])), c2, nm);
            mx = max3(mx, y.x, y.y);
          }
          // One barrier per block makes the outcome the same for all lanes.
          need = !named_sync_and(bar_id, 128, ok && mx <= kPagedTau);
        }
        if (need) {
          if (!named_sync_and(bar_id, 128, ok)) {
            alive = false;
            break;
          }
          float y[NC];
#pragma unroll
          for (int k = 0; k < NC; ++k) y[k] = cc.x * __uint_as_float(sr[k]);
          const float mk = warp_reduce_cols16<true>(y);
          if (lane < NC) red_s[lane * 4 + q4] = mk;
          named_sync(bar_id, 128);
          bool moved = false;
          if (wt < NC) {
            const float4 r4 = *reinterpret_cast<const float4*>(red_s + wt * 4);
            const float mb = fmaxf(fmaxf(r4.x, r4.y), fmaxf(r4.z, r4.w));
            const float mo = m_s[wt];
            const float mn = (mb > mo + kPagedTau || mo == -INFINITY) ? mb : mo;
            float a = 1.f;
            if (mn != mo) {
              a = ex2(mo - mn);
              moved = true;
            }
            m_s[wt] = mn;
            negm_s[wt] = mn == -INFINITY ? 0.f : -mn;
            alpha_s[wt] = a;
          }
          moved = !named_sync_and(bar_id, 128, !moved);
          if (jb + 1 < n) {
#pragma unroll
            for (int k = 0; k < NC; k += 4) {
              const float4 m4 = *reinterpret_cast<const float4*>(m_s + k);
              exact_max |= fminf(fminf(m4.x, m4.y), fminf(m4.z, m4.w)) == -INFINITY;
            }
          }
          if (moved && jb > 0) {
#pragma unroll
            for (int k = 0; k < NC; ++k) l[k] *= alpha_s[k];
            ok = warp_wait(&bar_pv[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag, p.err, p.wait_ns,
                           kErrTimeoutSoftmax);
            if (!named_sync_and(bar_id, 128, ok)) {
              alive = false;
              break;
            }
            tc_fence_after();
            uint32_t o16[NC];
            tmem_ld16(t_o, o16);
#pragma unroll
            for (int e = 0; e < NC; ++e) {
              const float a = alpha_s[e];  // 0: the row saw no key before
              o16[e] = a == 0.f ? 0u : __float_as_uint(__uint_as_float(o16[e]) * a);
            }
            tmem_st16(t_o, o16);
            tmem_st_wait();
          }
        }
        // P~ = 2^(c s - m) into the key's row of the P^T tile, rounded to 16 bits
        // (the product takes V as it lies in the cache, so both operands have its
        // type; a weight is off by 2^-8 of itself at most in bf16, 2^-11 in fp16);
        // the running sums take the unrounded values.
        uint8_t* prow = p_tile + (i & 1) * GP::kTileBytes;
#pragma unroll
        for (int k = 0; k < NC; k += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 nm = *reinterpret_cast<const float2*>(negm_s + k + e);
            const float2 y =
                __ffma2_rn(make_float2(__uint_as_float(sr[k + e]), __uint_as_float(sr[k + e + 1])), cc, nm);
            const float2 pe = make_float2(ex2(y.x), ex2(y.y));
            l[k + e] += pe.x;
            l[k + e + 1] += pe.y;
            pk[e / 2] = pack2<BF16>(pe.x, pe.y);
          }
          *reinterpret_cast<uint4*>(prow + swizzled<GP::kRowBytes>(key_lane, p_chunk + k / 8)) =
              make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        fence_proxy_async_smem();
        warp_arrive(&bar_pfull[i & 1]);
      }
      if (!alive) break;
      // ------------------------------------------------------------ segment's end
      const bool whole = n == u.n_blk;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (w.blk == 0 ? 1 : 0);
      bool ok =
          warp_wait(&bar_pv[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag, p.err, p.wait_ns, kErrTimeoutSoftmax);
      const float lk = warp_reduce_cols16<false>(l);
      if (lane < NC) red_s[lane * 4 + q4] = lk;
      if (!named_sync_and(bar_id, 128, ok)) {
        alive = false;
        break;
      }
      if (wt < NC) {
        const float4 r4 = *reinterpret_cast<const float4*>(red_s + wt * 4);
        const float lt = (r4.x + r4.y) + (r4.z + r4.w);
        const bool seen = lt != 0.f;  // (NaN scores make the sum NaN, and the row with it)
        alpha_s[wt] = seen ? 1.f / lt : 0.f;
        const float l2 = seen ? m_s[wt] + log2f(lt) : -INFINITY;
        const int row = g * NC + wt;
        if (row < n_rows) {
          if (whole)
            p.lse[static_cast<int64_t>(w.kvh * p.G + row % p.G) * p.total + u.tok0 + tok_s[wt]] =
                l2 * 0.69314718055994530942f;
          else
            p.lse_part[static_cast<int64_t>(slot) * N + row] = l2;
        }
      }
      if (!whole && w.blk == 0 && threadIdx.x == 0)
        p.desc[blockIdx.x] = make_int4(u.tok0, u.n_tok, w.kvh, static_cast<int>((at + u.n_blk - 1) / s_start->share));
      named_sync(bar_id, 128);
      tc_fence_after();
      // Lane d of the warps holds column d of every row's O: a row is one
      // coalesced store per warp.
      const int rows_here = n_rows - g * NC;
      float* part = p.o_part + (static_cast<int64_t>(slot) * N + g * NC) * D + key_lane;
      elem_t* out = static_cast<elem_t*>(p.o) + (static_cast<int64_t>(u.tok0) * p.H + w.kvh * p.G) * D + key_lane;
      if (rows_here > 0) {  // (warp-uniform)
        uint32_t o16[NC];
        tmem_ld16(t_o, o16);
        if (key_lane < D) {
          if (whole) {
#pragma unroll
            for (int e = 0; e < NC; ++e) {
              const float inv = alpha_s[e];
              const float v = inv == 0.f ? 0.f : __uint_as_float(o16[e]) * inv;
              if (e < rows_here) {
                elem_t* dst = out + static_cast<int64_t>(off_s[e]) * D;
                if constexpr (BF16) *dst = __float2bfloat16_rn(v);
                else *dst = __float2half_rn(v);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < NC; ++e) {
              const float inv = alpha_s[e];
              const float v = inv == 0.f ? 0.f : __uint_as_float(o16[e]) * inv;
              if (e < rows_here) part[e * D] = v;
            }
          }
        }
      }
      named_sync(bar_id, 128);  // the per-row arrays are free for the next segment
      tc_fence_before();
      at += n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
  if (p.after_tile) griddep_wait();
}

namespace {

template <int D, int N, bool BF16>
cudaError_t launch_paged_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                           int grid, cudaStream_t stream) {
  using L = PagedLayout<D, N>;
  auto kern = fa_paged_kernel<D, N, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(grid), L::kThreads, L::kSmemBytes, stream, tq, tk, tv, p);
}

template <int D>
cudaError_t launch_paged_n(int N, bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const PagedParams& p, int grid, cudaStream_t s) {
  switch (N) {
    case 16: return bf16 ? launch_paged_t<D, 16, true>(tq, tk, tv, p, grid, s)
                         : launch_paged_t<D, 16, false>(tq, tk, tv, p, grid, s);
    case 32: return bf16 ? launch_paged_t<D, 32, true>(tq, tk, tv, p, grid, s)
                         : launch_paged_t<D, 32, false>(tq, tk, tv, p, grid, s);
    case 64: return bf16 ? launch_paged_t<D, 64, true>(tq, tk, tv, p, grid, s)
                         : launch_paged_t<D, 64, false>(tq, tk, tv, p, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

}  // namespace fa
