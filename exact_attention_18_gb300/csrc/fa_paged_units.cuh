// What the two paged-attention kernels share: the units of a call, the run of
// blocks a CTA takes, and the walk over it.
#pragma once

#include "fa_kernel_common.cuh"
#include "fa_paged.cuh"

namespace fa {
using namespace ptx;

namespace {

// Geometry of one unit; n_blk = 0 when it does not exist.
struct Unit {
  int tok0;    // first token (row of Q, O)
  int n_tok;   // tokens
  int pos0;    // cache position of its first token
  int kv_len;
  int lo, hi;  // keys any of its rows sees: [lo, hi)
  int n_blk;   // blocks of 2^SHIFT keys, from block lo >> SHIFT
  int end_tile;  // tiles of the sequence (tiles from here on do not exist)
};

// Unit (b, tile) of the call.  A sequence whose lengths contradict the call is
// recorded as an error and has no units.  A unit whose rows see no key keeps
// one wholly masked block, which writes O = 0, L = -inf.
struct SeqLens {
  int a, e, kv;  // cu_seqlens[b], cu_seqlens[b + 1], kv_lens[b]
};
__device__ __forceinline__ SeqLens seq_lens(const PagedParams& p, int b) {
  return SeqLens{p.cu_seqlens[b], p.cu_seqlens[b + 1], p.kv_lens[b]};
}
template <int SHIFT>
__device__ __forceinline__ Unit paged_unit(const PagedParams& p, const SeqLens& s, int tile) {
  Unit u;
  const int a = s.a, e = s.e, kv = s.kv;
  u.n_blk = 0;
  u.end_tile = 0;
  u.tok0 = u.n_tok = u.pos0 = u.kv_len = u.lo = u.hi = 0;
  if (a < 0 || e < a || e - a > p.max_q || e > p.total) {
    record_error(p.err, kErrBadSeqlens);
    return u;
  }
  if (kv < 0 || kv > p.max_k) {
    record_error(p.err, kErrBadCache);
    return u;
  }
  const int n = e - a;
  if (n < p.tok_lo || n > p.tok_hi) return u;  // another kernel of the call takes this sequence
  u.end_tile = (n + p.tok_tile - 1) / p.tok_tile;
  const int t0 = tile * p.tok_tile;
  if (t0 >= n) return u;
  u.tok0 = a + t0;
  u.n_tok = min(p.tok_tile, n - t0);
  u.pos0 = kv - n + t0;
  u.kv_len = kv;
  u.lo = max(0, u.pos0 - p.win_left);
  u.hi = min(kv, u.pos0 + u.n_tok + p.win_right);
  if (u.hi <= u.lo) {
    u.lo = u.hi = 0;
    u.n_blk = 1;
  } else {
    u.n_blk = ((u.hi + (1 << SHIFT) - 1) >> SHIFT) - (u.lo >> SHIFT);
  }
  return u;
}

// Cost of one of a unit's blocks, for dealing the call's blocks to CTAs.  COSTS
// (the tile kernel): by the tiles of sub_tok tokens that the unit fills; else 1.
template <bool COSTS>
__device__ __forceinline__ int block_cost(const PagedParams& p, const Unit& u) {
  if constexpr (!COSTS) return 1;
  return static_cast<int>(p.costs >> (8 * ((u.n_tok - 1) / p.sub_tok))) & 255;
}

// Where a CTA's run of blocks starts (in shared memory).
struct RunStart {
  int b, tile, kvh, blk;  // unit and block within it
  long long at;           // cost of all blocks before that one
  long long left;         // cost of the run (0: no block starts in it)
  long long share;        // cost of a CTA's stretch
  Unit u;
};

// Walks the segments (runs of blocks of one unit) of a CTA's run of blocks.
template <int SHIFT, bool COSTS>
struct SegWalk {
  int b, tile, kvh;
  int blk;        // next block within the unit
  typename std::conditional<COSTS, long long, int>::type left;  // cost from the next block to the run's end
  int cost;       // of one of the unit's blocks
  Unit u;
  // Blocks of the current segment (0: the run is over).  A block is the CTA's
  // when it starts inside the stretch.
  __device__ __forceinline__ int seg_len() const {
    const int rest = u.n_blk - blk;
    if constexpr (!COSTS) return min(left, rest);
    if (left >= static_cast<long long>(rest) * cost) return rest;
    return (static_cast<int>(left) + cost - 1) / cost;
  }
  __device__ __forceinline__ void start(const PagedParams& p, const RunStart& s) {
    b = s.b;
    tile = s.tile;
    kvh = s.kvh;
    blk = s.blk;
    left = s.left;
    u = s.u;
    cost = 1;
    if (left == 0) return;
    if (COSTS && kvh == p.H_kv) next_unit(p);
    else cost = block_cost<COSTS>(p, u);
  }
  // Past the current segment of n blocks.
  __device__ __forceinline__ void next(const PagedParams& p, int n) {
    if constexpr (COSTS) left -= static_cast<long long>(n) * cost;
    else left -= n;
    blk = 0;
    if (left <= 0) {
      left = 0;
      return;
    }
    if (++kvh == p.H_kv) next_unit(p);
  }
  __device__ __forceinline__ void next_unit(const PagedParams& p) {
    kvh = 0;
    do {
      if (++tile >= u.end_tile) {
        tile = 0;
        ++b;
      }
      if (b >= p.batch) {  // past the last unit
        left = 0;
        return;
      }
      u = paged_unit<SHIFT>(p, seq_lens(p, b), tile);
    } while (u.n_blk == 0);
    cost = block_cost<COSTS>(p, u);
  }
};

// This CTA's run of blocks.  The blocks of all units (x = b * tiles + tile in
// order, H_kv heads each), laid end to end by their costs, are cut into equal
// stretches; a block belongs to the CTA in whose stretch it starts.  Every
// thread sums some units, and a block-wide scan gives the ones that hold the
// CTA's first block.  A stretch is at least the largest cost long, so that a
// unit which spans several CTAs has blocks in each.  `own`: the lengths of this thread's first unit, loaded
// by the caller before its other set-up so that they arrive meanwhile.
// s_warp: one entry per warp.  Ends with the writes to *start unsynchronised;
// start->left and start->u must be zero on entry.
__device__ __forceinline__ int paged_first_unit(const PagedParams& p, int threads, int* per) {
  const int X = p.batch * p.tiles;
  *per = X <= threads ? 1 : (X + threads - 1) / threads;
  return min(X, static_cast<int>(threadIdx.x) * *per);
}

// The unit index after x = b * tiles + tile, whose unit is u.  The tiles that a
// sequence does not have are stepped over: under a loose bound they are most.
__device__ __forceinline__ int next_tile(const PagedParams& p, const Unit& u, int x, int* b, int* tile) {
  if (*tile + 1 < u.end_tile) {
    ++*tile;
    return x + 1;
  }
  x += p.tiles - *tile;
  ++*b;
  *tile = 0;
  return x;
}

// I: int where the host has bounded the call's cost below 2^31 (64-bit scans
// and divisions cost a decoding call a microsecond), else long long.
template <int SHIFT, bool COSTS, int THREADS, typename I>
__device__ __forceinline__ void paged_find_run_t(const PagedParams& p, const SeqLens& own, I* s_warp, RunStart* start) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int per;
  const int x0 = paged_first_unit(p, THREADS, &per), x1 = min(p.batch * p.tiles, x0 + per);
  int b = p.tiles == 1 ? x0 : x0 / p.tiles, tile = x0 - b * p.tiles;
  Unit u0;
  u0.n_blk = 0;
  I mine = 0;
  if (x0 < x1) {
    u0 = paged_unit<SHIFT>(p, own, tile);
    mine = u0.n_blk * static_cast<I>(u0.n_blk ? block_cost<COSTS>(p, u0) : 0);
    for (int x = next_tile(p, u0, x0, &b, &tile); x < x1;) {
      const Unit u = paged_unit<SHIFT>(p, seq_lens(p, b), tile);
      if (u.n_blk) mine += u.n_blk * static_cast<I>(block_cost<COSTS>(p, u));
      x = next_tile(p, u, x, &b, &tile);
    }
  }
  I incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const I o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  I before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const I v = s_warp[w];
    if (w < warp) before += v;
    total += v;
  }
  total *= p.H_kv;
  I share = (total + static_cast<I>(gridDim.x) - 1) / static_cast<I>(gridDim.x);
  if (COSTS && share < kMaxBlockCost) share = kMaxBlockCost;
  const I s = share * static_cast<I>(blockIdx.x);
  I at = (before + incl - mine) * p.H_kv;  // where this thread's units start
  if (s >= at && s - at < mine * p.H_kv) {
    b = p.tiles == 1 ? x0 : x0 / p.tiles;
    tile = x0 - b * p.tiles;
    Unit u = u0;
    for (int x = x0; x < x1;) {
      if (x > x0) u = paged_unit<SHIFT>(p, seq_lens(p, b), tile);
      const int cost = u.n_blk ? block_cost<COSTS>(p, u) : 0;
      const I n = static_cast<I>(u.n_blk) * p.H_kv * cost;
      if (s - at < n) {
        // The first block that starts at s or later.  Behind the unit's last
        // one it is the next unit's first: the walk steps there.
        const I rem = COSTS ? (s - at + cost - 1) / cost : s - at;
        const int kvh = static_cast<int>(rem / u.n_blk);
        const I first = at + rem * cost;
        const I end = total < s + share ? total : s + share;
        start->b = b;
        start->tile = tile;
        start->kvh = kvh;
        start->blk = static_cast<int>(rem - static_cast<I>(kvh) * u.n_blk);
        start->at = first;
        start->left = end > first ? end - first : 0;
        start->u = u;
        break;
      }
      at += n;
      x = next_tile(p, u, x, &b, &tile);
    }
  }
  if (threadIdx.x == 0) start->share = share;
}

template <int SHIFT, bool COSTS, int THREADS>
__device__ __forceinline__ void paged_find_run(const PagedParams& p, const SeqLens& own, long long* s_warp,
                                               RunStart* start) {
  if (p.small) paged_find_run_t<SHIFT, COSTS, THREADS, int>(p, own, reinterpret_cast<int*>(s_warp), start);
  else paged_find_run_t<SHIFT, COSTS, THREADS, long long>(p, own, s_warp, start);
}

// The tile kernel's word to the few-row kernel behind it in the same call: the
// grids before the call have completed and their writes are visible.  A grid's
// own griddep_wait would say so too, but only when the tile kernel has ended;
// the release, in a thread that has waited itself, and the acquire hand the
// order on to a grid that runs beside it.
__device__ __forceinline__ void say_go(const PagedParams& p) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p.go), "l"(p.ticket) : "memory");
}
__device__ __forceinline__ bool heard_go(const PagedParams& p) {
  unsigned long long x;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(x) : "l"(p.go) : "memory");
  return x == p.ticket;
}
// Orders what this thread has seen before its later bulk copies from global memory.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

}  // namespace

}  // namespace fa
