// Rotary positions of packed Q and K rows, their gradient, and the append of
// new K and V rows to a paged cache (which rotates Q and K on the way).
//
// A row's first 2r columns are r pairs (a_i, b_i): columns (i, r + i) in the
// half layout, (2i, 2i + 1) in the interleaved one.  A token at position p
// turns pair i by the angle t = p f_i:
//
//   a' = mag (a cos t - b sin t),   b' = mag (b cos t + a sin t);
//
// columns past 2r pass unchanged.  The map is mag times an orthogonal one, so
// the gradient is the same map with -t.
//
// Angles.  f_i comes as a 64-bit step, f_i / (2 pi) in units of 2^-64 turns:
// p * step mod 2^64 is the angle's fraction of a turn, exactly, however far
// out p is (a 32-bit float product p f_i is already off by 2^-4 radians at
// p = 2^20).  Its top 32 bits, as a signed number of 2^-31 half turns, go to
// sincospif.  Everything after that is 32-bit, rounded once when stored.
//
// Every element is read once and written once and the arithmetic is a few
// operations an element, so memory bounds the kernel: 16384 tokens of 32 heads
// of 64 in 21.2 us, 8192 tokens of 36 heads of 128 in 24.0, 94 % of the copy
// rate.  A CTA takes a few
// tokens; the angles (r sine/cosine pairs a token) are computed once per
// token, into shared memory, and used by all of its heads.  A thread owns 16
// columns (two 16-byte vectors) of kRows rows at a time and loads them all
// before it works on the angles, so the angles' latency (positions, steps,
// sincospif, a barrier) passes while the rows are on their way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kernel_common.cuh"
#include "fa_paged.cuh"

namespace fa {

namespace {

constexpr int kRopeMaxThreads = 256;
constexpr int kRopeRows = 2;        // rows a thread has in flight
constexpr int kRopeMaxTok = 128;    // tokens per CTA at most
constexpr int kRopeMaxAngles = 1024;  // tokens x pairs per CTA at most
constexpr int kRopeIdle = 8 * kPagedSms;  // append: CTAs without tokens in a launch, at most

enum RopeForm {
  kInterleaved,   // pairs (2i, 2i+1): any r, a vector holds whole pairs
  kHalf,          // pairs (i, r + i), r a multiple of 8: vectors at 8j and r + 8j
  kHalfAny,       // any other r: partners come through shared memory, one element at a time (8192 tokens of 36
                  // heads of 128: r = 64 23.7 us, r = 50 78; that form is instructions, not memory)
};

enum RopeMode {
  kRotate,
  kAppend,        // as many CTAs for every sequence as the longest may need
  kAppendDealt,   // CTAs dealt by tokens
};

// Eight 16-bit elements.
union Vec8 {
  uint4 v;
  uint32_t w[4];  // pairs of neighbours
  uint16_t h[8];
};

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t h) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
  else return __half2float(__ushort_as_half(h));
}
// Two neighbours in a 32-bit word (the first in its low half).
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint16_t from_float(float x) {
  if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else return __half_as_ushort(__float2half_rn(x));
}

}  // namespace

namespace {

// First token, new tokens and cache length of sequence b.  One whose lengths
// contradict the call is recorded as an error, and has no tokens.
struct AppendLens {
  int first, len, kv_len;
};
__device__ __forceinline__ AppendLens append_lens(const RopeParams& p, int b) {
  const int a = p.cu_seqlens[b], e = p.cu_seqlens[b + 1], kv_len = p.kv_lens[b];
  int err = 0;
  if (a < 0 || e < a || e - a > p.max_len || e > p.total) err = kErrBadSeqlens;
  else if (e > a && (kv_len < e - a || kv_len > p.max_kv)) err = kErrBadCache;
  if (err == 0) return AppendLens{a, e - a, kv_len};
  if (threadIdx.x == 0) ptx::record_error(p.err, err);
  return AppendLens{0, 0, 0};
}

}  // namespace

// Append: rows of a packed batch; K rows go to their pages, and V rows (after
// the K rows of a token) are copied to theirs.
template <RopeForm FORM, bool BF16, RopeMode MODE>
__global__ void __launch_bounds__(kRopeMaxThreads) fa_rope_kernel(const RopeParams p) {
  constexpr bool APPEND = MODE != kRotate;
  __shared__ __align__(16) float2 s_cs[kRopeMaxAngles];
  __shared__ int64_t s_slot[APPEND ? kRopeMaxTok : 1];  // element offset of the token's rows in the caches; -1: none
  __shared__ uint4 s_rows[FORM == kHalfAny ? kRopeMaxThreads * 2 * kRopeRows : 1];

  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  int tile = blockIdx.x;
  int tok0, n_tok;  // the CTA's tokens
  int pos0 = 0;     // append: cache position of token tok0
  int b = 0;
  if constexpr (APPEND) {
    if constexpr (MODE == kAppend) {
      b = tile / p.tiles;
      tile -= b * p.tiles;
    } else {
      // Sequence b's CTAs are cu[b] / tok + b up to the next one's: at least as
      // many as it needs, and in order, so a search finds b.  No CTA may come to
      // a sequence whose offsets contradict the call: CTA x checks sequence x too.
      if (tile < p.batch && threadIdx.x == 0) append_lens(p, tile);
      int above = p.batch;  // b's first CTA is at or before this one, above's behind it
      while (above - b > 1) {
        const int mid = b + (above - b) / 2;
        if (static_cast<int64_t>(p.cu_seqlens[mid] / p.tok_per_cta) + mid <= tile) b = mid;
        else above = mid;
      }
      const int64_t own = tile - (static_cast<int64_t>(p.cu_seqlens[b] / p.tok_per_cta) + b);
      if (own < 0 || own > p.total / p.tok_per_cta) return;
      tile = static_cast<int>(own);
    }
    const AppendLens s = append_lens(p, b);
    tok0 = tile * p.tok_per_cta;
    n_tok = min(p.tok_per_cta, s.len - tok0);
    if (n_tok <= 0) return;
    pos0 = s.kv_len - s.len + tok0;
    tok0 += s.first;
  } else {
    tok0 = tile * p.tok_per_cta;
    n_tok = min(p.tok_per_cta, p.total - tok0);
  }

  const int r = p.r, D = p.D;
  // A token's angles in shared memory.  A thread that turns 8 pairs (8 col ..)
  // reads them as four 16-byte words, the words of neighbouring threads side by
  // side; side by side in pair order, eight threads would meet in two banks.
  const int groups = (r + 7) / 8;
  const int angles = FORM == kHalfAny ? r : 8 * groups;
  auto angle_at = [&](int j) {
    return FORM == kHalfAny ? j : 2 * (((j >> 1) & 3) * groups + (j >> 3)) + (j & 1);
  };
  const int rot_heads = p.H + p.H_kv;                  // rows that turn
  const int heads = rot_heads + (APPEND ? p.H_kv : 0);  // rows of a token: Q, K (and V)
  const int n_rows = n_tok * heads;
  const int threads = blockDim.x;
  const int lanes = threads >> p.log2_items;  // rows the CTA takes at once
  const int col = static_cast<int>(threadIdx.x) & ((1 << p.log2_items) - 1);
  // This thread's two vectors of a row that turns; of a V row they are 16 col, 16 col + 8.
  bool turns;  // kHalf: its columns turn
  int oa, ob;
  if (FORM == kHalf) {
    turns = 8 * col < r;
    oa = turns ? 8 * col : 2 * r + 16 * (col - r / 8);
    ob = turns ? oa + r : oa + 8;
  } else {
    turns = 16 * col < 2 * r;
    oa = 16 * col;
    ob = oa + 8;
  }

  for (int first = 0; first < n_rows; first += kRopeRows * lanes) {  // (one round, but for very many heads)
    const int base = first + (static_cast<int>(threadIdx.x) >> p.log2_items);
    Vec8 x[kRopeRows], y[kRopeRows];
    int tok[kRopeRows], head[kRopeRows];  // of each row
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
      const int row = base + u * lanes;
      if (row < n_rows) {
        const int t = row / heads, h = row - t * heads;
        tok[u] = t;
        head[u] = h;
        const int64_t tk = tok0 + t;
        const uint16_t* src;
        if (h < p.H) src = static_cast<const uint16_t*>(p.q) + tk * p.q_stride + h * D;
        else if (!APPEND || h < rot_heads) src = static_cast<const uint16_t*>(p.k) + tk * p.k_stride + (h - p.H) * D;
        else src = static_cast<const uint16_t*>(p.v) + tk * p.v_stride + (h - rot_heads) * D;
        const bool v_row = APPEND && h >= rot_heads;
        x[u].v = *reinterpret_cast<const uint4*>(src + (v_row ? 16 * col : oa));
        y[u].v = *reinterpret_cast<const uint4*>(src + (v_row ? 16 * col + 8 : ob));
      }
    }
    if (first == 0) {
      // Angles of the CTA's tokens, and (append) where their rows go.
      for (int i = threadIdx.x; i < n_tok * r; i += threads) {
        const int t = i / r, j = i - t * r;
        int pos;
        if (APPEND && p.positions == nullptr) pos = pos0 + t;
        else pos = p.positions[tok0 + t];
        const unsigned long long phase =
            static_cast<unsigned long long>(static_cast<long long>(pos)) * p.steps[j];
        float s, c;
        sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
        s_cs[t * angles + angle_at(j)] = make_float2(c * p.mag, s * p.mag_sin);
      }
      if constexpr (APPEND) {
        for (int i = threadIdx.x; i < n_tok; i += threads) {
          const int pos = pos0 + i;
          const int page = p.block_table[static_cast<int64_t>(b) * p.table_stride + (pos >> p.page_shift)];
          int64_t slot = -1;
          if (page >= 0 && page < p.num_pages)
            slot = static_cast<int64_t>(page) * p.page_stride +
                   static_cast<int64_t>(pos & ((1 << p.page_shift) - 1)) * p.row_stride;
          else
            ptx::record_error(p.err, kErrBadPage);
          s_slot[i] = slot;
        }
      }
      __syncthreads();
    }
    uint16_t* stage = reinterpret_cast<uint16_t*>(s_rows);
    if constexpr (FORM == kHalfAny) {
      // A row's threads are neighbours in one warp: each row's D elements side by side.
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kRopeRows; ++u) {
        s_rows[2 * (u * threads + static_cast<int>(threadIdx.x))] = x[u].v;
        s_rows[2 * (u * threads + static_cast<int>(threadIdx.x)) + 1] = y[u].v;
      }
      __syncwarp();
    }
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
      const int row = base + u * lanes;
      if (row >= n_rows) continue;
      const int t = tok[u], h = head[u];
      const int64_t tk = tok0 + t;
      uint16_t* dst;
      const bool v_row = APPEND && h >= rot_heads;
      if (h < p.H) {
        dst = static_cast<uint16_t*>(p.q_out) + tk * p.q_out_stride + h * D;
      } else if constexpr (APPEND) {
        if (s_slot[t] < 0) continue;
        dst = v_row ? static_cast<uint16_t*>(p.v_out) + s_slot[t] + (h - rot_heads) * p.head_stride
                    : static_cast<uint16_t*>(p.k_out) + s_slot[t] + (h - p.H) * p.head_stride;
      } else {
        dst = static_cast<uint16_t*>(p.k_out) + tk * p.k_out_stride + (h - p.H) * D;
      }
      if (turns && !v_row) {
        const float2* cs = s_cs + t * angles;
        const float4* cs4 = reinterpret_cast<const float4*>(cs) + col;
        if constexpr (FORM == kHalf) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 w = cs4[i * groups];
            const float2 a = unpack2<BF16>(x[u].w[i]), bb = unpack2<BF16>(y[u].w[i]);
            x[u].w[i] = pack2<BF16>(a.x * w.x - bb.x * w.y, a.y * w.z - bb.y * w.w);
            y[u].w[i] = pack2<BF16>(bb.x * w.x + a.x * w.y, bb.y * w.z + a.y * w.w);
          }
        } else if constexpr (FORM == kInterleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 w = cs4[i / 2 * groups];
            uint32_t* v = i < 4 ? &x[u].w[i] : &y[u].w[i - 4];
            const float2 a = unpack2<BF16>(v[0]), bb = unpack2<BF16>(v[1]);
            if (8 * col + i < r) v[0] = pack2<BF16>(a.x * w.x - a.y * w.y, a.y * w.x + a.x * w.y);
            if (8 * col + i + 1 < r) v[1] = pack2<BF16>(bb.x * w.z - bb.y * w.w, bb.y * w.z + bb.x * w.w);
          }
        } else {
          // Column c pairs with c + r (c < r) or c - r, read from the staged row.
          const uint16_t* line = stage + 16 * (u * threads + static_cast<int>(threadIdx.x) - col);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = oa + i;
            if (c < 2 * r) {
              Vec8& v = i < 8 ? x[u] : y[u];
              const bool low = c < r;
              const float2 w = cs[low ? c : c - r];
              const float own = to_float<BF16>(v.h[i & 7]), other = to_float<BF16>(line[low ? c + r : c - r]);
              v.h[i & 7] = from_float<BF16>(low ? own * w.x - other * w.y : own * w.x + other * w.y);
            }
          }
        }
      }
      *reinterpret_cast<uint4*>(dst + (v_row ? 16 * col : oa)) = x[u].v;
      *reinterpret_cast<uint4*>(dst + (v_row ? 16 * col + 8 : ob)) = y[u].v;
    }
  }
}

namespace {

template <RopeForm FORM, bool BF16>
cudaError_t launch_rope_f(const RopeParams& p, RopeMode mode, unsigned grid, int threads, cudaStream_t s) {
  auto kern = mode == kRotate ? fa_rope_kernel<FORM, BF16, kRotate>
                              : (mode == kAppend ? fa_rope_kernel<FORM, BF16, kAppend>
                                                 : fa_rope_kernel<FORM, BF16, kAppendDealt>);
  return launch_dependent(kern, dim3(grid), threads, 0, s, p);
}

template <bool BF16>
cudaError_t launch_rope_t(const RopeParams& p, RopeMode mode, unsigned grid, int threads, cudaStream_t s) {
  if (p.interleaved) return launch_rope_f<kInterleaved, BF16>(p, mode, grid, threads, s);
  if (p.r % 8 == 0) return launch_rope_f<kHalf, BF16>(p, mode, grid, threads, s);
  return launch_rope_f<kHalfAny, BF16>(p, mode, grid, threads, s);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, bool bf16, bool append, int batch, cudaStream_t stream) {
  p.log2_items = p.D == 16 ? 0 : (p.D == 32 ? 1 : (p.D == 64 ? 2 : 3));  // D / 16 threads a row
  // Tokens and threads of a CTA: all rows in one round (kRopeRows of them a
  // thread), with the fewest idle threads.  A second round's loads would wait
  // for the first round's stores: 8192 tokens of 36 heads of 128, one token a
  // CTA, took 29.4 us in two rounds of 128 threads (44 % of them idle).
  const int64_t rows_tok = p.H + (append ? 2 : 1) * p.H_kv;
  int64_t most = p.r > 0 ? kRopeMaxAngles / ((p.r + 7) / 8 * 8) : kRopeMaxTok;
  most = most < 1 ? 1 : (most > kRopeMaxTok ? kRopeMaxTok : most);
  const int64_t fits = (kRopeMaxThreads >> p.log2_items) * kRopeRows;  // rows of one round at most
  int64_t tok = 1, threads = kRopeMaxThreads;
  double best = -1.0;
  for (int64_t t = 1; t <= most && (t == 1 || t * rows_tok <= fits); ++t) {
    const int64_t rows = t * rows_tok;
    int64_t th = (((rows + kRopeRows - 1) / kRopeRows << p.log2_items) + 31) / 32 * 32;
    if (th > kRopeMaxThreads) th = kRopeMaxThreads;
    if (th < 128 && t < most && (t + 1) * rows_tok <= fits) continue;  // (a CTA of a few warps is mostly set-up)
    const int64_t round = (th >> p.log2_items) * kRopeRows;
    const double full = static_cast<double>(rows) / static_cast<double>((rows + round - 1) / round * round);
    if (full > best + 0.02) {
      best = full;
      tok = t;
      threads = th;
    }
  }
  p.tok_per_cta = static_cast<int>(tok);
  // No sequence has more tokens than there are, whatever the caller's bound.
  const int64_t longest = append && p.max_len < p.total ? p.max_len : p.total;
  p.tiles = static_cast<int>((longest + tok - 1) / tok);
  p.batch = batch;
  int64_t ctas = static_cast<int64_t>(p.tiles) * (append ? batch : 1);
  RopeMode mode = append ? kAppend : kRotate;
  // Under a loose bound, or with one sequence much longer than the others, most
  // of those CTAs have no tokens; dealt by tokens there are few of them, but each
  // searches its sequence.
  // Both ways (us, 36 heads of 128, the first way / dealt): 64 sequences of one
  // token 3.1 / 4.2, 8 of 128 5.2 / 6.3, 64 tokens beside 7 single ones (433 idle
  // CTAs) 3.2 / 3.7, 100 beside 9 of 10 (790 idle) 3.77 / 3.83; 100 beside 31 of
  // 10 (2750 idle) 5.7 / 4.5, 512 beside 63 single ones (32000 idle) 34 / 6.6.
  const int64_t dealt = p.total / tok + batch;
  if (append && ctas > dealt + kRopeIdle) {
    ctas = dealt;
    mode = kAppendDealt;
  }
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(ctas);
  return bf16 ? launch_rope_t<true>(p, mode, grid, static_cast<int>(threads), stream)
              : launch_rope_t<false>(p, mode, grid, static_cast<int>(threads), stream);
}

}  // namespace fa
