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
// operations an element, so memory bounds the kernel.  A CTA takes a few
// tokens, so the angles (r sine/cosine pairs a token) are computed once per
// token, into shared memory, and used by all of its heads.  A thread keeps
// its pair columns and walks over (token, head) rows, two rows in flight.
// Measured (see the cache operators' table in the design notes for all
// cases): 16384 tokens of 32 heads of 64 fp16 in 29 us, 4.6 TB/s of reads and
// writes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kernel_common.cuh"
#include "fa_paged.cuh"

namespace fa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTok = 16;   // tokens per CTA at most
constexpr int kRopeMaxPairs = 64;  // D / 2 at most
// Elements per CTA aimed at (tokens per CTA are chosen for it): four 16-pair
// items a thread at D = 128.
constexpr int kRopeElems = 16384;

// N consecutive 16-bit elements.
template <int N>
struct Vec16;
template <>
struct Vec16<8> { using type = uint4; };
template <>
struct Vec16<4> { using type = uint2; };
template <>
struct Vec16<2> { using type = uint32_t; };
template <>
struct Vec16<1> { using type = uint16_t; };

template <int N, bool BF16>
struct Pack {
  using V = typename Vec16<N>::type;
  union {
    V v;
    uint16_t h[N];
  };
  __device__ __forceinline__ float get(int i) const {
    if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(h[i]) << 16);
    else return __half2float(__ushort_as_half(h[i]));
  }
  __device__ __forceinline__ void set(int i, float x) {
    if constexpr (BF16) h[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    else h[i] = __half_as_ushort(__float2half_rn(x));
  }
};

// One thread's share of one row: VEC pairs (two vectors of VEC elements), or
// VEC elements past the rotated part to copy.
template <int VEC, bool BF16>
struct RopeItem {
  Pack<VEC, BF16> a, b;
  const uint16_t* src;
  uint16_t* dst;  // nullptr: nothing to store
};

}  // namespace

// VEC: pairs per item, the largest power of two up to 8 that divides r, so
// that every vector is aligned.  APPEND: rows of a packed batch whose K goes
// to its pages and whose V is copied there.
template <int VEC, bool INTER, bool BF16, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeParams p) {
  __shared__ float2 s_cs[kRopeMaxTok * kRopeMaxPairs];
  __shared__ int64_t s_slot[kRopeMaxTok];  // element offset of the token's K (and V) row in the cache; -1: none

  int tile = blockIdx.x;
  int tok0, n_tok;  // the CTA's tokens
  int pos0 = 0;  // append: cache position of token tok0
  int b = 0;
  if constexpr (APPEND) {
    b = tile / p.tiles;
    tile -= b * p.tiles;
    tok0 = tile * p.tok_per_cta;
    int a, len;
    if (!packed_sample(p.cu_seqlens, b, p.max_len, p.total, p.err, &a, &len)) return;
    const int kv_len = __ldg(p.kv_lens + b);
    if (len == 0) return;
    if (kv_len < len || kv_len > p.max_kv) {
      if (threadIdx.x == 0) ptx::record_error(p.err, kErrBadCache);
      return;
    }
    n_tok = min(p.tok_per_cta, len - tok0);
    pos0 = kv_len - len + tok0;
    tok0 += a;
  } else {
    tok0 = tile * p.tok_per_cta;
    n_tok = min(p.tok_per_cta, p.total - tok0);
  }
  if (n_tok <= 0) return;

  // Angles of the CTA's tokens, and (append) where their rows go.
  for (int i = threadIdx.x; i < n_tok * p.r; i += kRopeThreads) {
    const int t = i / p.r, j = i - t * p.r;
    int pos;
    if (APPEND && p.positions == nullptr) pos = pos0 + t;
    else pos = __ldg(p.positions + tok0 + t);
    const unsigned long long phase =
        static_cast<unsigned long long>(static_cast<long long>(pos)) * __ldg(p.steps + j);
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    s_cs[i] = make_float2(c * p.mag, s * p.mag_sin);
  }
  if constexpr (APPEND) {
    if (static_cast<int>(threadIdx.x) < n_tok) {
      const int pos = pos0 + static_cast<int>(threadIdx.x);
      const int page = __ldg(p.block_table + static_cast<int64_t>(b) * p.table_stride + (pos >> p.page_shift));
      int64_t slot = -1;
      if (page >= 0 && page < p.num_pages)
        slot = static_cast<int64_t>(page) * p.page_stride +
               static_cast<int64_t>(pos & ((1 << p.page_shift) - 1)) * p.row_stride;
      else
        ptx::record_error(p.err, kErrBadPage);
      s_slot[threadIdx.x] = slot;
    }
  }
  __syncthreads();

  // Items of a row: R of VEC pairs, then C copies of VEC elements.
  const int R = p.r / VEC;
  const int heads = p.H + p.H_kv;
  auto rows_of = [&](int row, const uint16_t** src, uint16_t** dst, int* t) {
    *t = row / heads;
    const int h = row - *t * heads;
    const int64_t tk = tok0 + *t;
    if (h < p.H) {
      *src = static_cast<const uint16_t*>(p.q) + tk * p.q_stride + h * p.D;
      *dst = static_cast<uint16_t*>(p.q_out) + tk * p.q_out_stride + h * p.D;
    } else {
      const int g = h - p.H;
      *src = static_cast<const uint16_t*>(p.k) + tk * p.k_stride + g * p.D;
      if constexpr (APPEND) {
        const int64_t slot = s_slot[*t];
        *dst = slot < 0 ? nullptr : static_cast<uint16_t*>(p.k_out) + slot + g * p.head_stride;
      } else {
        *dst = static_cast<uint16_t*>(p.k_out) + tk * p.k_out_stride + g * p.D;
      }
    }
  };
  using P = Pack<VEC, BF16>;
  using V = typename P::V;
  const int per = R + p.copies;  // items per row (at most 64)
  const int lanes = kRopeThreads / per;
  const int n_rows = n_tok * heads;
  const int col = static_cast<int>(threadIdx.x) % per, row_first = static_cast<int>(threadIdx.x) / per;
  if (row_first < lanes) {
    const bool turn = col < R;
    const int oa = turn ? (INTER ? 2 * VEC * col : VEC * col) : 2 * p.r + VEC * (col - R);
    const int ob = INTER ? oa + VEC : oa + p.r;
    for (int row = row_first; row < n_rows; row += 2 * lanes) {
      P a[2], bb[2];
      const uint16_t* src[2];
      uint16_t* dst[2] = {nullptr, nullptr};
      int t[2] = {0, 0};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (row + u * lanes < n_rows) {
          rows_of(row + u * lanes, &src[u], &dst[u], &t[u]);
          a[u].v = *reinterpret_cast<const V*>(src[u] + oa);
          if (turn) bb[u].v = *reinterpret_cast<const V*>(src[u] + ob);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (dst[u] == nullptr) continue;
        if (turn) {
          const float2* cs = s_cs + t[u] * p.r + VEC * col;
          P x, y;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            float va, vb;
            if constexpr (INTER) {  // pair i: elements 2i, 2i + 1 of the 2 VEC
              va = 2 * i < VEC ? a[u].get((2 * i) % VEC) : bb[u].get((2 * i) % VEC);
              vb = 2 * i + 1 < VEC ? a[u].get((2 * i + 1) % VEC) : bb[u].get((2 * i + 1) % VEC);
            } else {
              va = a[u].get(i);
              vb = bb[u].get(i);
            }
            const float2 w = cs[i];
            const float ra = va * w.x - vb * w.y, rb = vb * w.x + va * w.y;
            if constexpr (INTER) {
              if (2 * i < VEC) x.set((2 * i) % VEC, ra); else y.set((2 * i) % VEC, ra);
              if (2 * i + 1 < VEC) x.set((2 * i + 1) % VEC, rb); else y.set((2 * i + 1) % VEC, rb);
            } else {
              x.set(i, ra);
              y.set(i, rb);
            }
          }
          *reinterpret_cast<V*>(dst[u] + oa) = x.v;
          *reinterpret_cast<V*>(dst[u] + ob) = y.v;
        } else {
          *reinterpret_cast<V*>(dst[u] + oa) = a[u].v;
        }
      }
    }
  }
  if constexpr (APPEND) {  // V rows, 8 elements an item
    const int pv = p.D / 8;
    for (int i = threadIdx.x; i < n_tok * p.H_kv * pv; i += kRopeThreads) {
      const int c = i % pv, rh = i / pv;
      const int t = rh / p.H_kv, g = rh - t * p.H_kv;
      if (s_slot[t] < 0) continue;
      const uint16_t* src = static_cast<const uint16_t*>(p.v) + static_cast<int64_t>(tok0 + t) * p.v_stride +
                            g * p.D + 8 * c;
      uint16_t* dst = static_cast<uint16_t*>(p.v_out) + s_slot[t] + g * p.head_stride + 8 * c;
      *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
    }
  }
}

namespace {

template <int VEC, bool INTER, bool BF16>
cudaError_t launch_rope_t(RopeParams p, bool append, dim3 grid, cudaStream_t stream) {
  p.copies = p.copy_rest ? (p.D - 2 * p.r) / VEC : 0;
  if (append) fa_rope_kernel<VEC, INTER, BF16, true><<<grid, kRopeThreads, 0, stream>>>(p);
  else fa_rope_kernel<VEC, INTER, BF16, false><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int VEC>
cudaError_t launch_rope_v(const RopeParams& p, bool bf16, bool append, dim3 grid, cudaStream_t s) {
  if (p.interleaved)
    return bf16 ? launch_rope_t<VEC, true, true>(p, append, grid, s) : launch_rope_t<VEC, true, false>(p, append, grid, s);
  return bf16 ? launch_rope_t<VEC, false, true>(p, append, grid, s) : launch_rope_t<VEC, false, false>(p, append, grid, s);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, bool bf16, bool append, int batch, cudaStream_t stream) {
  const int64_t per_tok = static_cast<int64_t>(p.H + (append ? 2 : 1) * p.H_kv) * p.D;
  int64_t tok = kRopeElems / per_tok;
  p.tok_per_cta = static_cast<int>(tok < 1 ? 1 : (tok > kRopeMaxTok ? kRopeMaxTok : tok));
  const int longest = append ? p.max_len : p.total;
  p.tiles = (longest + p.tok_per_cta - 1) / p.tok_per_cta;
  const int64_t ctas = static_cast<int64_t>(p.tiles) * (append ? batch : 1);
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas));
  const int r = p.r;
  if (r % 8 == 0) return launch_rope_v<8>(p, bf16, append, grid, stream);
  if (r % 4 == 0) return launch_rope_v<4>(p, bf16, append, grid, stream);
  if (r % 2 == 0) return launch_rope_v<2>(p, bf16, append, grid, stream);
  return launch_rope_v<1>(p, bf16, append, grid, stream);
}

}  // namespace fa
