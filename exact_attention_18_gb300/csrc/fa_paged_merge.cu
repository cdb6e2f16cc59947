// Joins the partials of the units that the paged-attention kernels cut between
// CTAs (comment at the kernel).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kernel_common.cuh"
#include "fa_paged.cuh"

namespace fa {
using namespace ptx;

// L = log2 sum_s 2^(L_s), O = sum_s 2^(L_s - L) O_s, in CTA order: fixed by
// the lengths alone.  Slice c of the grid joins the unit whose first blocks CTA
// c of the main kernel computed; D / 4 threads span a row.  A CTA takes several
// rows at once; only a unit in many parts (a long context, few rows) has them
// one by one, the parts split over the CTA and summed in a fixed order.  The
// partials come from L2, so what bounds the kernel is its launch and the chain
// of reads: descriptor, then all of a row's parts at once.  Decoding over 4
// contexts of 131072 keys takes 161 us with a loop over the parts and 150 with
// their reads in flight together (the main kernel alone: 150).
// A part whose L is NaN (NaN scores) makes the row NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

constexpr int kMergeThreads = 128;
constexpr int kMergeFew = 24;  // parts up to which a CTA takes several rows at once
constexpr int kMergeBatch = 8;  // parts whose reads are in flight together

template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeThreads) fa_paged_merge_kernel(const PagedMergeParams p) {
  using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int kLanes = D / 4, kGroups = kMergeThreads / kLanes;
  __shared__ float4 s_o[kGroups][kLanes];
  __shared__ float s_w[kGroups];
  griddep_wait();
  griddep_launch_dependents();
  const int first = blockIdx.x;
  if (p.go && threadIdx.x == 0 && (blockIdx.x | blockIdx.y | blockIdx.z) == 0) *p.go = 0;
  // (an index into the parameters would put a copy of them on the stack)
  const bool z = blockIdx.z != 0;
  const PagedParts q{z ? p.parts[1].o_part : p.parts[0].o_part, z ? p.parts[1].lse_part : p.parts[0].lse_part,
                     z ? p.parts[1].desc : p.parts[0].desc,     z ? p.parts[1].rows : p.parts[0].rows,
                     z ? p.parts[1].grid : p.parts[0].grid,     z ? p.parts[1].by_chunk : p.parts[0].by_chunk};
  if (first >= q.grid) return;
  const int4 d = q.desc[first];
  const int n_rows = d.y * p.G;
  const int x = threadIdx.x % kLanes, y = threadIdx.x / kLanes;
  const int parts = d.w - first + 1;
  // Row `row` of part s: slot 2 first + 1 for the first CTA, 2 c for the later ones.
  auto at = [&](int s, int row) -> int64_t {
    return static_cast<int64_t>(s == 0 ? 2 * first + 1 : 2 * (first + s)) * q.rows + row;
  };
  auto add = [&](float4& o, float w, const float4 v) {
    o.x += w * v.x; o.y += w * v.y; o.z += w * v.z; o.w += w * v.w;
  };
  if (q.by_chunk) {
    // Lanes span rows, as the partials lie; a warp takes 32 rows x 16 columns
    // at a time (whole 32-byte sectors of the output).
    constexpr int kStrips = D / 16;
    const int lane = threadIdx.x & 31;
    const int tasks = (n_rows + 31) / 32 * kStrips;
    for (int task = static_cast<int>(blockIdx.y) * (kMergeThreads / 32) + static_cast<int>(threadIdx.x >> 5);
         task < tasks; task += gridDim.y * (kMergeThreads / 32)) {
      const int row = task / kStrips * 32 + lane, strip = task % kStrips;
      if (row >= n_rows) continue;
      float mx = -INFINITY, total = 0.f;
      float4 o[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kBatch = 3;  // units of the tile kernel are in two or three parts as a rule
      for (int s0 = 0; s0 < parts; s0 += kBatch) {
        float l[kBatch];
        float4 v[kBatch][4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          l[k] = -INFINITY;
          if (s0 + k < parts) {
            l[k] = q.lse_part[at(s0 + k, row)];
            const float4* src = reinterpret_cast<const float4*>(q.o_part + at(s0 + k, 0) * D) + 4 * strip * q.rows + row;
#pragma unroll
            for (int c = 0; c < 4; ++c) v[k][c] = src[c * q.rows];
          }
        }
        float m_new = mx;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) m_new = max_nan(m_new, l[k]);
        if (m_new == -INFINITY) continue;
        const float keep = exp2f(mx - m_new);
        mx = m_new;
        total *= keep;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = make_float4(o[c].x * keep, o[c].y * keep, o[c].z * keep, o[c].w * keep);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (l[k] != -INFINITY) {
            const float w = exp2f(l[k] - mx);
            total += w;
#pragma unroll
            for (int c = 0; c < 4; ++c) add(o[c], w, v[k][c]);
          }
        }
      }
      const bool seen = mx != -INFINITY;
      const float inv = seen ? 1.f / total : 0.f;
      const int tok = d.x + row / p.G, head = d.z * p.G + row % p.G;
      uint4* orow = reinterpret_cast<uint4*>(static_cast<elem_t*>(p.o) +
                                             (static_cast<int64_t>(tok) * p.H + head) * D + 16 * strip);
#pragma unroll
      for (int c = 0; c < 4; c += 2)
        orow[c / 2] = make_uint4(pack2<BF16>(o[c].x * inv, o[c].y * inv), pack2<BF16>(o[c].z * inv, o[c].w * inv),
                                 pack2<BF16>(o[c + 1].x * inv, o[c + 1].y * inv),
                                 pack2<BF16>(o[c + 1].z * inv, o[c + 1].w * inv));
      if (strip == 0)
        p.lse[static_cast<int64_t>(head) * p.total + tok] =
            seen ? (mx + log2f(total)) * 0.69314718055994530942f : -INFINITY;
    }
    return;
  }
  auto store = [&](int row, float4 a, float total, float mx) {
    const bool seen = mx != -INFINITY;
    const float inv = seen ? 1.f / total : 0.f;
    const int tok = d.x + row / p.G, head = d.z * p.G + row % p.G;
    elem_t* orow = static_cast<elem_t*>(p.o) + (static_cast<int64_t>(tok) * p.H + head) * D;
    *reinterpret_cast<uint2*>(orow + 4 * x) =
        make_uint2(pack2<BF16>(a.x * inv, a.y * inv), pack2<BF16>(a.z * inv, a.w * inv));
    if (x == 0)
      p.lse[static_cast<int64_t>(head) * p.total + tok] =
          seen ? (mx + log2f(total)) * 0.69314718055994530942f : -INFINITY;
  };
  if (parts <= kMergeFew) {
    for (int row = static_cast<int>(blockIdx.y) * kGroups + y; row < n_rows; row += gridDim.y * kGroups) {
      float mx = -INFINITY, total = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s0 = 0; s0 < parts; s0 += kMergeBatch) {
        float l[kMergeBatch];
        float4 v[kMergeBatch];
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
          l[k] = -INFINITY;
          if (s0 + k < parts) {
            l[k] = q.lse_part[at(s0 + k, row)];
            v[k] = *reinterpret_cast<const float4*>(q.o_part + at(s0 + k, row) * D + 4 * x);
          }
        }
        float m_new = mx;
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) m_new = max_nan(m_new, l[k]);
        if (m_new == -INFINITY) continue;
        const float keep = exp2f(mx - m_new);
        mx = m_new;
        total *= keep;
        o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
          if (l[k] != -INFINITY) {
            const float w = exp2f(l[k] - mx);
            total += w;
            add(o, w, v[k]);
          }
        }
      }
      store(row, o, total, mx);
    }
    return;
  }
  for (int row = blockIdx.y; row < n_rows; row += gridDim.y) {
    float mx = -INFINITY;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) mx = max_nan(mx, q.lse_part[at(s, row)]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float wsum = 0.f;
    if (mx != -INFINITY) {
#pragma unroll 4
      for (int s = y; s < parts; s += kGroups) {
        const float w = exp2f(q.lse_part[at(s, row)] - mx);
        wsum += w;
        add(o, w, *reinterpret_cast<const float4*>(q.o_part + at(s, row) * D + 4 * x));
      }
    }
    s_o[y][x] = o;
    if (x == 0) s_w[y] = wsum;
    __syncthreads();
    if (y == 0) {
      float total = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < kGroups; ++k) {
        total += s_w[k];
        add(a, 1.f, s_o[k][x]);
      }
      store(row, a, total, mx);
    }
    __syncthreads();
  }
}

namespace {

template <int D, bool BF16>
cudaError_t launch_paged_merge_t(const PagedMergeParams& p, int grid, int sets, cudaStream_t stream) {
  // Slices: two rounds of a CTA's strips (one is up to 3 % slower for calls of
  // chunks, where it makes thousands of CTAs), one of its rows.
  int slices = 1;
  for (int z = 0; z < sets; ++z) {
    const int rows = p.parts[z].rows, per = kMergeThreads / (D / 4);
    const int n = p.parts[z].by_chunk ? ((rows + 31) / 32 * (D / 16) + 7) / 8 : (rows + per - 1) / per;
    if (n > slices) slices = n;
  }
  return launch_dependent(fa_paged_merge_kernel<D, BF16>, dim3(grid, slices, sets),
                          kMergeThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_paged_merge(int D, bool bf16, const PagedMergeParams& p, int grid, int sets, cudaStream_t s) {
  switch (D) {
    case 16: return bf16 ? launch_paged_merge_t<16, true>(p, grid, sets, s) : launch_paged_merge_t<16, false>(p, grid, sets, s);
    case 32: return bf16 ? launch_paged_merge_t<32, true>(p, grid, sets, s) : launch_paged_merge_t<32, false>(p, grid, sets, s);
    case 64: return bf16 ? launch_paged_merge_t<64, true>(p, grid, sets, s) : launch_paged_merge_t<64, false>(p, grid, sets, s);
    case 128: return bf16 ? launch_paged_merge_t<128, true>(p, grid, sets, s) : launch_paged_merge_t<128, false>(p, grid, sets, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
