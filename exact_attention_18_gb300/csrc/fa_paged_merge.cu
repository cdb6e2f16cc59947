// Joins the partials of the units that the paged-attention kernels cut between
// CTAs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kernel_common.cuh"
#include "fa_paged.cuh"

namespace fa {
using namespace ptx;

// Joins the partials of the units that were cut between CTAs:
// L = log2 sum_s 2^(L_s), O = sum_s 2^(L_s - L) O_s, in CTA order.  CTA
// (c, y) takes rows y, y + gridDim.y, ... of the unit whose first blocks CTA c
// of the main kernel computed.  D / 4 threads span a row; the other threads
// split the partials, summed in a fixed order at the end.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) fa_paged_merge_kernel(const PagedMergeParams p) {
  using elem_t = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int kLanes = D / 4, kGroups = 128 / kLanes;
  __shared__ float4 s_o[kGroups][kLanes];
  __shared__ float s_w[kGroups];
  griddep_wait();
  const int first = blockIdx.x;
  const PagedParts q = p.parts[blockIdx.z];
  if (first >= q.grid) return;
  const int4 d = q.desc[first];
  const int n_rows = d.y * p.G;
  if (n_rows == 0) return;
  const int x = threadIdx.x % kLanes, y = threadIdx.x / kLanes;
  const int parts = d.w - first + 1;
  for (int row = blockIdx.y; row < n_rows; row += gridDim.y) {
    // Partial s: slot 2 first + 1 for the first CTA, 2 c for the later ones.
    auto slot = [&](int s) -> int64_t { return static_cast<int64_t>(s == 0 ? 2 * first + 1 : 2 * (first + s)) * q.rows + row; };
    float mx = -INFINITY;
    for (int s = 0; s < parts; ++s) mx = fmaxf(mx, q.lse_part[slot(s)]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float wsum = 0.f;
    if (mx != -INFINITY) {
      for (int s = y; s < parts; s += kGroups) {
        const int64_t at = slot(s);
        const float wt = exp2f(q.lse_part[at] - mx);
        const float4 v = *reinterpret_cast<const float4*>(q.o_part + at * D + 4 * x);
        wsum += wt;
        o.x += wt * v.x; o.y += wt * v.y; o.z += wt * v.z; o.w += wt * v.w;
      }
    }
    s_o[y][x] = o;
    if (x == 0) s_w[y] = wsum;
    __syncthreads();
    if (y == 0) {
      float total = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < kGroups; ++k) {
        const float4 v = s_o[k][x];
        total += s_w[k];
        a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
      }
      const bool seen = mx != -INFINITY;
      const float inv = seen ? 1.f / total : 0.f;
      const int tok = d.x + row / p.G, head = d.z * p.G + row % p.G;
      elem_t* orow = static_cast<elem_t*>(p.o) + (static_cast<int64_t>(tok) * p.H + head) * D;
      *reinterpret_cast<uint2*>(orow + 4 * x) =
          make_uint2(pack2<BF16>(a.x * inv, a.y * inv), pack2<BF16>(a.z * inv, a.w * inv));
      if (x == 0)
        p.lse[static_cast<int64_t>(head) * p.total + tok] =
            seen ? (mx + log2f(total)) * 0.69314718055994530942f : -INFINITY;
    }
    __syncthreads();
  }
}

namespace {

template <int D, bool BF16>
cudaError_t launch_paged_merge_t(const PagedMergeParams& p, int grid, int sets, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 16, sets);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_paged_merge_kernel<D, BF16>, p);
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
