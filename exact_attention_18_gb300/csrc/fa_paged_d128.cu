// The paged-cache attention kernels for head dimension 128.
#include "fa_paged_kernel.cuh"
#include "fa_paged_tile_kernel.cuh"

namespace fa {

cudaError_t launch_paged_d128(int N, bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, int grid, cudaStream_t stream) {
  return launch_paged_n<128, PagedParams>(N, bf16, tq, tk, tv, p, grid, stream);
}

cudaError_t launch_paged_tile_d128(bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const PagedParams& p, int grid, cudaStream_t stream) {
  return bf16 ? launch_paged_tile_t<128, true, PagedParams>(tq, tk, tv, p, grid, stream)
              : launch_paged_tile_t<128, false, PagedParams>(tq, tk, tv, p, grid, stream);
}

}  // namespace fa
