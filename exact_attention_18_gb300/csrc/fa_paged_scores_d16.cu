// The paged-cache attention kernels with modified scores and drafted trees for head
// dimension 16.
#include "fa_paged_kernel.cuh"
#include "fa_paged_tile_kernel.cuh"

namespace fa {

cudaError_t launch_paged_scored_d16(int N, bool tile, bool bf16, const CUtensorMap& tq, const CUtensorMap& tk,
                                   const CUtensorMap& tv, const PagedScoredParams& p, int grid, cudaStream_t stream) {
  if (!tile) return launch_paged_n<16, PagedScoredParams>(N, bf16, tq, tk, tv, p, grid, stream);
  return bf16 ? launch_paged_tile_t<16, true, PagedScoredParams>(tq, tk, tv, p, grid, stream)
              : launch_paged_tile_t<16, false, PagedScoredParams>(tq, tk, tv, p, grid, stream);
}

}  // namespace fa
