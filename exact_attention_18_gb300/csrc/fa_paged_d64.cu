// The paged-cache attention kernels for head dimension 64.
#include "fa_paged_kernel.cuh"

namespace fa {

cudaError_t launch_paged_d64(int N, bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, int grid, cudaStream_t stream) {
  return launch_paged_n<64>(N, bf16, tq, tk, tv, p, grid, stream);
}

}  // namespace fa
