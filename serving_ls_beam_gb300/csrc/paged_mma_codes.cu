// The single-token attention over pages of 8-bit codes (the kernel is in ls_paged_mma.cuh).
#include "ls_paged_mma.cuh"

namespace lsb {

cudaError_t launch_paged_mma_codes(const PagedParams& p, int dtype, int cache, bool by_warp, cudaStream_t stream) {
  return cache == LS_DTYPE_E4M3 ? run_paged_dim<KIND_E4M3>(p, dtype, by_warp, stream)
                                : run_paged_dim<KIND_I8>(p, dtype, by_warp, stream);
}

}  // namespace lsb
