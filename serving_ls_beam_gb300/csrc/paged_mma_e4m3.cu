// The single-token attention over pages of e4m3 codes (the kernel is in ls_paged_mma.cuh).
#include "ls_paged_mma.cuh"

namespace lsb {

cudaError_t launch_paged_mma_e4m3(const PagedParams& p, int dtype, bool by_warp, cudaStream_t stream) {
  return dtype == DT_BF16 ? run_paged_dim<KIND_E4M3, false>(p, dtype, by_warp, stream) : run_paged_dim<KIND_E4M3, true>(p, dtype, by_warp, stream);
}

}  // namespace lsb
