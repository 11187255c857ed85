// The single-token attention over 16-bit pages (the kernel is in ls_paged_mma.cuh), and what it goes by.
#include "ls_paged_mma.cuh"

namespace lsb {

int paged_mma_queries(int dim, int group) { return group <= 8 || dim > 128 ? 8 : 16; }
int paged_mma_ctas(int dim, int group) { return dim <= 64 ? (group <= 8 ? 4 : 3) : dim <= 128 && group <= 8 ? 3 : 2; }

// Whether a warp by itself is a worker: where the items are so many that the warps of a CTA would merge them
// one after the other.
bool paged_mma_warps(const PagedParams& p) {
  return 5ll * p.rows * p.per_row >= (long long)kPgWarps * kAtSms * paged_mma_ctas(p.dim, p.group);
}

cudaError_t launch_paged_mma(const PagedParams& p, int dtype, int cache, bool by_warp, cudaStream_t stream) {
  if (cache == LS_DTYPE_F16) return run_paged_dim<KIND_F16, true>(p, dtype, by_warp, stream);
  if (cache == LS_DTYPE_BF16) return run_paged_dim<KIND_BF16, true>(p, dtype, by_warp, stream);
  return cache == LS_DTYPE_E4M3 ? launch_paged_mma_e4m3(p, dtype, by_warp, stream) : launch_paged_mma_i8(p, dtype, by_warp, stream);
}

}  // namespace lsb
