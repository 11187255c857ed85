// The single-token attention over 16-bit pages (the kernel is in ls_paged_mma.cuh), and what it goes by.
#include "ls_paged_mma.cuh"

namespace lsb {

int paged_mma_queries(int dim, int group) { return group <= 8 || dim > 128 ? 8 : 16; }
int paged_mma_ctas(int dim, int group) { return dim <= 64 ? (group <= 8 ? 4 : 3) : dim <= 128 && group <= 8 ? 3 : 2; }

// Whether a warp by itself is a worker: where the items are so many that the warps of a CTA would merge them
// one after the other.  By warps and by CTAs, us: rows of 200 to 1000 positions, 16 heads of 64 f16, 4 rows 11.7 and 10.1,
// 16 19.9 and 20.7, 32 (from here on by warps) 25.0 and 26.1, 256 106 and 122; of 500 to 4000 positions, 8 key heads of 128
// with 4 queries, e4m3 32 rows 49 and 42, 64 (from here on) 72 and 71, 128 122 and 126, 256 219 and 238; bf16 32 rows 63
// and 55, 64 105 and 98, 256 352 and 349.
bool paged_mma_warps(const PagedParams& p) {
  return 5ll * p.rows * p.per_row >= (long long)kPgWarps * kAtSms * paged_mma_ctas(p.dim, p.group);
}

cudaError_t launch_paged_mma(const PagedParams& p, int dtype, int cache, bool by_warp, cudaStream_t stream) {
  if (cache == LS_DTYPE_F16) return run_paged_dim<KIND_F16, true>(p, dtype, by_warp, stream);
  if (cache == LS_DTYPE_BF16) return run_paged_dim<KIND_BF16, true>(p, dtype, by_warp, stream);
  return cache == LS_DTYPE_E4M3 ? launch_paged_mma_e4m3(p, dtype, by_warp, stream) : launch_paged_mma_i8(p, dtype, by_warp, stream);
}

}  // namespace lsb
