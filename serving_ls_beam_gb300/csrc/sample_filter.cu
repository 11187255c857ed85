// Sampling with filters of f32 logits (the kernel is in ls_filter.cuh), and its launch by type.
#include "ls_filter.cuh"

namespace lsb {

cudaError_t launch_sample_filter(const FilterParams& p, int dtype, cudaStream_t stream) {
  if (dtype == DT_F16) return launch_sample_filter_f16(p, stream);
  if (dtype == DT_BF16) return launch_sample_filter_bf16(p, stream);
  return p.bias ? plan_filter<DT_F32, true>(p, stream) : plan_filter<DT_F32, false>(p, stream);
}

}  // namespace lsb
