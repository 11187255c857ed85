// Sampling with filters of bf16 logits (the kernel is in ls_filter.cuh).
#include "ls_filter.cuh"

namespace lsb {

cudaError_t launch_sample_filter_bf16(const FilterParams& p, cudaStream_t stream) {
  return p.bias ? plan_filter<DT_BF16, true>(p, stream) : plan_filter<DT_BF16, false>(p, stream);
}

}  // namespace lsb
