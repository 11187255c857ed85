// Internal definitions of sampling with filters (sample_filter.cu, its entry point in api_paged.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace lsb {

constexpr int kSfThreads = 256;
constexpr int kSfMaxCluster = 8;
constexpr int kSfMaxUnits = 2048;  // units of a CTA's share of a row

struct FilterParams {
  const unsigned char* logits;
  long long row_bytes;       // from row to row
  const float* bias;         // may be null, as all up to min_p
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* out_token;
  float* out_logprob;        // may be null
  uint32_t* status;          // may be null
  int rows, vocab;
  int cluster;               // CTAs of a row
  int unit_vecs;             // 16-byte vectors per lane of a unit
  int units;                 // of a CTA
  int shift;                 // weights are sums of 2^-(29 + shift) of the largest
  int resident;              // a CTA's share of the row stays in shared memory
  int thread_vecs;           // vectors of a thread
  uint32_t thread_magic;     // division by them
  int thread_shift;
};
cudaError_t launch_sample_filter(const FilterParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_sample_filter_f16(const FilterParams& p, cudaStream_t stream);
cudaError_t launch_sample_filter_bf16(const FilterParams& p, cudaStream_t stream);

}  // namespace lsb
