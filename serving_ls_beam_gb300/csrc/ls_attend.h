// Internal definitions of the decoder's attention (cross attention and the draft tree's
// attention) and of the tree's commit, shared by the host entry points (api_attend.cu) and
// the kernels.  Nothing here is part of the public interface (include/ls_beam.h).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ls_beam.h"
#include "ls_internal.h"

namespace lsb {

constexpr int kAtMaxDim = 256;   // largest head size
constexpr int kAtMaxNodes = LS_MAX_NODES;
// positions of a row: the kernels add its drafted tokens and a block of up to 128 keys in 32 bits
constexpr int kAtMaxKeys = INT32_MAX - 1023;
constexpr int kAtSms = 152;

// Division of 0 <= n < 2^31 by a number known on the host (Granlund and Montgomery, 1994).
struct AtDivisor {
  uint32_t magic;
  int shift;
  void set(int d) { make_divisor((uint32_t)d, &magic, &shift); }
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int n) const { return (int)((__umulhi((uint32_t)n, magic) + (uint32_t)n) >> shift); }
#endif
};

// A tensor [row, pos, head, head_dim] by its byte strides (head_dim contiguous).
struct AtView {
  unsigned char* data;
  long long row, pos, head;
};

// One attention call.  The queries that read the same keys are one problem: the key / value
// row `r` and key head `h`, with m = tokens * group queries (token t = beam * q_len + pos,
// query i = t * group + its head within the group).
struct AttendParams {
  AtView q, out;          // [rows * beams, q_len, kv_heads * group, dim]
  AtView key, value;      // [rows, max_len, kv_heads, dim]
  AtView dkey, dvalue;    // [rows, nodes, kv_heads, dim] drafted tokens (nodes == 0: none)
  const int32_t* len;     // [rows] keys of each row
  const int32_t* parent;  // [rows, nodes]
  uint32_t* status;
  float scale_log2;       // scale * log2(e): the softmax runs in powers of two
  int rows, beams, q_len, kv_heads, group, dim, max_len, nodes;
  int tokens;             // beams * q_len
  int m;                  // tokens * group
  int m_step;             // queries per item
  int m_tiles;            // ceil(m / m_step)
  int warps;              // attend_step.cu, attend_mma.cu: warps per item (1 or 4)
  int splits;             // parts of a row's keys (each a CTA's); > 1: partial results
  float* part_o;          // [problem, m, split, dim] f32
  float2* part_ml;        // [problem, m, split]: maximum (log2 units) and sum
  long long items;        // rows * kv_heads * m_tiles * splits
  // item = ((row * kv_heads + head) * m_tiles + tile) * splits + split; query = token * group + head
  AtDivisor by_split, by_tile, by_head, by_group, by_q_len, by_m;
  long long spin_limit_ns;
  int negate;             // tensor-core kernels: scale_log2 is its absolute value, the sign goes into the queries
  // keys shared by all rows or heads (stride 0): their tensor maps have one row or head
  int kv_row_one, kv_head_one;
  int q_tma;              // attend_tc.cu: the queries' tensor map is there
};

// Partial results may take this many (query, split) rows of dim + 2 floats: the plan keeps
// its splits within it, so the workspace depends on the queries and the head size alone.
__host__ __device__ inline long long attend_part_rows(int m) { return 1024ll * (m < 80 ? m : 80); }

struct CommitParams {
  unsigned char* cache_key;
  unsigned char* cache_value;
  AtView dkey, dvalue;      // [layer][row, node, head, dim]
  long long dkey_layer, dvalue_layer;
  const int32_t* cache_len;
  const int32_t* parent;
  const int32_t* token;
  const int32_t* target;
  const uint8_t* finished;  // may be null
  int32_t* out_len;
  int32_t* out_path;
  int32_t* out_count;
  int32_t* out_token;
  uint8_t* out_finished;    // may be null
  uint32_t* status;         // may be null
  int layers, rows, nodes, heads, max_len, eos;
  int vec_units;            // copy units per head vector
  int unit;                 // bytes of a copy unit
  AtDivisor by_per, by_units;  // by heads * vec_units, by vec_units
};

// Raises a kernel's dynamic shared-memory limit once per device (`done`: a bit per device).
template <class Kernel>
inline cudaError_t allow_shared(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// CTAs of a kernel that an SM holds at once (at least 1); `known` keeps the last answer, its shared
// memory in the upper and the number in the lower half.
template <class Kernel>
inline cudaError_t resident_ctas(Kernel kernel, int threads, int bytes, std::atomic<uint64_t>& known, int* ctas) {
  const uint64_t k = known.load(std::memory_order_relaxed);
  if ((uint32_t)k != 0 && (k >> 32) == (uint64_t)bytes) {
    *ctas = (int)(uint32_t)k;
    return cudaSuccess;
  }
  int n = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, bytes);
  if (e != cudaSuccess) return e;
  *ctas = n < 1 ? 1 : n;
  known.store((uint64_t)bytes << 32 | (uint32_t)*ctas, std::memory_order_relaxed);
  return cudaSuccess;
}

cudaError_t launch_attend_simt(const AttendParams& p, int dtype, cudaStream_t stream);
int attend_simt_queries(int dtype, int m);  // queries per CTA
// f32, every stride and address a multiple of 16 bytes
cudaError_t launch_attend_step(const AttendParams& p, cudaStream_t stream);
int attend_step_queries(int dim, int m);  // queries per item
// f32, every stride and address a multiple of 16 bytes
cudaError_t launch_attend_tile(const AttendParams& p, cudaStream_t stream);
int attend_tile_queries(int m);  // queries per CTA
int attend_tile_ctas(int dim, int m);     // CTAs that an SM holds
// f16 / bf16, every stride and address a multiple of 16 bytes
cudaError_t launch_attend_mma(const AttendParams& p, int dtype, cudaStream_t stream);
int attend_mma_queries(int dim, int m);  // queries per item
// f16 / bf16, head size up to kAtTcDim, every stride and address a multiple of 16 bytes; maps: key,
// value, drafted key, drafted value, queries
constexpr int kAtTcDim = 128, kAtTcSlot = 128, kAtTcBox = 64;  // an item has one or two slots of queries
cudaError_t launch_attend_tc(const CUtensorMap (&maps)[5], const AttendParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_attend_join(const AttendParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_tree_commit(const CommitParams& p, cudaStream_t stream);

// Shared with api.cu.
bool pointers_reachable(const void* const* ptrs, int n);  // nulls are skipped
long long wait_limit_ns();
// LS_BEAM_DEBUG's choice of the attention kernel: 0 = the plan's, else one of these
constexpr int kAtForceSimt = 1, kAtForceMma = 2, kAtForceTc = 3;
struct AttendDebug {
  int kernel, warps, splits;
};
AttendDebug attend_debug();
bool maps_describe(const AttendParams& p);  // encode_keys can succeed
// encode_queries: tensor map of the queries [row, key head, token, group, dim] in boxes of 64 elements
// of `queries` queries in their order; false where one stride per dimension does not describe it.
// encode_attend: tensor map of a 16-bit tensor [row, head, pos, dim] by byte strides, in boxes of 64 elements by
// `box` positions (one swizzle row of 128 bytes each); reads past an extent return zeros.
// The tensor maps of the keys and the values in boxes of `box` keys; false where a map cannot
// describe them.
bool encode_keys(CUtensorMap* maps, const AttendParams& p, int dtype, int box);
bool encode_queries(CUtensorMap* map, const AttendParams& p, int dtype, int queries);
bool encode_attend(CUtensorMap* map, const AtView& v, int dtype, int dim, int pos, int heads, int rows, int box);
ls_status report_cuda(cudaError_t e);

}  // namespace lsb
