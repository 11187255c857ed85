// The end of a step on a tree of drafted tokens: the branch that the model's own choices
// confirm, and its keys and values appended to the cache of every layer.
//
// Node 0 holds the token chosen by the step before; node i > 0 guesses the token after its
// parent.  The model chose target[n] after node n, so a node is confirmed when its parent is
// and token[i] == target[parent[i]].  All nodes that agree with their parent's choice offer
// themselves to it at once (the least index wins, which takes the first of equal siblings); the
// branch then is a chase along the winners from the root, one shared-memory read a node.
//
// A CTA has one layer of one row, or a part of it where the trees are large and the rows few
// (branches of very different lengths: the longest would otherwise set the time).  Each repeats
// the walk (a few hundred bytes from L2 and that chase), which costs less than a launch for it, and copies its share of the accepted keys and values, 16 bytes per thread where
// the layout allows, eight copies under way per thread.  Nothing of the rejected nodes is read
// or written.  256 trees of 31 nodes (1 to 31 confirmed), 6 layers x 16 heads of 64 elements: 90 MB in
// 25 us, 0.53 of the copy rate; what is left is the chain load - walk - load - store of each CTA
// (128 threads a CTA: 28 us; twice the parts: 28 us).  60 registers a thread: an SM holds four CTAs, and the
// 1536 of this case are two and a half rounds.
#include "ls_device.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

constexpr int kTcThreads = 256;
constexpr int kTcBatch = 8;  // copies under way per thread
static_assert(kAtMaxNodes <= 64 && kTcThreads >= kAtMaxNodes, "a thread per node, masks of 64 bits");

// Units [first, first + stride, ..) of the branch's keys, then its values, to the cache.
template <class U>
__device__ __forceinline__ void append(const CommitParams& p, const int* path, int count, int row, int layer, int len,
                                       int first, int stride) {
  const int per = p.heads * p.vec_units, half = count * per, n = 2 * half;
  const long long slab = (long long)p.max_len * p.vec_units;  // in units
  const long long base = ((long long)layer * p.rows + row) * p.heads * slab + (long long)len * p.vec_units;
  const unsigned char* dk = p.dkey.data + layer * p.dkey_layer + row * p.dkey.row;
  const unsigned char* dv = p.dvalue.data + layer * p.dvalue_layer + row * p.dvalue.row;
  for (int i0 = first; i0 < n; i0 += stride * kTcBatch) {
    U x[kTcBatch];
    U* to[kTcBatch];
#pragma unroll
    for (int k = 0; k < kTcBatch; ++k) {
      const int i = i0 + k * stride;
      to[k] = nullptr;
      if (i < n) {
        const bool val = i >= half;
        const int j = val ? i - half : i, a = p.by_per(j), e = j - a * per, h = p.by_units(e), u = e - h * p.vec_units;
        const unsigned char* from = val ? dv + path[a] * p.dvalue.pos + h * p.dvalue.head : dk + path[a] * p.dkey.pos + h * p.dkey.head;
        x[k] = __ldg(reinterpret_cast<const U*>(from) + u);
        to[k] = reinterpret_cast<U*>(val ? p.cache_value : p.cache_key) + base + h * slab + (long long)a * p.vec_units + u;
      }
    }
#pragma unroll
    for (int k = 0; k < kTcBatch; ++k)
      if (to[k]) *to[k] = x[k];
  }
}

__global__ void __launch_bounds__(kTcThreads) tree_commit_kernel(const CommitParams p) {
  __shared__ int child[kAtMaxNodes], want[kAtMaxNodes], path[kAtMaxNodes];
  __shared__ int s_count;
  const int r = blockIdx.x, layer = blockIdx.y, part = blockIdx.z, tid = threadIdx.x, N = p.nodes;
  const bool lead = layer == 0 && part == 0;  // writes the row's results
  const long long at = (long long)r * N;
  int pi = -2, tok = 0;
  if (tid < N) {
    pi = __ldg(p.parent + at + tid);
    tok = __ldg(p.token + at + tid);
    child[tid] = kAtMaxNodes;
    want[tid] = __ldg(p.target + at + tid);
  }
  const int len = __ldg(p.cache_len + r);
  const bool done = p.finished && p.finished[r];
  __syncthreads();
  if (tid < N && pi >= 0 && pi < tid && tok == want[pi] && tok != p.eos) atomicMin(&child[pi], tid);
  __syncthreads();
  if (tid == 0) {
    const bool bad_len = len < 0 || len > p.max_len;
    const int room = bad_len ? 0 : p.max_len - len;
    int count = 0;
    if (!done && pi == -1 && room > 0) {
      for (int cur = 0; cur < kAtMaxNodes && count < room; cur = child[cur]) path[count++] = cur;
    }
    s_count = count;
    if (lead) {
      const int next = done ? p.eos : count > 0 ? want[path[count - 1]] : __ldg(p.token + at);
      p.out_len[r] = len + count;
      p.out_count[r] = count;
      p.out_token[r] = next;
      if (p.out_finished) p.out_finished[r] = done || (count > 0 && next == p.eos);
      if (p.status && (bad_len || (!done && room == 0) || (!done && pi != -1))) atomicOr(p.status, kDevInternal);
    }
  }
  __syncthreads();
  const int count = s_count;
  if (lead && tid < N) p.out_path[at + tid] = tid < count ? path[tid] : -1;
  if (count == 0 || p.heads == 0) return;
  const int first = part * kTcThreads + tid, stride = (int)gridDim.z * kTcThreads;
  if (p.unit == 16)
    append<uint4>(p, path, count, r, layer, len, first, stride);
  else if (p.unit == 4)
    append<uint32_t>(p, path, count, r, layer, len, first, stride);
  else
    append<uint16_t>(p, path, count, r, layer, len, first, stride);
}

}  // namespace

cudaError_t launch_tree_commit(const CommitParams& p, cudaStream_t stream) {
  // parts of a (row, layer): one batch per thread at most, and not above 16 CTAs per SM, four rounds
  const long long units = 2ll * p.nodes * p.heads * p.vec_units, pairs = (long long)p.rows * p.layers;
  const long long need = (units + kTcThreads * kTcBatch - 1) / (kTcThreads * kTcBatch), room = 2ll * kAtSms * 8 / pairs;
  const long long parts = need < room ? need : room;
  tree_commit_kernel<<<dim3((unsigned)p.rows, (unsigned)p.layers, (unsigned)(parts < 1 ? 1 : parts)), kTcThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace lsb
