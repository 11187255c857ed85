// The end of a step on a tree of drafted tokens: the branch that the model's own choices
// confirm, and its keys and values appended to the cache of every layer.
//
// Node 0 holds the token chosen by the step before; node i > 0 guesses the token after its
// parent.  The model chose target[n] after node n, so a node is confirmed when its parent is
// and token[i] == target[parent[i]].  Parents come before their children, so one pass over the
// candidates in ascending order, taking each whose parent is the branch's last node so far,
// walks the branch and takes the first of equal siblings.
//
// A CTA has one layer of one row.  Each repeats the walk (a few hundred bytes from L2, a loop
// over the candidates only), which costs less than a launch for it, and copies its layer's
// accepted keys and values, 16 bytes per thread where the layout allows.  Nothing of the
// rejected nodes is read or written.
#include "ls_device.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

constexpr int kTcThreads = 128;
static_assert(kAtMaxNodes <= 64 && kTcThreads >= kAtMaxNodes, "a thread per node, masks of 64 bits");

template <class U>
__device__ __forceinline__ void append(unsigned char* cache, const unsigned char* draft, long long node_stride,
                                       long long head_stride, const int* path, int count, int heads, int units,
                                       long long slab, int first, int tid) {
  const int per = heads * units, n = count * per;
#pragma unroll 4
  for (int i = tid; i < n; i += kTcThreads) {
    const int a = i / per, e = i - a * per, h = e / units, u = e - h * units;
    const U x = __ldg(reinterpret_cast<const U*>(draft + path[a] * node_stride + h * head_stride) + u);
    reinterpret_cast<U*>(cache + h * slab)[(long long)(first + a) * units + u] = x;
  }
}

__global__ void __launch_bounds__(kTcThreads) tree_commit_kernel(const CommitParams p) {
  __shared__ int par[kAtMaxNodes], want[kAtMaxNodes], path[kAtMaxNodes];
  __shared__ unsigned fits[kAtMaxNodes / 32];
  __shared__ int s_count;
  const int r = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, N = p.nodes;
  const long long at = (long long)r * N;
  int pi = -2, tok = 0;
  if (tid < N) {
    pi = __ldg(p.parent + at + tid);
    tok = __ldg(p.token + at + tid);
    par[tid] = pi;
    want[tid] = __ldg(p.target + at + tid);
  }
  const int len = __ldg(p.cache_len + r);
  const bool done = p.finished && p.finished[r];
  __syncthreads();
  const bool ok = tid < N && pi >= 0 && pi < tid && tok == want[pi >= 0 && pi < N ? pi : 0] && tok != p.eos;
  const unsigned b = __ballot_sync(~0u, ok);
  if ((tid & 31) == 0 && tid < kAtMaxNodes) fits[tid >> 5] = b;
  __syncthreads();
  if (tid == 0) {
    const bool bad_len = len < 0 || len > p.max_len;
    const int room = bad_len ? 0 : p.max_len - len;
    int count = 0;
    if (!done && par[0] == -1 && room > 0) {
      path[count++] = 0;
      int cur = 0;
      for (int w = 0; w < kAtMaxNodes / 32; ++w) {
        for (unsigned f = fits[w]; f && count < room; f &= f - 1) {
          const int i = w * 32 + __ffs(f) - 1;
          if (par[i] == cur) {
            path[count++] = i;
            cur = i;
          }
        }
      }
    }
    s_count = count;
    if (layer == 0) {
      const int next = done ? p.eos : count > 0 ? want[path[count - 1]] : __ldg(p.token + at);
      p.out_len[r] = len + count;
      p.out_count[r] = count;
      p.out_token[r] = next;
      if (p.out_finished) p.out_finished[r] = done || (count > 0 && next == p.eos);
      if (p.status && (bad_len || (!done && room == 0) || (!done && par[0] != -1))) atomicOr(p.status, kDevInternal);
    }
  }
  __syncthreads();
  const int count = s_count;
  if (layer == 0 && tid < N) p.out_path[at + tid] = tid < count ? path[tid] : -1;
  if (count == 0) return;
  const long long slab = (long long)p.max_len * p.vec_units * p.unit;
  const long long base = ((long long)layer * p.rows + r) * p.heads * slab;
  const unsigned char* dk = p.dkey.data + layer * p.dkey_layer + r * p.dkey.row;
  const unsigned char* dv = p.dvalue.data + layer * p.dvalue_layer + r * p.dvalue.row;
  if (p.unit == 16) {
    append<uint4>(p.cache_key + base, dk, p.dkey.pos, p.dkey.head, path, count, p.heads, p.vec_units, slab, len, tid);
    append<uint4>(p.cache_value + base, dv, p.dvalue.pos, p.dvalue.head, path, count, p.heads, p.vec_units, slab, len, tid);
  } else if (p.unit == 4) {
    append<uint32_t>(p.cache_key + base, dk, p.dkey.pos, p.dkey.head, path, count, p.heads, p.vec_units, slab, len, tid);
    append<uint32_t>(p.cache_value + base, dv, p.dvalue.pos, p.dvalue.head, path, count, p.heads, p.vec_units, slab, len, tid);
  } else {
    append<uint16_t>(p.cache_key + base, dk, p.dkey.pos, p.dkey.head, path, count, p.heads, p.vec_units, slab, len, tid);
    append<uint16_t>(p.cache_value + base, dv, p.dvalue.pos, p.dvalue.head, path, count, p.heads, p.vec_units, slab, len, tid);
  }
}

}  // namespace

cudaError_t launch_tree_commit(const CommitParams& p, cudaStream_t stream) {
  tree_commit_kernel<<<dim3((unsigned)p.rows, (unsigned)p.layers), kTcThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace lsb
