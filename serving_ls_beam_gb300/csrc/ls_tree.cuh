// Device helpers of a tree of drafted tokens, and the addresses of an attention problem.
#pragma once

#include <stdint.h>

#include "ls_attend.h"
#include "ls_internal.h"

namespace lsb {

// What the nodes of one row's tree see, in shared memory (tree_bytes of it, 8-byte aligned).
struct TreeSeen {
  unsigned long long* mask;  // bit j: the node sees node j (0: an empty place)
  int* up;
};
__host__ __device__ inline int tree_bytes(int nodes) { return nodes * 12; }
__device__ __forceinline__ TreeSeen tree_at(void* shared, int nodes) {
  TreeSeen t;
  t.mask = static_cast<unsigned long long*>(shared);
  t.up = reinterpret_cast<int*>(t.mask + nodes);
  return t;
}

// Fills t for a tree of `nodes` nodes with `n` threads (thread `tid`); `sync` orders those
// threads' shared memory.  Pointer doubling: after round r a node's mask holds its 2^r nearest
// ancestors, so a chain of 64 takes six rounds.  A node whose parent is below -1 is an empty
// place, one whose parent is not before it is invalid (returned true) and treated the same,
// and so are the nodes under either.
template <class Parent, class Sync>
__device__ __forceinline__ bool tree_seen_from(const TreeSeen& t, Parent parent, int nodes, int tid, int n, Sync sync) {
  bool bad = false;
  for (int i = tid; i < nodes; i += n) {
    const int p = parent(i);
    bad |= p >= i;
    const bool there = p >= -1 && p < i;
    t.mask[i] = there ? 1ull << i : 0ull;
    t.up[i] = there ? p : -2;
  }
  sync();
  for (int reach = 1; reach < nodes; reach <<= 1) {
    unsigned long long m[kAtMaxNodes / 32];
    int u[kAtMaxNodes / 32];
#pragma unroll
    for (int r = 0; r < kAtMaxNodes / 32; ++r) {
      const int i = tid + r * n;
      if (i >= nodes || i < 0) continue;
      m[r] = t.mask[i];
      u[r] = t.up[i];
      if (u[r] >= 0) {
        const int a = u[r];
        u[r] = t.up[a];
        m[r] = u[r] == -2 ? 0ull : m[r] | t.mask[a];
      }
    }
    sync();
#pragma unroll
    for (int r = 0; r < kAtMaxNodes / 32; ++r) {
      const int i = tid + r * n;
      if (i >= nodes) continue;
      t.mask[i] = m[r];
      t.up[i] = u[r];
    }
    sync();
  }
  return bad;
}

template <class Sync>
__device__ __forceinline__ bool tree_seen(const TreeSeen& t, const int32_t* parent, int nodes, int tid, int n, Sync sync) {
  return tree_seen_from(t, [&](int i) { return __ldg(parent + i); }, nodes, tid, n, sync);
}

// The eight 16-bit values of d: infinite and NaN ones become zero; true if there were any.  (An
// exponent of all ones carries out of its field when one is added to it.)
template <bool BF>
__device__ __forceinline__ bool clear_non_finite(uint4& d) {
  constexpr uint32_t E = BF ? 0x7f807f80u : 0x7c007c00u, U = BF ? 0x00800080u : 0x04000400u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&d);
  const uint32_t any = ((w[0] & E) + U) | ((w[1] & E) + U) | ((w[2] & E) + U) | ((w[3] & E) + U);
  if (!(any & 0x80008000u)) return false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = ((w[i] & E) + U) & 0x80008000u;
    w[i] &= ~((c & 0x8000u ? 0xffffu : 0u) | (c & 0x80000000u ? 0xffff0000u : 0u));
  }
  return true;
}

// The 16-bit kernels' weights are 2^(score - reference); the reference lies this far under a row's maximum,
// for the sums and the weighted values alike, so that it cancels.  f16 has 2^-24 as its smallest number:
// with weights of up to 2^15 (2^8 of a maximum that has not been raised yet) it keeps what is 2^-31 of the largest
// weight or more, where weights of up to 1 would lose a long flat tail under one large score at 2^-25.
// (One key at weight 1 and 131000 at 2^-25.1: -0.9966 for -0.9927.)  bf16 has the exponents of f32.
template <bool BF>
constexpr float kAtLift = BF ? 0.0f : 7.0f;

// acc + f * x of a part with the sum l: nothing of an empty part, and an infinite or NaN x as
// it is (f may have underflowed).
__device__ __forceinline__ float add_part(float acc, float f, float x, float l) {
  const float y = isfinite(x) ? f * x : x;
  return l != 0.0f ? acc + y : acc;
}

// The keys of a row, clamped to its places; out of range sets the status word (by `report`).
__device__ __forceinline__ int row_keys(const AttendParams& p, int r, bool report) {
  const int n = __ldg(p.len + r);
  const int c = min(max(n, 0), p.max_len);
  if (report && n != c) atomicOr(p.status, kDevInternal);
  return c;
}

// Query i of problem (r, h).
__device__ __forceinline__ long long query_offset(const AttendParams& p, const AtView& v, int r, int h, int i) {
  const int t = p.by_group(i), g = i - t * p.group;
  const int b = p.by_q_len(t), pos = t - b * p.q_len;
  return ((long long)r * p.beams + b) * v.row + (long long)pos * v.pos + (long long)(h * p.group + g) * v.head;
}

}  // namespace lsb
