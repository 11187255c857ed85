// Attention over a row's keys on the CUDA cores, for tensors whose layout the other kernels cannot
// read (a head size or stride that breaks 16-byte alignment).
//
//   o_i = sum_n exp(s_in - max) v_n / sum_n exp(s_in - max),   s_in = scale q_i . k_n
//
// in one pass over the keys with the running maximum and sum of the softmax (Milakov and
// Gimelshein, "Online normalizer calculation for softmax", 2018), everything in f32.
//
// A CTA of four warps has MQ queries of one problem and one part of its keys; its warps take
// blocks of 32 keys in turn.  A block's keys go to shared memory as f32 and lane n forms the
// MQ products of key n with the queries (read as broadcasts); the values are read from global
// memory, where a warp reads a whole value vector at a time, lane d holding the outputs'
// elements d, d + 32, ...  The warps' results are merged in shared memory at the end.
//
// It is the kernel that takes anything, bound by its shared-memory reads and by the values' latency:
// the single-token step of 1024 beams of 64 positions takes 423 us here (0.08 of the copy rate), 42
// in the kernel that such calls go to.
#include "ls_device.cuh"
#include "ls_dtype.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

constexpr int kSiWarps = 4;
constexpr int kSiThreads = kSiWarps * 32;

// floats of a staged key: a multiple of 4, an odd number of 16-byte vectors, so the 32 lanes'
// 16-byte reads of 32 keys have no bank conflicts
__host__ __device__ inline int simt_pitch(int dim) {
  const int v = (dim + 3) / 4;
  return 4 * (v | 1);
}
inline size_t simt_smem(int dim, int mq) {
  return (size_t)(mq + kSiWarps * 32) * simt_pitch(dim) * 4;
}

template <int DT>
__device__ __forceinline__ void store_elem(unsigned char* at, float x) {
  if constexpr (DT == DT_F32)
    *reinterpret_cast<float*>(at) = x;
  else if constexpr (DT == DT_F16)
    *reinterpret_cast<__half*>(at) = __float2half_rn(x);
  else
    *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(x);
}

// The warp's copy of `n` key vectors (stride `pos` bytes) to shared memory as f32.
template <int DT>
__device__ __forceinline__ void stage_keys(float* ks, int pitch, const unsigned char* src, long long pos, int n, int dim,
                                           bool vec, int lane) {
  constexpr int E = Traits<DT>::kVec, B = Traits<DT>::kBytes;
  if (vec) {  // whole 16-byte vectors
    const int nv = dim / E;
#pragma unroll 8
    for (int i = lane; i < n * nv; i += 32) {
      const int k = i / nv, c = i - k * nv;
      const uint4 d = __ldg(reinterpret_cast<const uint4*>(src + k * pos) + c);
      float x[E];
      unpack<DT>(d, x);
      float4* to = reinterpret_cast<float4*>(ks + k * pitch + c * E);
#pragma unroll
      for (int j = 0; j < E / 4; ++j) to[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
    }
  } else {
    for (int k = 0; k < n; ++k)
      for (int d = lane; d < pitch; d += 32) ks[k * pitch + d] = d < dim ? load_elem<DT>(src + k * pos + d * B) : 0.0f;
  }
}

template <int DT, int MQ, int ND>
__global__ void __launch_bounds__(kSiThreads) attend_simt_kernel(const AttendParams p) {
  constexpr int B = Traits<DT>::kBytes;
  extern __shared__ float4 si_smem[];
  __shared__ unsigned long long tree_raw[kAtMaxNodes * 12 / 8];
  const TreeSeen tree = tree_at(tree_raw, kAtMaxNodes);
  __shared__ float wm[kSiWarps][MQ], wl[kSiWarps][MQ];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pitch = simt_pitch(p.dim);
  float* qs = reinterpret_cast<float*>(si_smem);
  float* ks = qs + MQ * pitch + warp * 32 * pitch;

  const int it = (int)blockIdx.x, ia = p.by_split(it), split = it - ia * p.splits, ib = p.by_tile(ia);
  const int i0 = (ia - ib * p.m_tiles) * MQ, r = p.by_head(ib), h = ib - r * p.kv_heads;
  const int nq = min(MQ, p.m - i0);
  const int len = row_keys(p, r, tid == 0);

  for (int j = 0; j < MQ; ++j) {
    const unsigned char* q = p.q.data + query_offset(p, p.q, r, h, i0 + min(j, nq - 1));
    for (int d = tid; d < pitch; d += kSiThreads) qs[j * pitch + d] = d < p.dim ? load_elem<DT>(q + d * B) : 0.0f;
  }
  if (p.nodes) {
    if (tree_seen(tree, p.parent + (long long)r * p.nodes, p.nodes, tid, kSiThreads, [] { __syncthreads(); }))
      atomicOr(p.status, kDevInternal);
  }
  __syncthreads();

  // blocks [0, nb) of the row's keys, then the drafted ones; this CTA has [b_lo, b_hi)
  const int nb = (len + 31) / 32, nbt = nb + (p.nodes + 31) / 32;
  const int per = (nbt + p.splits - 1) / p.splits;
  const int b_lo = min(split * per, nbt), b_hi = min(b_lo + per, nbt);
  bool alive[MQ];
#pragma unroll
  for (int j = 0; j < MQ; ++j) alive[j] = j < nq && (!p.nodes || tree.mask[p.by_group(i0 + j)] != 0);

  float mx[MQ], sum[MQ], o[MQ][ND];
#pragma unroll
  for (int j = 0; j < MQ; ++j) {
    mx[j] = -INFINITY;
    sum[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < ND; ++i) o[j][i] = 0.0f;
  }
  const bool vec = p.dim % Traits<DT>::kVec == 0 && ((p.key.row | p.key.pos | p.key.head) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(p.key.data) & 15) == 0;
  const bool dvec = p.nodes && p.dim % Traits<DT>::kVec == 0 && ((p.dkey.row | p.dkey.pos | p.dkey.head) & 15) == 0 &&
                    (reinterpret_cast<uintptr_t>(p.dkey.data) & 15) == 0;
  for (int b = b_lo + warp; b < b_hi; b += kSiWarps) {
    const bool draft = b >= nb;
    const int n0 = draft ? (b - nb) * 32 : b * 32;
    const int n = min(32, (draft ? p.nodes : len) - n0);
    const AtView& kv = draft ? p.dkey : p.key;
    const AtView& vv = draft ? p.dvalue : p.value;
    __syncwarp();
    stage_keys<DT>(ks, pitch, kv.data + (long long)r * kv.row + (long long)h * kv.head + (long long)n0 * kv.pos, kv.pos, n,
                   p.dim, draft ? dvec : vec, lane);
    __syncwarp();
    float s[MQ];
#pragma unroll
    for (int j = 0; j < MQ; ++j) s[j] = 0.0f;
    const float4* kr = reinterpret_cast<const float4*>(ks + lane * pitch);
    if (lane < n) {
#pragma unroll 4
      for (int c = 0; c < (p.dim + 3) / 4; ++c) {
        const float4 k4 = kr[c];
#pragma unroll
        for (int j = 0; j < MQ; ++j) {
          const float4 q4 = reinterpret_cast<const float4*>(qs + j * pitch)[c];
          s[j] = fmaf(k4.x, q4.x, s[j]);
          s[j] = fmaf(k4.y, q4.y, s[j]);
          s[j] = fmaf(k4.z, q4.z, s[j]);
          s[j] = fmaf(k4.w, q4.w, s[j]);
        }
      }
    }
    unsigned seen[MQ];  // draft blocks: the keys each query sees
    float pr[MQ];
#pragma unroll
    for (int j = 0; j < MQ; ++j) {
      seen[j] = draft && alive[j] ? (unsigned)(tree.mask[p.by_group(i0 + j)] >> n0) : (alive[j] ? ~0u : 0u);
      const bool ok = lane < n && ((seen[j] >> lane) & 1u);
      const float t = ok ? s[j] * p.scale_log2 : -INFINITY;
      float bm = t;
#pragma unroll
      for (int x = 16; x; x >>= 1) bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, x));
      const float mn = fmaxf(mx[j], bm);
      const float base = mn == -INFINITY ? 0.0f : mn;
      const float f = fast_exp2(mx[j] - base);
      pr[j] = ok ? fast_exp2(t - base) : 0.0f;
      sum[j] = sum[j] * f + pr[j];  // this lane's share, added up at the end
#pragma unroll
      for (int i = 0; i < ND; ++i) o[j][i] *= f;
      mx[j] = mn;
    }
    const unsigned char* vr = vv.data + (long long)r * vv.row + (long long)h * vv.head + (long long)n0 * vv.pos + lane * B;
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      float v[ND];
#pragma unroll
      for (int i = 0; i < ND; ++i) v[i] = lane + 32 * i < p.dim ? load_elem<DT>(vr + k * vv.pos + 32 * i * B) : 0.0f;
#pragma unroll
      for (int j = 0; j < MQ; ++j) {
        const float w = __shfl_sync(~0u, pr[j], k);
        // a value that the query does not see is left out, not multiplied by 0 (it may be
        // anything)
        const bool use = (seen[j] >> k) & 1u;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[j][i] = use ? fmaf(w, v[i], o[j][i]) : o[j][i];
      }
    }
  }

  // the warps' results, one after the other, in the first warp's order
#pragma unroll
  for (int j = 0; j < MQ; ++j) {
    float t = sum[j];
#pragma unroll
    for (int x = 16; x; x >>= 1) t += __shfl_xor_sync(~0u, t, x);
    sum[j] = t;
    if (lane == 0) {
      wm[warp][j] = mx[j];
      wl[warp][j] = t;
    }
  }
  __syncthreads();
  float* acc = reinterpret_cast<float*>(si_smem) + MQ * pitch;  // [warp][MQ][ND * 32]
#pragma unroll
  for (int j = 0; j < MQ; ++j)
#pragma unroll
    for (int i = 0; i < ND; ++i) acc[(warp * MQ + j) * ND * 32 + i * 32 + lane] = o[j][i];
  __syncthreads();
  for (int e = tid; e < nq * p.dim; e += kSiThreads) {
    const int j = e / p.dim, d = e - j * p.dim;
    float M = wm[0][j];
#pragma unroll
    for (int w = 1; w < kSiWarps; ++w) M = fmaxf(M, wm[w][j]);
    const float base = M == -INFINITY ? 0.0f : M;
    float L = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < kSiWarps; ++w) {
      const float f = fast_exp2(wm[w][j] - base);
      L = fmaf(f, wl[w][j], L);
      O = add_part(O, f, acc[(w * MQ + j) * ND * 32 + d], wl[w][j]);
    }
    if (p.splits == 1) {
      store_elem<DT>(p.out.data + query_offset(p, p.out, r, h, i0 + j) + d * B, L == 0.0f ? 0.0f : O / L);
    } else {
      const long long row = (((long long)r * p.kv_heads + h) * p.m + i0 + j) * p.splits + split;
      p.part_o[row * p.dim + d] = O;
      if (d == 0) p.part_ml[row] = make_float2(M, L);
    }
  }
}

// The parts of each query joined, a CTA to a query: its warps take the parts in turn, a lane four
// elements (two of them for head sizes above 128), and add up in the warps' order.  What counts is
// that all of a query's parts are under way at once: with a warp to a query and the parts one after
// the other, 19 parts of 512 queries took 21 us instead of 6 (alone, cold).
// With up to four parts a warp takes a query by itself (EACH): 32 problems of 700 queries, two parts, the whole
// call 327 -> 313 us; 6656 queries of two parts 54 -> 51 us.
constexpr int kJoinWarps = 4;
template <int DT, bool EACH>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttendParams p) {
  constexpr int B = Traits<DT>::kBytes, VEC = kAtMaxDim / 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = EACH ? (int)blockIdx.x * kJoinWarps + warp : (int)blockIdx.x;
  if (EACH && w >= p.rows * p.kv_heads * p.m) return;
  const int pb = p.by_m(w), i = w - pb * p.m, r = p.by_head(pb), h = pb - r * p.kv_heads;
  const float2* ml = p.part_ml + (long long)w * p.splits;
  const float* po = p.part_o + (long long)w * p.splits * p.dim;
  grid_dependency_wait();
  float M = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, x));
  const float base = M == -INFINITY ? 0.0f : M;
  float L = 0.0f, o[VEC][4];
#pragma unroll
  for (int c = 0; c < VEC; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.0f;
  const bool four = p.dim % 4 == 0;
#pragma unroll 4
  for (int s = EACH ? 0 : warp; s < p.splits; s += EACH ? 1 : kJoinWarps) {
    const float2 e = ml[s];
    const float f = fast_exp2(e.x - base);
    L = fmaf(f, e.y, L);
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const int d = c * 128 + lane * 4;
      const float* at = po + (long long)s * p.dim + d;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (four) {
        if (d < p.dim) v = *reinterpret_cast<const float4*>(at);
      } else {
        if (d < p.dim) v.x = at[0];
        if (d + 1 < p.dim) v.y = at[1];
        if (d + 2 < p.dim) v.z = at[2];
        if (d + 3 < p.dim) v.w = at[3];
      }
      o[c][0] = add_part(o[c][0], f, v.x, e.y);
      o[c][1] = add_part(o[c][1], f, v.y, e.y);
      o[c][2] = add_part(o[c][2], f, v.z, e.y);
      o[c][3] = add_part(o[c][3], f, v.w, e.y);
    }
  }
  unsigned char* out = p.out.data + query_offset(p, p.out, r, h, i);
  if constexpr (EACH) {
#pragma unroll
    for (int c = 0; c < VEC; ++c)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int d = c * 128 + lane * 4 + x;
        if (d < p.dim) store_elem<DT>(out + d * B, L == 0.0f ? 0.0f : o[c][x] / L);
      }
  } else {
    __shared__ float acc[kJoinWarps][kAtMaxDim], sums[kJoinWarps];
#pragma unroll
    for (int c = 0; c < VEC; ++c)
      *reinterpret_cast<float4*>(&acc[warp][c * 128 + lane * 4]) = make_float4(o[c][0], o[c][1], o[c][2], o[c][3]);
    if (lane == 0) sums[warp] = L;
    __syncthreads();
    float total = 0.0f;
#pragma unroll
    for (int x = 0; x < kJoinWarps; ++x) total += sums[x];
    for (int d = threadIdx.x; d < p.dim; d += kJoinWarps * 32) {
      float y = 0.0f;
#pragma unroll
      for (int x = 0; x < kJoinWarps; ++x) y += acc[x][d];
      store_elem<DT>(out + d * B, total == 0.0f ? 0.0f : y / total);
    }
  }
}

template <int DT, int MQ, int ND>
cudaError_t run_simt(const AttendParams& p, cudaStream_t stream) {
  auto bytes = [](int dim) {
    const size_t acc = (size_t)MQ * simt_pitch(dim) * 4 + (size_t)kSiWarps * MQ * ND * 32 * 4;
    return simt_smem(dim, MQ) > acc ? simt_smem(dim, MQ) : acc;
  };
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(attend_simt_kernel<DT, MQ, ND>, (int)bytes(ND * 32), allowed);
  if (e != cudaSuccess) return e;
  attend_simt_kernel<DT, MQ, ND><<<(unsigned)p.items, kSiThreads, bytes(p.dim), stream>>>(p);
  return cudaGetLastError();
}

template <int DT, int MQ>
cudaError_t run_simt_dim(const AttendParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return run_simt<DT, MQ, 2>(p, stream);
  if (p.dim <= 128) return run_simt<DT, MQ, 4>(p, stream);
  return run_simt<DT, MQ, 8>(p, stream);
}

}  // namespace

int attend_simt_queries(int dtype, int m) {
  if (dtype != DT_F32) return 4;
  return m == 1 ? 1 : m <= 4 ? 4 : 8;
}

cudaError_t launch_attend_simt(const AttendParams& p, int dtype, cudaStream_t stream) {
  if (dtype == DT_F16) return run_simt_dim<DT_F16, 4>(p, stream);
  if (dtype == DT_BF16) return run_simt_dim<DT_BF16, 4>(p, stream);
  switch (attend_simt_queries(dtype, p.m)) {
    case 1: return run_simt_dim<DT_F32, 1>(p, stream);
    case 4: return run_simt_dim<DT_F32, 4>(p, stream);
    default: return run_simt_dim<DT_F32, 8>(p, stream);
  }
}

template <int DT>
static cudaError_t run_join(const AttendParams& p, cudaStream_t stream) {
  const long long queries = (long long)p.rows * p.kv_heads * p.m;
  const bool each = p.splits <= 4;
  PdlLaunch l(dim3((unsigned)(each ? (queries + kJoinWarps - 1) / kJoinWarps : queries)), dim3(kJoinWarps * 32), 0, stream);
  return each ? cudaLaunchKernelEx(&l.cfg, attend_join_kernel<DT, true>, p) : cudaLaunchKernelEx(&l.cfg, attend_join_kernel<DT, false>, p);
}

cudaError_t launch_attend_join(const AttendParams& p, int dtype, cudaStream_t stream) {
  if (dtype == DT_F32) return run_join<DT_F32>(p, stream);
  return dtype == DT_F16 ? run_join<DT_F16>(p, stream) : run_join<DT_BF16>(p, stream);
}

}  // namespace lsb
