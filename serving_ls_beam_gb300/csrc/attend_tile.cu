// Attention of many queries over a row's keys in f32, on the CUDA cores (the tensor cores have no
// product of f32's precision).
//
//   S = scale Q K^T,  P = 2^(S - max),  O = O * correction + P V,  out = O / sum P
//
// in one pass over the keys with the running maximum and sum (Milakov and Gimelshein, 2018), all in
// f32: the weights are not rounded.
//
// Both products are matrix products, so a CTA takes BM queries and goes over the keys in tiles of BN.
// Its 128 threads form a grid of 8 x 16: thread (ty, tx) has the scores of queries ty + 8 i and keys
// tx + 16 j, and of the sums the same queries' elements 2 tx + 32 n.  A vector of four elements that a
// thread reads from shared memory serves TK (a query's) or TQ (a key's) scores, in packed f32
// multiply-adds over even and odd elements.  The weights of a query are written and read by the same half
// warp, so they cross shared memory without a barrier.  Keys and values have one buffer each: the
// next keys are on their way during the values' product and the next values during the scores'.
// Rows are padded by 16 bytes: the 16 keys (and the two queries) of a load lie in distinct banks.
//
// The drafted tokens follow the row's keys without a gap.
//
// What bounds it: the multiply-adds and the latencies between them with 16 to 20 warps per SM.  4 x 1000
// queries x 8 heads of 64 over 900 to 1000 keys: 214 us, 36 TFLOP/s; 64 trees of 13 nodes x 8 heads of
// 64, 100 to 500 positions: 51 us with the join; 1024 problems of 12 queries, head 256, 300 to 700 positions: 445 us,
// 1.1 GB.  What mattered: CTAs per SM (8 queries per thread, two thirds of the loads and half the CTAs,
// takes 288 us on the first of these as it was then, 4 queries 257) and one running address per whole
// tile (257 -> 214 us).  16 queries to a tile where there are no more: 60 -> 54 us on the second.
#include "ls_device.cuh"
#include "ls_dtype.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

constexpr int kAlThreads = 128;

template <int DP, int TQ, int TK>
struct TileShape {
  static constexpr int BM = 8 * TQ, BN = 16 * TK;
  static constexpr int ROW = DP + 4, PROW = BN + 4;  // floats
  static constexpr int K = BM * ROW, V = K + BN * ROW, P = V + BN * DP, FLOATS = P + BM * PROW;
  static constexpr int BYTES = FLOATS * 4;
  static constexpr int FIT = 232448 / (BYTES + 2048), CTAS = FIT < 5 ? FIT : 5;  // per SM
};

template <int DP, int TQ, int TK>
__global__ void __launch_bounds__(kAlThreads, TileShape<DP, TQ, TK>::CTAS) attend_tile_kernel(const AttendParams p) {
  using T = TileShape<DP, TQ, TK>;
  constexpr int BM = T::BM, BN = T::BN, ND = DP / 32, VI = (DP + 63) / 64;
  extern __shared__ float4 al_smem[];
  __shared__ unsigned long long tree_raw[kAtMaxNodes * 12 / 8];
  float* qs = reinterpret_cast<float*>(al_smem);
  float* ks = qs + T::K;
  float* vs = qs + T::V;
  float* ps = qs + T::P;
  const TreeSeen tree = tree_at(tree_raw, kAtMaxNodes);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int it = (int)blockIdx.x, ia = p.by_split(it), split = it - ia * p.splits, ib = p.by_tile(ia);
  const int i0 = (ia - ib * p.m_tiles) * BM, r = p.by_head(ib), h = ib - r * p.kv_heads;
  const int nq = min(BM, p.m - i0);
  const int len = row_keys(p, r, tid == 0);
  const int total = len + p.nodes, nbt = (total + BN - 1) / BN, per = (nbt + p.splits - 1) / p.splits;
  const int lo = min(split * per, nbt), hi = min(lo + per, nbt);
  const int vecs = p.dim / 4;

  const unsigned char* kb = p.key.data + (long long)r * p.key.row + (long long)h * p.key.head;
  const unsigned char* vb = p.value.data + (long long)r * p.value.row + (long long)h * p.value.head;
  const unsigned char* dkb = p.dkey.data + (long long)r * p.dkey.row + (long long)h * p.dkey.head;
  const unsigned char* dvb = p.dvalue.data + (long long)r * p.dvalue.row + (long long)h * p.dvalue.head;
  // tile b of the keys or values, 16 threads to a row; zeros past the row's end
  auto fetch = [&](int b, float* to, int row, const unsigned char* cache, long long pos, const unsigned char* draft,
                   long long dpos) {
    if (b < hi && b * BN + BN <= len) {
      const unsigned char* at = cache + (b * BN + ty) * pos + tx * 16;
      const uint32_t dst = smem_addr(to + ty * row + tx * 4);
#pragma unroll
      for (int k = 0; k < BN / 8; ++k, at += 8 * pos)
#pragma unroll
        for (int i = 0; i < VI; ++i)
          if (tx + 16 * i < vecs) cp_async16_fill(dst + k * 32 * row + i * 256, at + i * 256, 16);
    } else if (b < hi) {
      const int n = (min(BN, total - b * BN) + 15) & ~15;  // the rows that the products read
      for (int k = ty; k < n; k += 8) {
        const int j = b * BN + k;
        const unsigned char* at = j < len ? cache + j * pos : j < total ? draft + (j - len) * dpos : p.q.data;
        const int stride = j < total ? 16 : 0;
        const uint32_t dst = smem_addr(to + k * row);
        for (int v = tx; v < vecs; v += 16) cp_async16_fill(dst + v * 16, at + v * stride, stride);
      }
    }
    cp_async_commit();
  };
  for (int i = ty; i < BM; i += 8) {
    const unsigned char* q = p.q.data + query_offset(p, p.q, r, h, i0 + min(i, nq - 1));
    const uint32_t dst = smem_addr(qs + i * T::ROW);
    for (int v = tx; v < vecs; v += 16) cp_async16_fill(dst + v * 16, q + v * 16, 16);
  }
  fetch(lo, ks, T::ROW, kb, p.key.pos, dkb, p.dkey.pos);
  fetch(lo, vs, DP, vb, p.value.pos, dvb, p.dvalue.pos);
  if (p.nodes) {
    if (tree_seen(tree, p.parent + (long long)r * p.nodes, p.nodes, tid, kAlThreads, [] { __syncthreads(); }))
      atomicOr(p.status, kDevInternal);
  }
  __syncthreads();
  unsigned alive = 0;  // bit i: query ty + 8 i (the last one's copies behind it) sees something
#pragma unroll
  for (int i = 0; i < TQ; ++i)
    if (!p.nodes || tree.mask[p.by_group(i0 + min(ty + 8 * i, nq - 1))] != 0) alive |= 1u << i;
  const bool all_alive = __all_sync(~0u, alive == (1u << TQ) - 1u);

  float m[TQ], l[TQ];
  float2 o[TQ][ND];
#pragma unroll
  for (int i = 0; i < TQ; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int n = 0; n < ND; ++n) o[i][n] = make_float2(0.0f, 0.0f);
  }
  const float* qrow = qs + ty * T::ROW;
  float* prow = ps + ty * T::PROW;

  for (int b = lo; b < hi; ++b) {
    const int n0 = b * BN, left = min(BN, total - n0);
    const bool edge = n0 + BN > len;
    cp_async_wait<1>();
    __syncthreads();  // the keys (and queries) are there
    // the scores against the tile's first 16 J keys, their maximum and weights
    auto scores = [&](auto groups) {
      constexpr int J = decltype(groups)::value;
      float2 s2[TQ][J];
#pragma unroll
      for (int i = 0; i < TQ; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) s2[i][j] = make_float2(0.0f, 0.0f);
#pragma unroll 2
      for (int v = 0; v < vecs; ++v) {
        float4 k4[J];
#pragma unroll
        for (int j = 0; j < J; ++j) k4[j] = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * T::ROW + 4 * v);
#pragma unroll
        for (int i = 0; i < TQ; ++i) {
          const float4 q4 = *reinterpret_cast<const float4*>(qrow + 8 * i * T::ROW + 4 * v);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            s2[i][j] = __ffma2_rn(make_float2(q4.x, q4.y), make_float2(k4[j].x, k4[j].y), s2[i][j]);
            s2[i][j] = __ffma2_rn(make_float2(q4.z, q4.w), make_float2(k4[j].z, k4[j].w), s2[i][j]);
          }
        }
      }
      __syncthreads();  // all threads are done with the keys
      fetch(b + 1, ks, T::ROW, kb, p.key.pos, dkb, p.dkey.pos);
      float f[TQ];
      bool grown = false;
#pragma unroll
      for (int i = 0; i < TQ; ++i) {
        float s[J], bm = -INFINITY;
#pragma unroll
        for (int j = 0; j < J; ++j) s[j] = (s2[i][j].x + s2[i][j].y) * p.scale_log2;
        if (edge || !all_alive) {
          const bool live = (alive >> i) & 1u;
          const unsigned long long sees = edge && p.nodes && live ? tree.mask[p.by_group(i0 + min(ty + 8 * i, nq - 1))] : 0ull;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const int key = n0 + tx + 16 * j;
            if (!(live && key < total && (key < len || ((sees >> (key - len)) & 1ull)))) s[j] = -INFINITY;
          }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) bm = fmaxf(bm, s[j]);
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, x));
        const float mn = fmaxf(m[i], bm), sub = mn == -INFINITY ? 0.0f : mn;
        f[i] = fast_exp2(m[i] - sub);
        grown |= mn > m[i];
        m[i] = mn;
        l[i] *= f[i];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float w = fast_exp2(s[j] - sub);
          l[i] += w;
          prow[8 * i * T::PROW + tx + 16 * j] = w;
        }
      }
      if (__any_sync(~0u, grown)) {
#pragma unroll
        for (int i = 0; i < TQ; ++i)
#pragma unroll
          for (int n = 0; n < ND; ++n) o[i][n] = __fmul2_rn(o[i][n], make_float2(f[i], f[i]));
      }
    };
    if (left <= 16)
      scores(std::integral_constant<int, 1>{});
    else if (left <= 32 || TK == 2)
      scores(std::integral_constant<int, 2>{});
    else
      scores(std::integral_constant<int, TK>{});
    cp_async_wait<1>();
    __syncthreads();  // the values are there
    const float* vcol = vs + 2 * tx;
    if (edge && p.nodes) {
      // a drafted value that the query does not see may be anything: left out, not times 0
      for (int k = 0; k < left; ++k) {
        float2 v[ND];
#pragma unroll
        for (int n = 0; n < ND; ++n) v[n] = *reinterpret_cast<const float2*>(vcol + k * DP + 32 * n);
#pragma unroll
        for (int i = 0; i < TQ; ++i) {
          const float w = prow[8 * i * T::PROW + k];
#pragma unroll
          for (int n = 0; n < ND; ++n) {
            const float2 y = __ffma2_rn(make_float2(w, w), v[n], o[i][n]);
            o[i][n].x = w != 0.0f ? y.x : o[i][n].x;
            o[i][n].y = w != 0.0f ? y.y : o[i][n].y;
          }
        }
      }
    } else {
      for (int k = 0; k < left; k += 4) {
        float4 w4[TQ];
#pragma unroll
        for (int i = 0; i < TQ; ++i) w4[i] = *reinterpret_cast<const float4*>(prow + 8 * i * T::PROW + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 v[ND];
#pragma unroll
          for (int n = 0; n < ND; ++n) v[n] = *reinterpret_cast<const float2*>(vcol + (k + e) * DP + 32 * n);
#pragma unroll
          for (int i = 0; i < TQ; ++i) {
            const float w = e == 0 ? w4[i].x : e == 1 ? w4[i].y : e == 2 ? w4[i].z : w4[i].w;
#pragma unroll
            for (int n = 0; n < ND; ++n) o[i][n] = __ffma2_rn(make_float2(w, w), v[n], o[i][n]);
          }
        }
      }
    }
    __syncthreads();  // all threads are done with the values
    fetch(b + 1, vs, DP, vb, p.value.pos, dvb, p.dvalue.pos);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < TQ; ++i) {
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) l[i] += __shfl_xor_sync(~0u, l[i], x);
    const int q = ty + 8 * i;
    if (q >= nq) continue;
    const bool zero = l[i] == 0.0f;
    float* to;
    float inv = 1.0f;
    if (p.splits == 1) {
      inv = zero ? 0.0f : 1.0f / l[i];
      to = reinterpret_cast<float*>(p.out.data + query_offset(p, p.out, r, h, i0 + q));
    } else {
      const long long pr = (((long long)r * p.kv_heads + h) * p.m + i0 + q) * p.splits + split;
      to = p.part_o + pr * p.dim;
      if (tx == 0) p.part_ml[pr] = make_float2(m[i], l[i]);
    }
#pragma unroll
    for (int n = 0; n < ND; ++n) {
      const int d = 2 * tx + 32 * n;
      if (d < p.dim)
        *reinterpret_cast<float2*>(to + d) = zero ? make_float2(0.0f, 0.0f) : make_float2(o[i][n].x * inv, o[i][n].y * inv);
    }
  }
}

template <int DP, int TQ, int TK>
cudaError_t run_tile(const AttendParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(attend_tile_kernel<DP, TQ, TK>, TileShape<DP, TQ, TK>::BYTES, allowed);
  if (e != cudaSuccess) return e;
  attend_tile_kernel<DP, TQ, TK><<<(unsigned)p.items, kAlThreads, TileShape<DP, TQ, TK>::BYTES, stream>>>(p);
  return cudaGetLastError();
}

template <int DP, int TK>
cudaError_t run_tile_queries(const AttendParams& p, cudaStream_t stream) {
  return p.m_step == 16 ? run_tile<DP, 2, TK>(p, stream) : run_tile<DP, 4, TK>(p, stream);
}
template <int DP, int TK>
int tile_ctas(int queries) {
  return queries == 16 ? TileShape<DP, 2, TK>::CTAS : TileShape<DP, 4, TK>::CTAS;
}

}  // namespace

int attend_tile_queries(int m) { return m <= 16 ? 16 : 32; }

int attend_tile_ctas(int dim, int m) {
  const int q = attend_tile_queries(m);
  if (dim <= 32) return tile_ctas<32, 4>(q);
  if (dim <= 64) return tile_ctas<64, 4>(q);
  if (dim <= 96) return tile_ctas<96, 4>(q);
  return dim <= 128 ? tile_ctas<128, 2>(q) : tile_ctas<256, 2>(q);
}

cudaError_t launch_attend_tile(const AttendParams& p, cudaStream_t stream) {
  if (p.dim <= 32) return run_tile_queries<32, 4>(p, stream);
  if (p.dim <= 64) return run_tile_queries<64, 4>(p, stream);
  if (p.dim <= 96) return run_tile_queries<96, 4>(p, stream);
  if (p.dim <= 128) return run_tile_queries<128, 2>(p, stream);
  return run_tile_queries<256, 2>(p, stream);
}

}  // namespace lsb
