// Attention over a row's keys in f32, one to eight queries at a time, on the CUDA cores.  What
// counts is how many bytes are under way and how few instructions a key takes.
//
//   s_n = (scale q) . k_n,  o = sum_n 2^(s_n - max) v_n / sum_n 2^(s_n - max)
//
// in one pass with the running maximum and sum (Milakov and Gimelshein, 2018), all in f32: the
// weights are not rounded.
//
// Keys and values go straight from memory into registers, 16 bytes per lane and load: LPK lanes
// hold one vector (above 128 elements two halves of it), so a load instruction covers 32 / LPK keys, and
// a block is 8 such loads of keys and 8 of values, 8 KB under way per warp.  The keys' registers are loaded again as soon as
// the block's scores are formed, the values' when its sums are.  The 8 dot products of a lane
// group are reduced together, each exchange halving the products that a lane still holds (7
// exchanges instead of 24), which leaves every lane with the score of its own key: one
// exponential per key, not one per lane.  One and two queries keep four CTAs per SM (512 rows of 64
// positions 47 -> 42 us); with four queries the same cap spills and costs a third.  The drafted tokens follow the row's keys without a gap.
//
// What bounds it: bytes under way for one query (512 rows x 16 heads of 64 elements, 40 to 63
// positions: 222 MB in 42 us, 0.78 of the measured copy rate), instructions and registers for four
// (256 x 16 heads, 24 to 128 states: 167 MB in 55 us, 0.45) and eight.  Heads of 256: 64 rows x 16 heads,
// one query, 300 to 700 positions: 1.05 GB in 172 us, 0.90.
//
// A warp takes whole problems in turn (AttendParams::warps 1), or the four warps of a CTA take
// the blocks of one (part of a) problem in turn and merge through shared memory (4).
#include "ls_device.cuh"
#include "ls_dtype.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

constexpr int kAsWarps = 4;
constexpr int kAsThreads = kAsWarps * 32;
constexpr int kAsLoads = 8;  // loads of keys (and of values) per block

__device__ __forceinline__ uint4 load_stream(const unsigned char* p) {
  uint4 d;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(d.x), "=r"(d.y), "=r"(d.z), "=r"(d.w) : "l"(p));
  return d;
}

__device__ __forceinline__ uint4 pack_vec(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// The N values (8 or 4) of each lane summed over the lanes that differ in the bits below LPK: afterwards
// lane l holds the sum of value (l & 1) << 2 | (l & 2) | (l >> 2 & 1), of four (l & 1) << 1 | (l >> 1 & 1).
template <int LPK, int N>
__device__ __forceinline__ float reduce_values(const float (&v)[N], int lane) {
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = v[i];
#pragma unroll
  for (int x = 1, left = N / 2; left; x <<= 1, left >>= 1) {
    const bool hi = lane & x;
#pragma unroll
    for (int i = 0; i < left; ++i) {
      const float keep = hi ? a[i + left] : a[i], give = hi ? a[i] : a[i + left];
      a[i] = keep + __shfl_xor_sync(~0u, give, x);
    }
  }
#pragma unroll
  for (int x = N; x < LPK; x <<= 1) a[0] += __shfl_xor_sync(~0u, a[0], x);
  return a[0];
}

template <int LPK, int V, int MQ>
__global__ void __launch_bounds__(kAsThreads, MQ * V <= 2 ? 4 : 1) attend_step_kernel(const AttendParams p) {
  constexpr int DT = DT_F32, E = 4, EV = E * V, ES = 4, U = kAsLoads / V, KPL = 32 / LPK, KB = U * KPL;
  constexpr int STEP = LPK * E;  // elements from one of a lane's vectors to its next
  __shared__ unsigned long long trees[kAsWarps][kAtMaxNodes * 12 / 8];
  __shared__ float wm[kAsWarps][MQ], wl[kAsWarps][MQ];
  __shared__ float acc[kAsWarps][MQ][STEP * V + 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LPK, gk = lane / LPK;
  const int W = p.warps, wi = W == 1 ? 0 : warp;
  bool cv[V];  // this lane holds a part of the vectors
#pragma unroll
  for (int v = 0; v < V; ++v) cv[v] = c + LPK * v < p.dim / E;
  const int my_u = U == 8 ? (lane & 1) << 2 | (lane & 2) | (lane >> 2 & 1) : (lane & 1) << 1 | (lane >> 1 & 1);
  const TreeSeen tree = tree_at(trees[warp], kAtMaxNodes);
  // (unsigned: an item's number plus the stride, each below 2^31, may pass it)
  const uint32_t items = (uint32_t)p.items, stride = W == 1 ? gridDim.x * kAsWarps : gridDim.x;
  uint32_t it = W == 1 ? blockIdx.x * kAsWarps + warp : blockIdx.x;
  int next_len = it < items ? __ldg(p.len + p.by_head(p.by_tile(p.by_split(it)))) : 0;
  for (; it < items; it += stride) {
    const int ia = p.by_split(it), split = (int)it - ia * p.splits, ib = p.by_tile(ia);
    const int i0 = (ia - ib * p.m_tiles) * MQ, r = p.by_head(ib), h = ib - r * p.kv_heads;
    const int nq = min(MQ, p.m - i0);
    const int len = min(max(next_len, 0), p.max_len);
    if (len != next_len && lane == 0) atomicOr(p.status, kDevInternal);
    if (it + stride < items) next_len = __ldg(p.len + p.by_head(p.by_tile(p.by_split(it + stride))));
    const int total = len + p.nodes, nbt = (total + KB - 1) / KB, per = (nbt + p.splits - 1) / p.splits;
    const int lo = min(split * per, nbt), hi = min(lo + per, nbt);
    int b = lo + wi;

    const unsigned char* kb = p.key.data + (long long)r * p.key.row + (long long)h * p.key.head + c * 16;
    const unsigned char* vb = p.value.data + (long long)r * p.value.row + (long long)h * p.value.head + c * 16;
    const unsigned char* dkb = p.dkey.data + (long long)r * p.dkey.row + (long long)h * p.dkey.head + c * 16;
    const unsigned char* dvb = p.dvalue.data + (long long)r * p.dvalue.row + (long long)h * p.dvalue.head + c * 16;
    auto fetch = [&](uint4(&d)[U][V], int blk, const unsigned char* cache, uint32_t pos, const unsigned char* draft,
                     long long dpos) {
      const int j0 = blk * KB + gk;
      if (blk * KB + KB <= len) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int v = 0; v < V; ++v)
            d[u][v] = cv[v] ? load_stream(cache + (unsigned long long)(uint32_t)(j0 + u * KPL) * pos + v * STEP * ES)
                            : make_uint4(0u, 0u, 0u, 0u);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * KPL;
          const unsigned char* at = j < len ? cache + (unsigned long long)(uint32_t)j * pos : draft + (long long)(j - len) * dpos;
#pragma unroll
          for (int v = 0; v < V; ++v)
            d[u][v] = cv[v] && j < total && blk < hi ? load_stream(at + v * STEP * ES) : make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    uint4 kr[U][V], vr[U][V];
    if (b < hi) {
      fetch(kr, b, kb, (uint32_t)p.key.pos, dkb, p.dkey.pos);
      fetch(vr, b, vb, (uint32_t)p.value.pos, dvb, p.dvalue.pos);
    }
    float q[MQ][EV];
#pragma unroll
    for (int j = 0; j < MQ; ++j) {
      const unsigned char* src = p.q.data + query_offset(p, p.q, r, h, i0 + min(j, nq - 1)) + c * 16;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint4 d = cv[v] ? __ldg(reinterpret_cast<const uint4*>(src + v * STEP * ES)) : make_uint4(0u, 0u, 0u, 0u);
        float x4[E];
        unpack<DT>(d, x4);
#pragma unroll
        for (int x = 0; x < E; ++x) q[j][v * E + x] = x4[x] * p.scale_log2;
      }
    }
    unsigned alive = ~0u;
    if (p.nodes) {
      __syncwarp();
      if (tree_seen(tree, p.parent + (long long)r * p.nodes, p.nodes, lane, 32, [] { __syncwarp(); }))
        atomicOr(p.status, kDevInternal);
      alive = 0;
#pragma unroll
      for (int j = 0; j < MQ; ++j)
        if (j < nq && tree.mask[p.by_group(i0 + j)]) alive |= 1u << j;
    }
    float m[MQ], l[MQ], o[MQ][EV];
#pragma unroll
    for (int j = 0; j < MQ; ++j) {
      m[j] = -INFINITY;
      l[j] = 0.0f;
#pragma unroll
      for (int x = 0; x < EV; ++x) o[j][x] = 0.0f;
    }
    for (; b < hi; b += W) {
      float part[MQ][U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float k[EV];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float x4[E];
          unpack<DT>(kr[u][v], x4);
#pragma unroll
          for (int x = 0; x < E; ++x) k[v * E + x] = x4[x];
        }
#pragma unroll
        for (int j = 0; j < MQ; ++j) {
          float2 a = __fmul2_rn(make_float2(q[j][0], q[j][1]), make_float2(k[0], k[1]));
#pragma unroll
          for (int x = 2; x < EV; x += 2) a = __ffma2_rn(make_float2(q[j][x], q[j][x + 1]), make_float2(k[x], k[x + 1]), a);
          part[j][u] = a.x + a.y;
        }
      }
      if (b + W < hi) fetch(kr, b + W, kb, (uint32_t)p.key.pos, dkb, p.dkey.pos);
      const int key = b * KB + my_u * KPL + gk;  // this lane's key
      const bool edge = b * KB + KB > len;
      float w[MQ];
#pragma unroll
      for (int j = 0; j < MQ; ++j) {
        float s = reduce_values<LPK>(part[j], lane);
        bool sees = (alive >> j) & 1u;
        if (edge) {
          if (key >= len) sees = sees && key < total && (tree.mask[p.by_group(i0 + min(j, nq - 1))] >> (key - len) & 1ull);
        }
        s = sees ? s : -INFINITY;
        float bm = s;
#pragma unroll
        for (int x = 1; x < U; x <<= 1) bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, x));
#pragma unroll
        for (int x = LPK; x < 32; x <<= 1) bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, x));
        const float mn = fmaxf(m[j], bm), sub = mn == -INFINITY ? 0.0f : mn;
        w[j] = fast_exp2(s - sub);
        if (mn > m[j]) {  // the same in every lane
          const float f = fast_exp2(m[j] - sub);
          l[j] *= f;
#pragma unroll
          for (int x = 0; x < EV; ++x) o[j][x] *= f;
          m[j] = mn;
        }
        l[j] += w[j];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float y4[V][E];
#pragma unroll
        for (int v = 0; v < V; ++v) unpack<DT>(vr[u][v], y4[v]);
        const int from = gk * LPK + (U == 8 ? (u >> 2) | (u & 2) | (u & 1) << 2 : (u >> 1) | (u & 1) << 1);
#pragma unroll
        for (int j = 0; j < MQ; ++j) {
          const float wu = __shfl_sync(~0u, w[j], from);
          // a drafted value that the query does not see may be anything: left out, not times 0
          if (!edge || wu != 0.0f) {
#pragma unroll
            for (int x = 0; x < EV; x += 2) {
              const float2 y = __ffma2_rn(make_float2(wu, wu), make_float2(y4[x / E][x % E], y4[x / E][x % E + 1]),
                                          make_float2(o[j][x], o[j][x + 1]));
              o[j][x] = y.x;
              o[j][x + 1] = y.y;
            }
          }
        }
      }
      if (b + W < hi) fetch(vr, b + W, vb, (uint32_t)p.value.pos, dvb, p.dvalue.pos);
    }
    // over the lane groups
#pragma unroll
    for (int j = 0; j < MQ; ++j) {
#pragma unroll
      for (int x = 1; x < U; x <<= 1) l[j] += __shfl_xor_sync(~0u, l[j], x);
#pragma unroll
      for (int x = LPK; x < 32; x <<= 1) {
        l[j] += __shfl_xor_sync(~0u, l[j], x);
#pragma unroll
        for (int y = 0; y < EV; ++y) o[j][y] += __shfl_xor_sync(~0u, o[j][y], x);
      }
    }
    if (W == 1) {  // never split
#pragma unroll
      for (int j = 0; j < MQ; ++j) {
        if (j < nq && gk == j % KPL) {
          const float inv = l[j] == 0.0f ? 0.0f : 1.0f / l[j];
          unsigned char* to = p.out.data + query_offset(p, p.out, r, h, i0 + j) + c * 16;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            float y[E];
#pragma unroll
            for (int x = 0; x < E; ++x) y[x] = l[j] == 0.0f ? 0.0f : o[j][v * E + x] * inv;
            if (cv[v]) *reinterpret_cast<uint4*>(to + v * STEP * ES) = pack_vec(y);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < MQ; ++j) {
        if (lane == 0) {
          wm[warp][j] = m[j];
          wl[warp][j] = l[j];
        }
        if (gk == j % KPL) {
#pragma unroll
          for (int v = 0; v < V; ++v)
            *reinterpret_cast<float4*>(&acc[warp][j][c * E + v * STEP]) =
                make_float4(o[j][v * E], o[j][v * E + 1], o[j][v * E + 2], o[j][v * E + 3]);
        }
      }
      __syncthreads();
      for (int e2 = threadIdx.x; e2 < nq * (p.dim / E); e2 += kAsThreads) {
        const int j = e2 / (p.dim / E), x0 = (e2 - j * (p.dim / E)) * E;
        float M = wm[0][j];
#pragma unroll
        for (int w2 = 1; w2 < kAsWarps; ++w2) M = fmaxf(M, wm[w2][j]);
        const float sub = M == -INFINITY ? 0.0f : M;
        float L = 0.0f, y[E];
#pragma unroll
        for (int x = 0; x < E; ++x) y[x] = 0.0f;
#pragma unroll
        for (int w2 = 0; w2 < kAsWarps; ++w2) {
          const float lw = wl[w2][j], f = fast_exp2(wm[w2][j] - sub);
          L = fmaf(f, lw, L);
#pragma unroll
          for (int x = 0; x < E; ++x) y[x] = add_part(y[x], f, acc[w2][j][x0 + x], lw);
        }
        if (p.splits == 1) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
          for (int x = 0; x < E; ++x) y[x] = L == 0.0f ? 0.0f : y[x] * inv;
          *reinterpret_cast<uint4*>(p.out.data + query_offset(p, p.out, r, h, i0 + j) + x0 * ES) = pack_vec(y);
        } else {
          const long long row = (((long long)r * p.kv_heads + h) * p.m + i0 + j) * p.splits + split;
#pragma unroll
          for (int x = 0; x < E; x += 4)
            *reinterpret_cast<float4*>(p.part_o + row * p.dim + x0 + x) = make_float4(y[x], y[x + 1], y[x + 2], y[x + 3]);
          if (x0 == 0) p.part_ml[row] = make_float2(M, L);
        }
      }
    }
  }
}

template <int LPK, int V, int MQ>
cudaError_t run_step(const AttendParams& p, cudaStream_t stream) {
  long long grid = p.items;
  if (p.warps == 1) {
    static std::atomic<uint64_t> known{0};
    int occ = 0;
    const cudaError_t e = resident_ctas(attend_step_kernel<LPK, V, MQ>, kAsThreads, 0, known, &occ);
    if (e != cudaSuccess) return e;
    const long long need = (p.items + kAsWarps - 1) / kAsWarps, fit = (long long)kAtSms * occ;
    grid = need < fit ? need : fit;
  }
  attend_step_kernel<LPK, V, MQ><<<(unsigned)grid, kAsThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int LPK>
cudaError_t run_step_queries(const AttendParams& p, cudaStream_t stream) {
  switch (p.m_step) {
    case 1: return run_step<LPK, 1, 1>(p, stream);
    case 2: return run_step<LPK, 1, 2>(p, stream);
    case 4: return run_step<LPK, 1, 4>(p, stream);
    default: return run_step<LPK, 1, 8>(p, stream);
  }
}

}  // namespace

int attend_step_queries(int dim, int m) { return m <= 1 ? 1 : m <= 2 ? 2 : m <= 4 || dim > 128 ? 4 : 8; }

cudaError_t launch_attend_step(const AttendParams& p, cudaStream_t stream) {
  if (p.dim <= 32) return run_step_queries<8>(p, stream);
  if (p.dim <= 64) return run_step_queries<16>(p, stream);
  if (p.dim <= 128) return run_step_queries<32>(p, stream);
  if (p.m_step == 1) return run_step<32, 2, 1>(p, stream);
  return p.m_step == 2 ? run_step<32, 2, 2>(p, stream) : run_step<32, 2, 4>(p, stream);
}

}  // namespace lsb
