// Attention of one new token per row over a paged cache on the CUDA cores: f32 queries, and tensors
// whose layout the tensor-core kernel cannot read (a head size or stride that breaks 16-byte alignment).
//
//   s_n = (scale q) . k_n,  o = sum_n 2^(s_n - max) v_n / sum_n 2^(s_n - max)
//
// in one pass with the running maximum and sum (Milakov and Gimelshein, 2018), all in f32.  An 8-bit
// head vector's scale multiplies its score and its weight, not its elements.
//
// Keys and values go straight from memory into registers, 16 bytes per lane and load: LPK lanes hold
// one vector (V loads each), so that a load covers 32 / LPK keys, and a block is 8 / V such loads of keys
// and as many of values.  Lane n looks up the page of key n of the block after next.  The keys' registers
// are loaded again as soon as the block's scores are formed, the values' when its sums are.  The dot
// products of a lane group are reduced together, each exchange halving the products that a lane still
// holds, which leaves every lane with the score of its own key.  Four warps take a part's blocks in turn
// and merge through shared memory.
//
// What bounds it: the bytes under way (12 to 16 warps of 8 KB less what is at work) and, with four queries or codes,
// instructions.  64 rows x 16 heads of 64 f32, 100 to 700 positions: 66 us, 0.47 of the measured copy rate (three CTAs per
// SM 76); x 8 key heads of 128 with 4 queries 83 us, 0.38; e4m3 pages of 300 to 2700 positions 160 us, 0.19.
#include "ls_paged.cuh"

namespace lsb {
namespace {

enum { CT_F32 = LS_DTYPE_F32, CT_F16 = LS_DTYPE_F16, CT_BF16 = LS_DTYPE_BF16, CT_E4M3 = LS_DTYPE_E4M3, CT_I8 = LS_DTYPE_I8 };

template <int CT>
constexpr int kBytes = CT == CT_F32 ? 4 : CT == CT_F16 || CT == CT_BF16 ? 2 : 1;

// The elements of one 16-byte vector as floats (exact).
template <int CT>
__device__ __forceinline__ void unpack_cache(const uint4& d, float (&x)[16 / kBytes<CT>]) {
  if constexpr (CT <= CT_BF16) {
    unpack<CT>(d, x);
  } else {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (CT == CT_E4M3) {
        const float2 a = e4m3x2_float(w[i] & 0xffffu), b = e4m3x2_float(w[i] >> 16);
        x[4 * i] = a.x;
        x[4 * i + 1] = a.y;
        x[4 * i + 2] = b.x;
        x[4 * i + 3] = b.y;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = (float)(signed char)(w[i] >> 8 * j);
      }
    }
  }
}

// Elements [d0, d0 + 16 / bytes) of a head vector, zeros past dim.
template <int CT, bool VEC>
__device__ __forceinline__ uint4 load_vector(const unsigned char* head, int d0, int dim) {
  constexpr int B = kBytes<CT>;
  if constexpr (VEC) {
    uint4 d;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(d.x), "=r"(d.y), "=r"(d.z), "=r"(d.w)
                 : "l"(head + d0 * B));
    return d;
  } else {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 16 / B; ++e) {
      uint32_t x = 0;
      if (d0 + e < dim) {
        const unsigned char* at = head + (d0 + e) * B;
        if constexpr (B == 4)
          x = __ldg(reinterpret_cast<const uint32_t*>(at));
        else if constexpr (B == 2)
          x = __ldg(reinterpret_cast<const uint16_t*>(at));
        else
          x = __ldg(at);
      }
      w[e * B / 4] |= x << (e * B % 4 * 8);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The N values of each lane summed over the lanes that differ in the bits below LPK; lane l then holds the
// sum of value bit-reversed(l mod N).
template <int LPK, int N>
__device__ __forceinline__ float reduce_lanes(const float (&v)[N], int lane) {
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
template <int N>
__device__ __forceinline__ int reversed(int l) {
  return N == 8 ? (l & 1) << 2 | (l & 2) | (l >> 2 & 1) : (l & 1) << 1 | (l >> 1 & 1);
}

// CTAs of an SM, by the registers that two blocks' loads and the queries take
constexpr int paged_simt_ctas_of(bool vec, bool codes, int queries) { return !vec || (codes && queries > 1) ? 2 : queries > 1 || codes ? 3 : 4; }

template <int CT, bool VEC, int LPK, int V, int MQ>
__global__ void __launch_bounds__(kPgThreads, paged_simt_ctas_of(VEC, kBytes<CT> == 1, MQ)) paged_simt_kernel(const __grid_constant__ PagedParams p, int dtype) {
  constexpr int B = kBytes<CT>, E = 16 / B, EV = E * V, U = 8 / V, KPL = 32 / LPK, KB = U * KPL, STEP = LPK * E;
  constexpr bool Q8 = B == 1;
  __shared__ float wm[kPgWarps][MQ], wl[kPgWarps][MQ];
  __shared__ __align__(16) float acc[kPgWarps][MQ][STEP * V + 4];
  __shared__ int flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LPK, gk = lane / LPK;
  const int my_key = reversed<U>(lane % U) * KPL + gk;  // of a block: the key whose score this lane gets
  bool cv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) cv[v] = (c + LPK * v) * E < p.dim;
  bool bad = false;
  __shared__ PgShare share;
  PgWalk<KB> walk(p, share, blockIdx.x, warp, lane);
  __shared__ PgPart parts[kPgWarps];  // (the warps' own, all the same)
  while (true) {
    {
      PgPart y;
      if (!walk.next(y)) break;
      if (lane == 0) parts[warp] = y;
      __syncwarp();
    }
    const PgPart& x = parts[warp];
    const long long table = (long long)x.r * p.pages.table_row;
    const unsigned char* kh = p.pages.key.data + (long long)x.h * p.pages.key.head;
    const unsigned char* vh = p.pages.value.data + (long long)x.h * p.pages.value.head;
    const unsigned char* ksh = p.pages.kscale.data + (long long)x.h * p.pages.kscale.head;
    const unsigned char* vsh = p.pages.vscale.data + (long long)x.h * p.pages.vscale.head;
    int b = x.lo + warp, place = 0, page = -1;
    auto look_up = [&](int blk) {
      page = -1;
      if (lane < KB && blk < x.hi) page = pg_page(p, table, blk * KB + lane, x.len, place, bad);
    };
    auto fetch = [&](uint4(&d)[U][V], const unsigned char* head, const AtView& view) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int pg = __shfl_sync(~0u, page, u * KPL + gk), pl = __shfl_sync(~0u, place, u * KPL + gk);
        const unsigned char* at = head + (long long)pg * view.row + (long long)pl * view.pos;
#pragma unroll
        for (int v = 0; v < V; ++v)
          d[u][v] = cv[v] && pg >= 0 ? load_vector<CT, VEC>(at, c * E + v * STEP, p.dim) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    float ks = 1.0f, vs = 1.0f;
    bool there = false;
    auto fetch_key_side = [&](uint4(&d)[U][V]) {  // and what the lane's own key needs
      fetch(d, kh, p.pages.key);
      const int pg = __shfl_sync(~0u, page, my_key), pl = __shfl_sync(~0u, place, my_key);
      there = pg >= 0;
      if constexpr (Q8) {
        if (there) {
          ks = __ldg(reinterpret_cast<const float*>(ksh + (long long)pg * p.pages.kscale.row + (long long)pl * p.pages.kscale.pos));
          vs = __ldg(reinterpret_cast<const float*>(vsh + (long long)pg * p.pages.vscale.row + (long long)pl * p.pages.vscale.pos));
        }
      }
    };
    uint4 kr[U][V], vr[U][V];
    look_up(b);
    fetch_key_side(kr);
    fetch(vr, vh, p.pages.value);
    look_up(b + kPgWarps);
    float q[MQ][EV];
#pragma unroll
    for (int j = 0; j < MQ; ++j) {
      const unsigned char* src = p.q.data + (long long)x.r * p.q.row + (long long)(x.h * p.group + x.i0 + min(j, x.nq - 1)) * p.q.head;
#pragma unroll
      for (int e = 0; e < EV; ++e) {
        const int d = c * E + e / E * STEP + e % E;
        float y = 0.0f;
        if (d < p.dim)
          y = dtype == DT_F32 ? load_elem<DT_F32>(src + d * 4) : dtype == DT_F16 ? load_elem<DT_F16>(src + d * 2) : load_elem<DT_BF16>(src + d * 2);
        q[j][e] = y * p.scale_log2;
      }
    }
    float m[MQ], l[MQ], o[MQ][EV];
#pragma unroll
    for (int j = 0; j < MQ; ++j) {
      m[j] = -INFINITY;
      l[j] = 0.0f;
#pragma unroll
      for (int e = 0; e < EV; ++e) o[j][e] = 0.0f;
    }
    for (; b < x.hi; b += kPgWarps) {
      float part[MQ][U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float k[EV];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float y[E];
          unpack_cache<CT>(kr[u][v], y);
#pragma unroll
          for (int e = 0; e < E; ++e) k[v * E + e] = y[e];
        }
#pragma unroll
        for (int j = 0; j < MQ; ++j) {
          float2 a = __fmul2_rn(make_float2(q[j][0], q[j][1]), make_float2(k[0], k[1]));
#pragma unroll
          for (int e = 2; e < EV; e += 2) a = __ffma2_rn(make_float2(q[j][e], q[j][e + 1]), make_float2(k[e], k[e + 1]), a);
          part[j][u] = a.x + a.y;
        }
      }
      const float ks_now = ks, vs_now = vs;
      const bool sees = there;
      if (b + kPgWarps < x.hi) fetch_key_side(kr);
      float w[MQ];
#pragma unroll
      for (int j = 0; j < MQ; ++j) {
        float s = reduce_lanes<LPK>(part[j], lane);
        if constexpr (Q8) s *= ks_now;
        s = sees ? s : -INFINITY;
        float bm = s;
#pragma unroll
        for (int y = 1; y < U; y <<= 1) bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, y));
#pragma unroll
        for (int y = LPK; y < 32; y <<= 1) bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, y));
        const float mn = fmaxf(m[j], bm), sub = mn == -INFINITY ? 0.0f : mn;
        w[j] = fast_exp2(s - sub);
        if (mn > m[j]) {  // the same in every lane
          const float f = fast_exp2(m[j] - sub);
          l[j] *= f;
#pragma unroll
          for (int e = 0; e < EV; ++e) o[j][e] *= f;
          m[j] = mn;
        }
        l[j] += w[j];
        if constexpr (Q8) w[j] = sees ? w[j] * vs_now : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float y[V][E];
#pragma unroll
        for (int v = 0; v < V; ++v) unpack_cache<CT>(vr[u][v], y[v]);
        const int from = gk * LPK + reversed<U>(u);
#pragma unroll
        for (int j = 0; j < MQ; ++j) {
          const float wu = __shfl_sync(~0u, w[j], from);
#pragma unroll
          for (int e = 0; e < EV; e += 2) {
            const float2 z = __ffma2_rn(make_float2(wu, wu), make_float2(y[e / E][e % E], y[e / E][e % E + 1]), make_float2(o[j][e], o[j][e + 1]));
            o[j][e] = z.x;
            o[j][e + 1] = z.y;
          }
        }
      }
      if (b + kPgWarps < x.hi) {
        fetch(vr, vh, p.pages.value);
        look_up(b + 2 * kPgWarps);
      }
    }
    // over the lane groups, then over the warps in their order
#pragma unroll
    for (int j = 0; j < MQ; ++j) {
#pragma unroll
      for (int y = 1; y < U; y <<= 1) l[j] += __shfl_xor_sync(~0u, l[j], y);
#pragma unroll
      for (int y = LPK; y < 32; y <<= 1) {
        l[j] += __shfl_xor_sync(~0u, l[j], y);
#pragma unroll
        for (int e = 0; e < EV; ++e) o[j][e] += __shfl_xor_sync(~0u, o[j][e], y);
      }
      if (lane == 0) {
        wm[warp][j] = m[j];
        wl[warp][j] = l[j];
      }
      if (gk == j % KPL) {
#pragma unroll
        for (int e = 0; e < EV; ++e) acc[warp][j][c * E + e / E * STEP + e % E] = o[j][e];
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < x.nq * p.dim; e += kPgThreads) {
      const int j = e / p.dim, d = e - j * p.dim;
      float M = wm[0][j];
#pragma unroll
      for (int w = 1; w < kPgWarps; ++w) M = fmaxf(M, wm[w][j]);
      const float sub = M == -INFINITY ? 0.0f : M;
      float L = 0.0f, y = 0.0f;
#pragma unroll
      for (int w = 0; w < kPgWarps; ++w) {
        const float f = fast_exp2(wm[w][j] - sub);
        L = fmaf(f, wl[w][j], L);
        y = fmaf(f, acc[w][j][d], y);
      }
      if (x.parts == 1) {
        pg_store_as(dtype, pg_out(p, x, j) + (long long)d * (dtype == DT_F32 ? 4 : 2), L == 0.0f ? 0.0f : y / L);
      } else {
        const long long at = (long long)pg_slot(x.base, x.part) * p.tile + j;
        p.part_o[at * p.dim + d] = y;
        if (d == 0) p.part_ml[at] = make_float2(M, L);
      }
    }
    if (x.parts > 1) {
      if (pg_last(p, x, threadIdx.x, &flag, [] { __syncthreads(); })) pg_join(p, x, dtype, warp, kPgWarps, lane);
    }
    __syncthreads();
  }
  if (bad) atomicOr(p.status, kDevInternal);
  if (blockIdx.x == 0) {  // lengths out of range
    for (int r = threadIdx.x; r < p.rows; r += kPgThreads) {
      const int n = __ldg(p.len + r);
      if (n < 0 || n > p.pages.places) atomicOr(p.status, kDevInternal);
    }
  }
}

template <int CT, bool VEC, int LPK, int V>
cudaError_t run_simt(const PagedParams& p, int dtype, cudaStream_t stream) {
  const unsigned grid = (unsigned)p.workers;
  if constexpr (VEC) {
    if (p.tile == 1) {
      paged_simt_kernel<CT, VEC, LPK, V, 1><<<grid, kPgThreads, 0, stream>>>(p, dtype);
      return cudaGetLastError();
    }
  }
  paged_simt_kernel<CT, VEC, LPK, V, 4><<<grid, kPgThreads, 0, stream>>>(p, dtype);
  return cudaGetLastError();
}

template <int CT, bool VEC>
cudaError_t run_simt_dim(const PagedParams& p, int dtype, cudaStream_t stream) {
  const int vectors = (p.dim * kBytes<CT> + 15) / 16;
  if (vectors <= 8) return run_simt<CT, VEC, 8, 1>(p, dtype, stream);
  if (vectors <= 16) return run_simt<CT, VEC, 16, 1>(p, dtype, stream);
  if constexpr (kBytes<CT> >= 2) {
    if (vectors <= 32) return run_simt<CT, VEC, 32, 1>(p, dtype, stream);
  }
  if constexpr (kBytes<CT> == 4) return run_simt<CT, VEC, 32, 2>(p, dtype, stream);
  return cudaErrorInvalidValue;  // (not reached: head vectors of up to 256 elements)
}

}  // namespace

int paged_simt_queries(int group, bool vec) { return vec && group == 1 ? 1 : 4; }
int paged_simt_ctas(bool vec, bool codes, int tile) { return paged_simt_ctas_of(vec, codes, tile); }

cudaError_t launch_paged_simt(PagedParams p, int dtype, int cache, bool vec, cudaStream_t stream) {
  if (vec) {  // f32 queries
    if (cache == CT_F32) return run_simt_dim<CT_F32, true>(p, dtype, stream);
    return cache == CT_E4M3 ? run_simt_dim<CT_E4M3, true>(p, dtype, stream) : run_simt_dim<CT_I8, true>(p, dtype, stream);
  }
  switch (cache) {
    case CT_F32: return run_simt_dim<CT_F32, false>(p, dtype, stream);
    case CT_F16: return run_simt_dim<CT_F16, false>(p, dtype, stream);
    case CT_BF16: return run_simt_dim<CT_BF16, false>(p, dtype, stream);
    case CT_E4M3: return run_simt_dim<CT_E4M3, false>(p, dtype, stream);
    default: return run_simt_dim<CT_I8, false>(p, dtype, stream);
  }
}

}  // namespace lsb
