// Device side shared by the kernels of the single-token attention over pages: how the work is shared
// out, the page look-up and the join of an item's parts.
//
// An item is a row, a key head and up to `tile` of its query heads; its keys are blocks of KB.  The
// lengths are on the GPU only, so every warp adds up the rows' blocks for itself (32 lanes, a run of
// rows each) and finds its own share:
//   long rows:  all blocks in one order, each worker an equal run of them, whatever items it cuts;
//   short ones: a part per `least` blocks of an item, the workers in turn.
// A cut item's parts leave their sums in the workspace, and the worker that comes last joins them, in
// the order of the keys: the result does not depend on which comes last.
#pragma once

#include "ls_device.cuh"
#include "ls_dtype.cuh"
#include "ls_paged.h"

namespace lsb {

using PgCount = unsigned long long;

// A worker's part of an item: blocks [lo, hi).
struct PgPart {
  int r, h, i0, nq, len, lo, hi;
  int parts, part, base;  // the item's parts, this one's number, and (if there are others) where their places begin
};
__device__ __forceinline__ int pg_slot(int base, int part) { return 2 * (base + part) + (part == 0); }

__device__ __forceinline__ PgCount pg_scan(PgCount v, int lane) {  // inclusive, over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const PgCount t = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

struct PgChunk {  // a run of rows: their blocks, and the parts of one item each
  PgCount blocks, parts;
};
struct PgState {  // a warp's place in its share (the same for all lanes; shared memory, read and written now and then)
  PgCount at, end;      // long rows: blocks; short: parts, by steps of the workers
  PgCount total, each;  // blocks of all items, and of a worker; `rest` workers have one more between them
  PgCount row_u;        // blocks before the row that `at` lies in
  int rest, r, len, nb, item;
  bool cut;             // long rows
};
struct PgShare {
  PgChunk chunks[32];
  PgState state[kPgWarps];
};

template <int KB>
struct PgWalk {
  const PagedParams& p;
  PgShare& sh;
  PgState& st;
  const int worker, lane;
  int next_len;         // of the row after (long rows)

  __device__ __forceinline__ int keys_of(int row) const { return row < p.rows ? __ldg(p.len + row) : 0; }
  __device__ __forceinline__ int clamp_len(int n) const { return min(max(n, 0), p.pages.places); }
  __device__ __forceinline__ static int blocks_of(int n) { return max((n + KB - 1) / KB, 1); }
  __device__ __forceinline__ int parts_of(int blocks) const { return (blocks + p.least - 1) / p.least; }

  // by all threads of the CTA
  __device__ __forceinline__ PgWalk(const PagedParams& params, PgShare& share, int worker_, int warp, int lane_)
      : p(params), sh(share), st(share.state[warp]), worker(worker_), lane(lane_), next_len(0) {
    {
      constexpr int PER = kPgThreads / 32;  // threads of a chunk
      const int c = threadIdx.x / PER, run = (p.rows + 31) / 32;
      PgCount u = 0, n = 0;
      const int last = (int)min((long long)(c + 1) * run, (long long)p.rows);
#pragma unroll 4
      for (long long i = (long long)c * run + threadIdx.x % PER; i < last; i += PER) {
        const int b = blocks_of(clamp_len(__ldg(p.len + i)));
        u += b;
        n += parts_of(b);
      }
#pragma unroll
      for (int o = 1; o < PER; o <<= 1) {
        u += __shfl_xor_sync(~0u, u, o);
        n += __shfl_xor_sync(~0u, n, o);
      }
      if (threadIdx.x % PER == 0) sh.chunks[c] = PgChunk{u, n};
    }
    __syncthreads();
    PgState s;
    const PgChunk mine = sh.chunks[lane];
    s.total = __shfl_sync(~0u, pg_scan(mine.blocks, lane), 31) * p.per_row;
    s.cut = s.total >= (PgCount)p.workers * p.least;
    s.each = s.total / p.workers;
    s.rest = (int)(s.total - s.each * p.workers);
    s.row_u = 0;
    s.r = s.len = s.nb = s.item = 0;
    if (s.cut) {
      s.at = start_of(s, worker);
      s.end = start_of(s, worker + 1);
      PgCount unused;
      locate(s, unused);
      s.item = (int)((s.at - s.row_u) / s.nb);
    } else {
      s.at = worker;
      s.end = __shfl_sync(~0u, pg_scan(mine.parts, lane), 31) * p.per_row;
    }
    if (lane == 0) st = s;
    __syncwarp();
  }
  // worker * total / workers, without the product's overflow
  __device__ __forceinline__ PgCount start_of(const PgState& s, long long w) const { return s.each * w + (PgCount)s.rest * w / (unsigned)p.workers; }

  // The row that s.at (blocks, or parts) lies in, by all lanes; row_p: parts before it.
  __device__ __forceinline__ void locate(PgState& s, PgCount& row_p) {
    const PgChunk mine = sh.chunks[lane];
    const PgCount per = p.per_row, up_u = pg_scan(mine.blocks, lane), up_n = pg_scan(mine.parts, lane);
    const PgCount upto = s.cut ? up_u : up_n;
    const unsigned over = __ballot_sync(~0u, s.at < upto * per);
    const int src = over ? __ffs(over) - 1 : 31;
    PgCount u = __shfl_sync(~0u, up_u - mine.blocks, src), n = __shfl_sync(~0u, up_n - mine.parts, src);
    const long long run = (p.rows + 31) / 32;
    const int last = (int)min((src + 1) * run, (long long)p.rows);
    for (int i = (int)min(src * run, (long long)p.rows);; i += 32) {
      const int row = i + lane;
      const bool in = row < last;
      const int l = in ? clamp_len(__ldg(p.len + row)) : 0, b = in ? blocks_of(l) : 0, k = in ? parts_of(b) : 0;
      const PgCount su = pg_scan((PgCount)b, lane) + u, sn = pg_scan((PgCount)k, lane) + n;
      const unsigned past = __ballot_sync(~0u, in && s.at < (s.cut ? su : sn) * per);
      if (past || i + 32 >= last) {
        const int j = past ? __ffs(past) - 1 : 0;
        s.r = i + j;
        s.len = __shfl_sync(~0u, l, j);
        s.nb = max(__shfl_sync(~0u, b, j), 1);
        s.row_u = __shfl_sync(~0u, su - b, j) * per;
        row_p = __shfl_sync(~0u, sn - k, j) * per;
        break;
      }
      u = __shfl_sync(~0u, su, 31);
      n = __shfl_sync(~0u, sn, 31);
    }
    if (s.cut) next_len = keys_of(s.r + 1);
  }

  // The next part (by all lanes), or false.
  __device__ __forceinline__ bool next(PgPart& x) {
    const PgCount at = st.at, end = st.end;
    if (at >= end) return false;
    int r = st.r, len = st.len, nb = st.nb, item = st.item;
    PgCount row_u = st.row_u, step = p.workers;
    const bool cut = st.cut;
    bool moved = false;  // to another row
    if (cut) {
      if (item == p.per_row) {
        moved = true;
        ++r;
        row_u += (PgCount)nb * p.per_row;
        len = clamp_len(next_len);
        nb = blocks_of(len);
        item = 0;
        next_len = keys_of(r + 1);
      }
      const PgCount item_u = row_u + (PgCount)item * nb;
      x.lo = (int)(at - item_u);
      x.hi = (int)min((PgCount)nb, x.lo + (end - at));
      x.parts = 1;
      if (x.lo > 0 || x.hi < nb) {
        const PgState s = st;
        x.base = owner(s, item_u);
        x.parts = owner(s, item_u + nb - 1) - x.base + 1;
        x.part = worker - x.base;
      }
      step = x.hi - x.lo;
    } else {
      moved = true;
      PgState s = st;
      PgCount row_p;
      locate(s, row_p);
      r = s.r;
      len = s.len;
      nb = s.nb;
      row_u = s.row_u;
      const int k = parts_of(nb);
      const unsigned off = (unsigned)(at - row_p);  // (below parts of an item * items of a row, on the short path)
      item = (int)(off / (unsigned)k);
      x.part = (int)(off - (unsigned)item * k);
      x.lo = x.part * p.least;
      x.hi = min(x.lo + p.least, nb);
      x.parts = k;
      x.base = k > 1 ? (int)((row_u + (PgCount)item * nb) / p.least) : 0;
    }
    x.r = r;
    x.h = p.by_tiles(item);
    x.i0 = (item - x.h * p.tiles) * p.tile;
    x.nq = min(p.tile, p.group - x.i0);
    x.len = len;
    __syncwarp();
    if (lane == 0) {
      st.at = at + step;
      st.item = cut && x.hi == nb ? item + 1 : item;
      if (moved) {
        st.r = r;
        st.len = len;
        st.nb = nb;
        st.row_u = row_u;
      }
    }
    __syncwarp();
    return true;
  }

  // The worker whose run holds block u: the last w with start_of(w) <= u.  An estimate, put right.
  __device__ __forceinline__ int owner(const PgState& s, PgCount u) const {
    long long w = (long long)((float)u * (float)p.workers / (float)s.total);
    w = max(0ll, min(w, (long long)p.workers - 1));
    while (w + 1 < p.workers && start_of(s, w + 1) <= u) ++w;
    while (w > 0 && start_of(s, w) > u) --w;
    return (int)w;
  }
};

// Where position n of row r lies: its page and its place in it; page -1 where there is none (past
// len, or a page out of range, which `bad` notes).
__device__ __forceinline__ int pg_page(const PagedParams& p, long long table, int n, int len, int& place, bool& bad) {
  const int s = p.pages.by_page(n);
  place = n - s * p.pages.page_size;
  if (n >= len) return -1;
  const int page = __ldg(p.pages.table + table + s);
  if ((unsigned)page < (unsigned)p.pages.num_pages) return page;
  bad = true;
  return -1;
}

template <int DT>
__device__ __forceinline__ void pg_store(unsigned char* at, float x) {
  if constexpr (DT == DT_F32)
    *reinterpret_cast<float*>(at) = x;
  else if constexpr (DT == DT_F16)
    *reinterpret_cast<__half*>(at) = __float2half_rn(x);
  else
    *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(x);
}
__device__ __forceinline__ void pg_store_as(int dtype, unsigned char* at, float x) {
  if (dtype == DT_F32)
    pg_store<DT_F32>(at, x);
  else if (dtype == DT_F16)
    pg_store<DT_F16>(at, x);
  else
    pg_store<DT_BF16>(at, x);
}

__device__ __forceinline__ unsigned char* pg_out(const PagedParams& p, const PgPart& x, int q) {
  return p.out.data + (long long)x.r * p.out.row + (long long)(x.h * p.group + x.i0 + q) * p.out.head;
}

// Whether this worker's part is the last of its item to come; by all its N threads (thread t), which have
// stored the part before.  The counter is left at zero for the next launch.
template <class Sync>
__device__ __forceinline__ bool pg_last(const PagedParams& p, const PgPart& x, int t, int* flag, Sync sync) {
  __threadfence();
  sync();
  if (t == 0) {
    const bool last = atomicAdd(p.arrived + x.base, 1u) + 1u == (unsigned)x.parts;
    if (last) p.arrived[x.base] = 0;
    *flag = last;
  }
  sync();
  const bool last = *(volatile int*)flag != 0;
  if (last) __threadfence();
  return last;
}

// The parts of an item added up, in their order, by `warps` warps, a query each.  The lanes first take a part each
// for its factor, then the elements, 8 parts' loads under way at once.
template <int EL>  // elements of a lane's load: 4 where the head size is a multiple of 4
__device__ __forceinline__ void pg_join_by(const PagedParams& p, const PgPart& x, int dtype, int warp, int warps, int lane) {
  const int es = dtype == DT_F32 ? 4 : 2;
  for (int q = warp; q < x.nq; q += warps) {
    float m = -INFINITY;
    for (int j = lane; j < x.parts; j += 32) m = fmaxf(m, __ldcg(p.part_ml + (long long)pg_slot(x.base, j) * p.tile + q).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    const float sub = m == -INFINITY ? 0.0f : m;
    for (int d0 = 0; d0 < p.dim; d0 += 32 * EL) {
      const int d = d0 + lane * EL;
      const bool mine = d < p.dim;
      float l = 0.0f, o[EL];
#pragma unroll
      for (int i = 0; i < EL; ++i) o[i] = 0.0f;
      for (int j0 = 0; j0 < x.parts; j0 += 32) {
        float f = 0.0f;
        if (j0 + lane < x.parts) {
          const float2 ml = __ldcg(p.part_ml + (long long)pg_slot(x.base, j0 + lane) * p.tile + q);
          f = fast_exp2(ml.x - sub);
          l = fmaf(f, ml.y, l);
        }
        constexpr int AT_ONCE = 8;
        for (int k = 0; k < min(32, x.parts - j0); k += AT_ONCE) {
          float v[AT_ONCE][EL];
#pragma unroll
          for (int y = 0; y < AT_ONCE; ++y) {
            const bool there = mine && j0 + k + y < x.parts;
            const float* from = p.part_o + ((long long)pg_slot(x.base, there ? j0 + k + y : 0) * p.tile + q) * p.dim + (mine ? d : 0);
            if constexpr (EL == 4) {
              const float4 z = there ? __ldcg(reinterpret_cast<const float4*>(from)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              v[y][0] = z.x;
              v[y][1] = z.y;
              v[y][2] = z.z;
              v[y][3] = z.w;
            } else {
              v[y][0] = there ? __ldcg(from) : 0.0f;
            }
          }
#pragma unroll
          for (int y = 0; y < AT_ONCE; ++y) {
            const float fy = __shfl_sync(~0u, f, k + y);
#pragma unroll
            for (int i = 0; i < EL; ++i) o[i] = fmaf(fy, v[y][i], o[i]);
          }
        }
      }
#pragma unroll
      for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(~0u, l, k);
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      unsigned char* out = pg_out(p, x, q) + (long long)d * es;
#pragma unroll
      for (int i = 0; i < EL; ++i)
        if (mine) pg_store_as(dtype, out + i * es, o[i] * inv);
    }
  }
}
__device__ __forceinline__ void pg_join(const PagedParams& p, const PgPart& x, int dtype, int warp, int warps, int lane) {
  if (p.dim % 4 == 0)
    pg_join_by<4>(p, x, dtype, warp, warps, lane);
  else
    pg_join_by<1>(p, x, dtype, warp, warps, lane);
}

// Eight-bit codes as floats.
__device__ __forceinline__ float2 e4m3x2_float(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace lsb
