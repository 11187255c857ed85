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

// A worker's part of an item: blocks [lo, hi) of nb.
struct PgPart {
  int r, h, i0, nq, len, nb, lo, hi;
  int parts, part, base;  // of a cut item: their number, this one's, and where their places begin
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

template <int KB>
struct PgWalk {
  const PagedParams& p;
  const int worker, lane;
  int run;              // rows of a lane
  PgCount before_u, sum_u, before_p, sum_p;  // blocks and parts (of one item) before the lane's rows, and in them
  PgCount total;        // blocks of all items
  PgCount at, end;      // long rows: blocks; short: parts, by steps of the workers
  bool cut;             // long rows
  // the row that `at` lies in
  int r, len, nb, next_len;
  PgCount row_u, row_p;
  int item;             // of the row, the next to take (long rows)

  __device__ __forceinline__ int keys_of(int row) const { return row < p.rows ? __ldg(p.len + row) : 0; }
  __device__ __forceinline__ int clamp_len(int n) const { return min(max(n, 0), p.pages.places); }
  __device__ __forceinline__ static int blocks_of(int n) { return max((n + KB - 1) / KB, 1); }
  __device__ __forceinline__ int parts_of(int blocks) const { return (blocks + p.least - 1) / p.least; }

  __device__ __forceinline__ PgWalk(const PagedParams& params, int worker_, int lane_) : p(params), worker(worker_), lane(lane_) {
    run = (p.rows + 31) / 32;
    PgCount u = 0, n = 0;
    const int first = min(lane * run, p.rows), last = min(first + run, p.rows);
#pragma unroll 4
    for (int i = first; i < last; ++i) {
      const int b = blocks_of(clamp_len(__ldg(p.len + i)));
      u += b;
      n += parts_of(b);
    }
    sum_u = u;
    sum_p = n;
    before_u = pg_scan(u, lane);
    before_p = pg_scan(n, lane);
    const PgCount all_u = __shfl_sync(~0u, before_u, 31), all_p = __shfl_sync(~0u, before_p, 31);
    before_u -= u;
    before_p -= n;
    total = all_u * p.per_row;
    const PgCount workers = p.workers;
    cut = total >= workers * p.least;
    if (cut) {
      // worker * total / workers, without the product's overflow
      const PgCount q = total / workers, rest = total - q * workers;
      at = q * worker + rest * worker / workers;
      end = q * (worker + 1) + rest * (worker + 1) / workers;
      locate();
      const PgCount off = at - row_u;
      item = (int)(off / nb);
    } else {
      at = worker;
      end = all_p * p.per_row;
    }
  }

  // The row that holds `at` (blocks, or parts), by all lanes.
  __device__ __forceinline__ void locate() {
    const PgCount per = p.per_row, mine = cut ? before_u : before_p, sum = cut ? sum_u : sum_p;
    const unsigned hit = __ballot_sync(~0u, at >= mine * per && at < (mine + sum) * per);
    const int src = hit ? __ffs(hit) - 1 : 0;
    PgCount u = __shfl_sync(~0u, before_u, src), n = __shfl_sync(~0u, before_p, src);
    const int first = src * run, last = min(first + run, p.rows);
    for (int i = first;; i += 32) {
      const int row = i + lane, l = row < last ? clamp_len(__ldg(p.len + row)) : 0, b = row < last ? blocks_of(l) : 0;
      const int k = row < last ? parts_of(b) : 0;
      const PgCount su = pg_scan((PgCount)b, lane) + u, sn = pg_scan((PgCount)k, lane) + n;
      const unsigned past = __ballot_sync(~0u, at < (cut ? su : sn) * per);
      if (past || i + 32 >= last) {
        const int j = past ? __ffs(past) - 1 : 0;
        r = i + j;
        len = __shfl_sync(~0u, l, j);
        nb = __shfl_sync(~0u, b, j);
        row_u = __shfl_sync(~0u, su - b, j) * per;
        row_p = __shfl_sync(~0u, sn - k, j) * per;
        break;
      }
      u = __shfl_sync(~0u, su, 31);
      n = __shfl_sync(~0u, sn, 31);
    }
    nb = max(nb, 1);
    next_len = keys_of(r + 1);
  }

  __device__ __forceinline__ bool next(PgPart& x) {
    if (at >= end) return false;
    PgCount item_u;
    if (cut) {
      if (item == p.per_row) {
        ++r;
        row_u += (PgCount)nb * p.per_row;
        len = clamp_len(next_len);
        nb = blocks_of(len);
        next_len = keys_of(r + 1);
        item = 0;
      }
      item_u = row_u + (PgCount)item * nb;
      x.lo = (int)(at - item_u);
      x.hi = (int)min((PgCount)nb, x.lo + (end - at));
    } else {
      locate();
      const int k = parts_of(nb);
      const PgCount off = at - row_p;
      item = (int)(off / k);
      x.part = (int)(off - (PgCount)item * k);
      x.lo = x.part * p.least;
      x.hi = min(x.lo + p.least, nb);
      item_u = row_u + (PgCount)item * nb;
    }
    x.r = r;
    x.h = p.by_tiles(item);
    x.i0 = (item - x.h * p.tiles) * p.tile;
    x.nq = min(p.tile, p.group - x.i0);
    x.len = len;
    x.nb = nb;
    x.parts = 1;
    if (x.lo > 0 || x.hi < nb) {
      if (cut) {
        const PgCount w = p.workers;
        x.base = owner(item_u, w);
        x.parts = owner(item_u + nb - 1, w) - x.base + 1;
        x.part = worker - x.base;
      } else {
        x.base = (int)(item_u / p.least);
        x.parts = parts_of(nb);
      }
    }
    if (cut) {
      at += x.hi - x.lo;
      if (x.hi == nb) ++item;
    } else {
      at += p.workers;
    }
    return true;
  }

  // The worker whose run holds block u: the last c with floor(c total / workers) <= u.
  __device__ __forceinline__ int owner(PgCount u, PgCount workers) const {
    const PgCount q = total / workers, rest = total - q * workers;
    // an estimate, put right against the exact bounds
    long long c = (long long)((double)(u + 1) * (double)workers / (double)total);
    c = max(0ll, min(c, (long long)workers - 1));
    while (c + 1 < (long long)workers && q * (c + 1) + rest * (c + 1) / workers <= u) ++c;
    while (c > 0 && q * c + rest * c / workers > u) --c;
    return (int)c;
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

// The parts of an item added up, in their order, by N threads.
__device__ __forceinline__ void pg_join(const PagedParams& p, const PgPart& x, int dtype, int t, int n) {
  const bool four = p.dim % 4 == 0;
  const int step = four ? 4 : 1, per = p.dim / step;
  for (int e = t; e < x.nq * per; e += n) {
    const int q = e / per, d = (e - q * per) * step;
    float m = -INFINITY;
    for (int j = 0; j < x.parts; ++j) m = fmaxf(m, __ldcg(p.part_ml + (long long)pg_slot(x.base, j) * p.tile + q).x);
    const float sub = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int j = 0; j < x.parts; ++j) {
      const long long at = (long long)pg_slot(x.base, j) * p.tile + q;
      const float2 ml = __ldcg(p.part_ml + at);
      const float f = fast_exp2(ml.x - sub);
      const float* from = p.part_o + at * p.dim + d;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (four) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(from));
        v[0] = y.x;
        v[1] = y.y;
        v[2] = y.z;
        v[3] = y.w;
      } else {
        v[0] = __ldcg(from);
      }
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(f, v[i], o[i]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    unsigned char* out = pg_out(p, x, q);
    const int es = dtype == DT_F32 ? 4 : 2;
    for (int i = 0; i < step; ++i) pg_store_as(dtype, out + (long long)(d + i) * es, o[i] * inv);
  }
}

// Eight-bit codes as floats.
__device__ __forceinline__ float2 e4m3x2_float(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace lsb
