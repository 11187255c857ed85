// Attention of many queries over a row's keys (f16 / bf16, head size up to 128) on the 5th
// generation tensor cores: forced prefixes and scored targets of a cross attention, trees of
// drafts whose nodes share their key heads, long rows.
//
//   S = Q K^T,  P = exp2(c S - max),  O = O * correction + P V,  out = O / sum P
//
// with the running maximum and sum of the softmax (Milakov and Gimelshein, 2018).  One CTA per
// SM takes item after item (up to 256 queries of one problem and one part of its keys), in tiles
// of 128 keys (64 for head sizes above 64); twelve warps:
//   warp 8     loads the keys by TMA into a ring of swizzled tiles (64-element panels of 128-byte
//              rows; a tile's second 64 keys are not fetched when the row ends before), and the
//              queries, by TMA where their layout lets it read them in order, else by
//              asynchronous copies;
//   warp 11    the values, in a ring of their own so that neither waits for the other, and what
//              each node of the item's tree sees;
//   warp 9     owns the 512 tensor-memory columns and issues S = Q K^T (Q and K from shared
//              memory, M 128, N the tile's keys);
//   warp 10    issues O += P V (P from tensor memory, V read as the transposed operand from the
//              same [key][element] tile).  Two warps, because a job's waits, commits and
//              products take one warp longer to issue than the tensor cores to run.  Each walks
//              the jobs as a whole, so that the compiler sees one path and keeps the operands in
//              uniform registers; an elected lane issues;
//   warps 0-3, 4-7  the softmax of slot 0 and slot 1: a thread has one query (one lane of tensor
//              memory), reads its scores of the tile, and writes its weights over them as 16-bit
//              values (rounded to the tensors' type; sums are of the unrounded f32 weights).
// Jobs (a key tile of one slot) alternate between the slots, so that the tensor cores work for
// one slot while the other's softmax runs.  With more than 128 queries the slots are two tiles of
// queries over the same key tiles (each fetched once for 256 queries); with fewer they are the
// even and the odd key tiles of the same queries, joined at the end: both warpgroups read both
// accumulators and each writes half of the columns.  Three or four score buffers let scores run
// ahead of the values, also into the next item.
//
// What bounds it:
// - head size 128: the scores' products, which read 6 KB of shared memory per 64-key instruction
//   (at its 128 bytes a clock 48 cycles, for 32 of tensor work).  509 queries over up to 2048
//   states, 32 x 16 heads: 217 us, 1090 TFLOP/s, 0.57 of the measured bf16 rate;
// - head size 64: the chain of a job (the wait for its scores, their load, maximum, exponentials, store and
//   hand-over) with two softmax warps a scheduler: 40% of the issue slots and 28% of the tensor pipe are
//   used; then the turn from item to item.  400 queries over up to 1021 states, 24 x 16 heads: 63 us,
//   537 TFLOP/s;
// - rows of different lengths: items go to CTAs by their index.  32 trees of 64 nodes x 4 query heads over
//   1025 to 4000 positions, 8 key heads: 107 us, where the longest CTA has 113 key tiles and the mean is 68;
// - few queries over long rows: memory.  64 queries over 131000 positions, 8 heads: 537 MB in 88 us with
//   the joining of the parts, 0.90 of the measured copy rate.
//
// The accumulator is rescaled only when a query's maximum has grown by more than 2^8 since the
// last time: until then its weights are at most 2^8 times as large (in f16 2^15, kAtLift), which f32
// sums and the 16-bit types hold without loss.  Every wait is bounded: one that runs out sets the timeout bit of the
// status word, and the CTA lets its copies and products finish, frees its tensor memory and
// returns.
#include <cuda.h>

#include <type_traits>

#include "ls_device.cuh"
#include "ls_dtype.cuh"
#include "ls_tc.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

constexpr int kTaThreads = 384;
constexpr int kTaM = 128;   // queries of a slot
constexpr uint32_t kTaPanel = 128 * 128;  // a panel of queries: 128 rows of 64 16-bit elements
constexpr uint32_t kTaCols = 512;
constexpr long long kTaDrainNs = 2000000000LL;
constexpr float kTaLazy = 8.0f;           // growth of the maximum (log2) that is let pass

template <int DP>
struct TcShape {
  static constexpr int PANELS = DP / 64;
  // Keys of a tile.  512 columns of tensor memory hold the sums of both slots and the score
  // buffers: at 128 elements and 128 keys only two, and each job would wait for the products of
  // the job before (509 queries over 2048 states: 234 us); at 64 keys four (220 us), although the
  // scores' products then read the queries from shared memory twice as often.
  static constexpr int N = DP == 64 ? 128 : 64;
  static constexpr int NSB = DP == 64 ? 3 : 4;                 // score buffers
  static constexpr int NST = 4;                                // stages of either ring
  static constexpr int NQB = DP == 64 ? 2 : 1;                 // pairs of query tiles
  static constexpr uint32_t QT = PANELS * kTaPanel;            // 128 queries of DP elements
  static constexpr uint32_t PANEL = N * 128, TILE = PANELS * PANEL;  // N keys or values
  static constexpr uint32_t Q = 0, K = 2 * NQB * QT, V = K + NST * TILE, BAR = V + NST * TILE;
  static constexpr uint32_t O = NSB * N;                       // tensor-memory column of slot 0's sums
  // barriers: full / empty of K and V and of the queries, scores, score buffer free, weights, sums x
  // slots, sums read, join, tree there / read x turns, all products issued x 2
  static constexpr int B_KF = 0, B_KE = NST, B_VF = 2 * NST, B_VE = 3 * NST, B_QF = 4 * NST, B_QE = B_QF + NQB,
                       B_S = B_QE + NQB, B_SE = B_S + NSB, B_P = B_SE + NSB, B_O = B_P + NSB, B_OE = B_O + 2, B_J = B_OE + 1, B_T = B_J + 1, B_TE = B_T + 2,
                       B_DONE = B_TE + 2, NBAR = B_DONE + 2;
  static constexpr uint32_t WORDS = BAR + 8 * NBAR;            // tensor-memory address, abort flag, value flag
  static constexpr uint32_t BYTES = WORDS + 16 + 1024;         // + alignment of the tiles
};

// Shared-memory matrix descriptors of tiles in panels with the 128-byte swizzle.
// K-major (Q, K): rows of 128 bytes, 8-row atoms.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// MN-major (V as the operand whose rows are head elements): atoms of 64 elements by 8 keys; a
// panel further for the next 64 elements, 1024 bytes for the next 8 keys.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t panel) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(panel >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

template <bool BF>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Waits of this kernel: bounded, and given up when another role gave up.
struct Waits {
  volatile int* abort;
  uint32_t* status;
  long long limit;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_test_wait(bar, parity)) return true;
    if (limit <= 0) return give_up();
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
      // (a try_wait puts the warp aside for a while; a loop of plain tests would take issue slots
      // and shared-memory cycles from the softmax warps)
      if (mbar_try_wait(bar, parity)) return true;
      if ((n & 15u) == 0) {  // the timer and the flag are slow to read
        if (*abort) return false;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if ((long long)(now - t0) >= limit) return give_up();
      }
    }
  }
  __device__ __forceinline__ bool give_up() const {
    *abort = 1;
    atomicOr(status, kDevTimeout);
    return false;
  }
};

// One item: the queries i0 .. i0 + nq of problem (r, h) and tiles t_lo .. t_lo + nt of its keys
// (tile nb: the drafted tokens), in `jobs` jobs: job j belongs to slot j & 1.
template <int N>
struct TcItem {
  int r, h, i0, nq, split, len, nb, t_lo, nt, jobs;
  bool wide;  // two tiles of queries; otherwise the slots share one
  __device__ __forceinline__ int tile(int j) const { return wide ? j >> 1 : j; }
  __device__ __forceinline__ bool draft(int t) const { return t_lo + t >= nb; }
  __device__ __forceinline__ int keys(int t, int nodes) const { return draft(t) ? nodes : min(N, len - (t_lo + t) * N); }
};
__device__ __forceinline__ int tc_row(const AttendParams& p, int it) { return p.by_head(p.by_tile(p.by_split(it))); }
template <int N>
__device__ __forceinline__ TcItem<N> tc_item(const AttendParams& p, int it, int len) {
  TcItem<N> x;
  const int a = p.by_split(it), b = p.by_tile(a);
  x.split = it - a * p.splits;
  x.i0 = (a - b * p.m_tiles) * p.m_step;
  x.r = p.by_head(b);
  x.h = b - x.r * p.kv_heads;
  x.nq = min(p.m_step, p.m - x.i0);
  x.wide = x.nq > kTaM;
  x.len = min(max(len, 0), p.max_len);
  x.nb = (x.len + N - 1) / N;
  const int nbt = x.nb + (p.nodes ? 1 : 0), per = p.splits == 1 ? nbt : (nbt + p.splits - 1) / p.splits;
  x.t_lo = min(x.split * per, nbt);
  x.nt = min(per, nbt - x.t_lo);
  x.jobs = x.wide ? 2 * x.nt : x.nt;
  return x;
}

// A walk over this CTA's items that have tiles: the next length is loaded while an item is worked on.
template <int N>
struct TcWalk {
  unsigned it;  // (unsigned: an item's number plus the stride, each below 2^31, may pass it)
  int next_len;
  int active;   // items with tiles before this one
  int job, tile;  // jobs and tiles before this item's
  TcItem<N> x;
  bool valid;
  __device__ __forceinline__ void load(const AttendParams& p, unsigned i) {
    // the shuffle tells the compiler that the value is one for the warp
    next_len = __shfl_sync(~0u, i < (unsigned)p.items ? __ldg(p.len + tc_row(p, i)) : 0, 0);
  }
  __device__ __forceinline__ void find(const AttendParams& p) {
    for (; it < (unsigned)p.items; it += gridDim.x) {
      x = tc_item<N>(p, it, next_len);
      load(p, it + gridDim.x);
      if (x.nt > 0) {
        valid = true;
        return;
      }
    }
    valid = false;
  }
  __device__ __forceinline__ void begin(const AttendParams& p) {
    it = blockIdx.x;
    active = job = tile = 0;
    load(p, it);
    find(p);
  }
  __device__ __forceinline__ void next(const AttendParams& p) {
    ++active;
    job += x.jobs;
    tile += x.nt;
    it += gridDim.x;
    find(p);
  }
};

template <bool BF, int DP>
__global__ void __launch_bounds__(kTaThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ CUtensorMap map_dk, const __grid_constant__ CUtensorMap map_dv,
                     const __grid_constant__ CUtensorMap map_q, const AttendParams p) {
  using S = TcShape<DP>;
  constexpr int NST = S::NST, NSB = S::NSB, NQB = S::NQB, N = S::N, DT = BF ? DT_BF16 : DT_F16;
  extern __shared__ unsigned char ta_raw[];
  __shared__ unsigned long long trees[2][kAtMaxNodes * 12 / 8];  // by turns
  __shared__ float2 join_ml[2][2][kTaM];
  __shared__ uint4 stage[8][32 * 4];
  const uint32_t raw = smem_addr(ta_raw), base = (raw + 1023u) & ~1023u;
  unsigned char* gbase = ta_raw + (base - raw);
  auto bar = [&](int i) { return base + S::BAR + 8u * (uint32_t)i; };
  volatile uint32_t* tmem_at = reinterpret_cast<volatile uint32_t*>(gbase + S::WORDS);
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + S::WORDS + 4);
  // [2] item + 1, by turns of the items that have tiles: one slot's softmax may be one such item ahead of
  // the other's, and any number of items without tiles
  volatile int* bad_values = reinterpret_cast<volatile int*>(gbase + S::WORDS + 8);

  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const int kd = (p.dim + 15) / 16;
  if (tid == 0) {
    for (int i = 0; i < S::NBAR; ++i) {
      const bool weights = i >= S::B_P && i < S::B_O;  // one arrival per warp of the slot's softmax
      const bool all = i == S::B_OE || i == S::B_J || (i >= S::B_TE && i < S::B_TE + 2);  // one per softmax warp
      mbar_init(bar(i), weights ? 4 : all ? 8 : 1);
    }
    *abort = 0;
    bad_values[0] = bad_values[1] = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    __syncwarp();
    tmem_alloc(base + S::WORDS, kTaCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, *tmem_at, 0);
  const Waits wait{abort, p.status, p.spin_limit_ns};
  auto wait_all = [&](int i, int phase) { return (bool)__all_sync(~0u, wait(bar(i), (uint32_t)phase & 1u)); };

  // the softmax threads hold 128 scores each: they get the registers that the other warps do not
  // need (2 * 128 * 208 + 128 * 88 = 384 * 168, the launch's)
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---------------------------------------------------------------- softmax
    const int slot = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane, wg = tid - slot * 128;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t to = lanes + S::O + slot * DP, other_o = lanes + S::O + (slot ^ 1) * DP;
    const float c = p.scale_log2;  // not negative: a negative scale is in Q's sign
    int next_len = blockIdx.x < p.items ? __ldg(p.len + tc_row(p, blockIdx.x)) : 0;
    int jobs_before = 0, tiles_before = 0, joins = 0, active = 0;
    int sums[2] = {0, 0};  // items before in which the slot had a job
    bool ok = true;
    for (unsigned it = blockIdx.x; it < (unsigned)p.items && ok; it += gridDim.x) {
      const TcItem<N> x = tc_item<N>(p, it, next_len);
      const int turn = active & 1;
      if (x.len != next_len && tid == 0) atomicOr(p.status, kDevInternal);
      if (it + gridDim.x < p.items) next_len = __ldg(p.len + tc_row(p, it + gridDim.x));
      const int qn = x.wide ? min(kTaM, x.nq - slot * kTaM) : x.nq;  // queries of the slot
      const int qi = x.i0 + (x.wide ? slot * kTaM : 0) + row;
      const bool mine = row < qn, warp_live = quarter * 32 < qn;
      unsigned long long sees = 0ull;
      if (p.nodes && x.nt > 0) {
        if (!(ok = wait_all(S::B_T + (active & 1), active / 2))) break;
        if (mine) sees = tree_at(trees[active & 1], kAtMaxNodes).mask[p.by_group(qi)];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::B_TE + (active & 1)));
      }
      const bool alive = mine && (!p.nodes || sees != 0);
      const bool dead_any = __any_sync(~0u, mine && !alive);  // (lanes without a query may hold anything)
      float m_run = -INFINITY, l_run = 0.0f;
      for (int j = slot; j < x.jobs; j += 2) {
        const int t = x.tile(j), n = x.keys(t, p.nodes), b = (jobs_before + j) % NSB;
        const uint32_t ts = lanes + b * N;
        const bool draft = x.draft(t);
        if (!(ok = wait_all(S::B_S + b, (jobs_before + j) / NSB))) break;
        tc_fence_after();
        // (only after the scores' wait: it says that the ring's slot has been through its last tile)
        // values of the tile's last 16 keys that lie past the row's end, and infinite and NaN
        // values of drafted tokens, must not meet weights of 0: they are made zero (the latter
        // are added back at the end to the queries that see them)
        if ((n & 15 || (draft && p.nodes > 1)) && (!x.wide || slot == 0)) {
          const int g = tiles_before + t;
          if (!(ok = wait_all(S::B_VF + g % NST, g / NST))) break;
          unsigned char* v = gbase + S::V + (g % NST) * S::TILE;
          const int fill = (16 - (n & 15)) & 15;
          for (int e = wg; e < fill * (DP / 8); e += 128) {
            const int key = n + e / (DP / 8), xx = e % (DP / 8);
            *reinterpret_cast<uint4*>(v + (xx >> 3) * S::PANEL + key * 128 + (xx & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          if (draft && p.nodes > 1) {
            for (int e = wg; e < n * (DP / 8); e += 128) {
              const int key = e / (DP / 8), xx = e % (DP / 8);
              uint4* at = reinterpret_cast<uint4*>(v + (xx >> 3) * S::PANEL + key * 128 + (xx & 7) * 16);
              uint4 d = *at;
              if (clear_non_finite<BF>(d)) {
                *at = d;
                bad_values[turn] = (int)it + 1;
              }
            }
          }
          fence_async_shared();
        }
        __syncwarp();
        // the tile's first CH * 32 keys (the others are past the row's end)
        auto softmax = [&](auto chunks) {
          constexpr int CH = decltype(chunks)::value;
          uint32_t s[CH][32];
#pragma unroll
          for (int k = 0; k < CH; ++k) tmem_ld32_issue(ts + k * 32, s[k]);
          tmem_wait_ld(s[0]);
#pragma unroll
          for (int k = 1; k < CH; ++k) tmem_after_wait(s[k]);
          if (CH < N / 32 || n < N || dead_any || draft) {
#pragma unroll
            for (int k = 0; k < CH; ++k) {
              unsigned see = draft ? (k < 2 ? (unsigned)(sees >> (32 * k)) : 0u) : ~0u;
              if (!alive) see = 0u;
              const int left = n - 32 * k;
              if (left < 32) see &= left <= 0 ? 0u : (1u << left) - 1u;
#pragma unroll
              for (int i = 0; i < 32; ++i) s[k][i] = (see >> i) & 1u ? s[k][i] : 0xff800000u;
            }
          }
          float m4[CH];
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            float a = max3(__uint_as_float(s[k][0]), __uint_as_float(s[k][1]), __uint_as_float(s[k][2]));
            float bb = max3(__uint_as_float(s[k][3]), __uint_as_float(s[k][4]), __uint_as_float(s[k][5]));
#pragma unroll
            for (int i = 6; i < 30; i += 4) {
              a = max3(a, __uint_as_float(s[k][i]), __uint_as_float(s[k][i + 1]));
              bb = max3(bb, __uint_as_float(s[k][i + 2]), __uint_as_float(s[k][i + 3]));
            }
            m4[k] = max3(a, bb, fmaxf(__uint_as_float(s[k][30]), __uint_as_float(s[k][31])));
          }
          float mn = m4[0];
#pragma unroll
          for (int k = 1; k < CH; ++k) mn = fmaxf(mn, m4[k]);
          mn = fmaf(mn, c, -kAtLift<BF>);
          const bool grow = mn > m_run + kTaLazy;  // from -inf at the first finite score
          if (__any_sync(~0u, grow)) {
            const float to_m = fmaxf(m_run, mn), sub = to_m == -INFINITY ? 0.0f : to_m;
            const float f = fast_exp2(m_run - sub);
            m_run = to_m;
            l_run *= f;
            if (j >= 2) {
              // the slot's last product has to end first (it may still run): it frees its buffer
              const int g = jobs_before + j - 2;
              if (!wait_all(S::B_SE + g % NSB, g / NSB)) return false;
              tc_fence_after();
#pragma unroll 1
              for (int k = 0; k < kd * 16; k += 32) {
                uint32_t o[32];
                tmem_ld32_issue(to + k, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st32(to + k, o);
              }
              tmem_wait_st();
            }
          }
          const float sub = m_run == -INFINITY ? 0.0f : m_run;
          const float2 c2 = make_float2(c, c), b2 = make_float2(-sub, -sub);
          float2 l0 = make_float2(0.0f, 0.0f), l1 = l0;
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            uint32_t wt[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = make_float2(__uint_as_float(s[k][2 * i]), __uint_as_float(s[k][2 * i + 1]));
              float2 e = __ffma2_rn(y, c2, b2);
              e.x = fast_exp2(e.x);
              e.y = fast_exp2(e.y);
              if (i & 1)
                l1 = __fadd2_rn(l1, e);
              else
                l0 = __fadd2_rn(l0, e);
              wt[i] = pack_pair<BF>(e.x, e.y);
            }
            tmem_st16(ts + k * 16, wt);
          }
          l_run += (l0.x + l1.x) + (l0.y + l1.y);
          tmem_wait_st();
          return true;
        };
        if (warp_live) {
          ok = n > N / 2 ? softmax(std::integral_constant<int, N / 32>{}) : softmax(std::integral_constant<int, N / 64>{});
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::B_P + b));  // the weights, and the fixed-up values
      }
      // the slot's sums (when the slots share the queries, both slots')
      if (ok && x.jobs > slot) {
        ok = wait_all(S::B_O + slot, sums[slot]);
      }
      // an item of one job: slot 1 keeps pace with it (it says below that the sums are read)
      if (ok && x.jobs == 1 && slot == 1) ok = wait_all(S::B_O, sums[0]);
      const bool joined = !x.wide && x.jobs > 1;
      float f = 1.0f, f_other = 0.0f;
      if (joined && ok) {
        ok = wait_all(S::B_O + (slot ^ 1), sums[slot ^ 1]);
        join_ml[joins & 1][slot][row] = make_float2(m_run, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::B_J));
        ok = ok && wait_all(S::B_J, joins);
        if (ok) {
          const float2 o = join_ml[joins & 1][slot ^ 1][row];
          const float M = fmaxf(m_run, o.x), sub = M == -INFINITY ? 0.0f : M;
          f = fast_exp2(m_run - sub);
          f_other = fast_exp2(o.x - sub);
          l_run = f * l_run + f_other * o.y;
          m_run = M;
        }
        ++joins;
      }
      if (!ok) break;
      tc_fence_after();
      if (warp_live && (x.wide || joined || slot == 0)) {
        const bool zero = mine && l_run == 0.0f;
        if (p.splits == 1) {
          const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
          f *= inv;
          f_other *= inv;
        }
        const bool has_bad = bad_values[turn] == (int)it + 1;
        const bool rare = has_bad || __any_sync(~0u, zero);
        const unsigned char* dv = p.dvalue.data + (long long)x.r * p.dvalue.row + (long long)x.h * p.dvalue.head;
        const long long pr = (((long long)x.r * p.kv_heads + x.h) * p.m + qi) * p.splits + x.split;
        // where this lane's row goes; rows leave through shared memory, 64 bytes of a row by four lanes
        // (a lane storing its own row would touch 32 lines per instruction)
        const long long at = p.splits > 1 ? pr * p.dim * 4 : (mine ? query_offset(p, p.out, x.r, x.h, qi) : 0);
        unsigned char* to_all = p.splits > 1 ? reinterpret_cast<unsigned char*>(p.part_o) : p.out.data;
        uint4* mystage = stage[warp];
        auto store_rows = [&](const uint4 (&v)[4], int byte0, int bytes) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) mystage[lane * 4 + (i ^ ((lane >> 1) & 3))] = v[i];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = i * 8 + (lane >> 2), ch = lane & 3;
            const long long off = __shfl_sync(~0u, at, rr);
            if (quarter * 32 + rr < qn && byte0 + ch * 16 < bytes)
              *reinterpret_cast<uint4*>(to_all + off + byte0 + ch * 16) = mystage[rr * 4 + (ch ^ ((rr >> 1) & 3))];
          }
        };
        if (mine && p.splits > 1 && (!joined || slot == 0)) p.part_ml[pr] = make_float2(m_run, l_run);
#pragma unroll 1
        for (int k = joined ? 32 * slot : 0; k < p.dim; k += joined ? 64 : 32) {
          uint32_t o[32];
          __syncwarp();  // the loads are warp-wide
          if (x.nt > 0) {
            tmem_ld32_issue(to + k, o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          float y[32];
          if (joined) {
            uint32_t o2[32];
            tmem_ld32_issue(other_o + k, o2);
            tmem_wait_ld(o);
            tmem_after_wait(o2);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = fmaf(__uint_as_float(o2[i]), f_other, __uint_as_float(o[i]) * f);
          } else {
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(o[i]) * f;
          }
          if (rare) {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = zero ? 0.0f : y[i];
            if (has_bad)
              for (int nd = 0; nd < p.nodes; ++nd)
                if ((sees >> nd) & 1ull)
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (k + i < p.dim) {
                      const float v = load_elem<DT>(dv + nd * p.dvalue.pos + (k + i) * 2);
                      if (!isfinite(v)) y[i] += v;
                    }
          }
          if (p.splits > 1) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint4 v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[i] = make_uint4(__float_as_uint(y[hf * 16 + 4 * i]), __float_as_uint(y[hf * 16 + 4 * i + 1]),
                                  __float_as_uint(y[hf * 16 + 4 * i + 2]), __float_as_uint(y[hf * 16 + 4 * i + 3]));
              store_rows(v, (k + hf * 16) * 4, p.dim * 4);
            }
          } else {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[i] = make_uint4(pack_pair<BF>(y[8 * i], y[8 * i + 1]), pack_pair<BF>(y[8 * i + 2], y[8 * i + 3]),
                                pack_pair<BF>(y[8 * i + 4], y[8 * i + 5]), pack_pair<BF>(y[8 * i + 6], y[8 * i + 7]));
            store_rows(v, k * 2, p.dim * 2);
          }
        }
      }
      __syncwarp();
      if (x.nt > 0) {
        tc_fence_before();
        if (lane == 0) mbar_arrive(bar(S::B_OE));
        ++active;
        jobs_before += x.jobs;
        tiles_before += x.nt;
        ++sums[0];
        sums[1] += x.jobs > 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    constexpr uint32_t ab = BF ? 1u : 0u;  // instruction descriptors of the products
    constexpr uint32_t id0 = (1u << 4) | (ab << 7) | (ab << 10) | ((uint32_t)(kTaM >> 4) << 24);
    constexpr uint32_t id_s = id0 | ((uint32_t)(S::N >> 3) << 17);
    const uint32_t id_o = id0 | (1u << 16) | ((uint32_t)(kd * 2) << 17);  // N = the head size; B is MN-major
  // Tile t of a walk's item into a ring (keys or values).
  auto load = [&](const TcWalk<N>& w, int t, uint32_t ring, int full, int empty, const CUtensorMap* map,
                  const CUtensorMap* dmap) {
    const TcItem<N>& x = w.x;
    const int g = w.tile + t, st = g % NST;
    if (g >= NST && !wait_all(empty + st, g / NST - 1)) return false;
    if (elect_one()) {
      const bool draft = x.draft(t);
      const int halves = draft || x.keys(t, p.nodes) <= 64 ? 1 : N / 64;
      mbar_arrive_expect_tx(bar(full + st), (uint32_t)(halves * S::PANELS) * (64 * 128));
      for (int c = 0; c < S::PANELS; ++c)
        for (int hf = 0; hf < halves; ++hf) {
          const uint32_t dst = base + ring + st * S::TILE + c * S::PANEL + hf * (64 * 128);
          if (draft)
            tma_load_4d(dst, dmap, c * 64, 0, x.h, x.r, bar(full + st));
          else
            tma_load_4d(dst, map, c * 64, (x.t_lo + t) * N + hf * 64, p.kv_head_one ? 0 : x.h, p.kv_row_one ? 0 : x.r,
                        bar(full + st));
        }
    }
    __syncwarp();
    return true;
  };
  // The ring's copies up to number n land before the CTA may exit (after a run without a lapsed wait
  // they have; after one of another role's they may not).
  auto drain = [&](int n, int slots, int full) {
    for (int g = max(0, n - slots); g < n; ++g) mbar_wait_bounded(bar(full + g % slots), (uint32_t)(g / slots) & 1u, kTaDrainNs);
  };

  if (warp == 8) {
    // ---------------------------------------------------------------- keys and queries
    TcWalk<N> w;
    bool ok = true;
    int kn = 0, qn = 0;  // tiles and query sets asked for
    for (w.begin(p); w.valid && ok; w.next(p)) {
      const TcItem<N>& x = w.x;
      if (!(ok = load(w, 0, S::K, S::B_KF, S::B_KE, &map_k, &map_dk))) break;
      kn = w.tile + 1;
      const int st = w.active % NQB;
      if (w.active >= NQB && !(ok = wait_all(S::B_QE + st, w.active / NQB - 1))) break;
      if (p.q_tma) {
        if (elect_one()) {
          const int slots = x.wide ? 2 : 1, token = p.by_group(x.i0);
          mbar_arrive_expect_tx(bar(S::B_QF + st), (uint32_t)slots * S::QT);
          for (int s = 0; s < slots; ++s)
            for (int c = 0; c < S::PANELS; ++c)
              tma_load_5d(base + S::Q + (2 * st + s) * S::QT + c * kTaPanel, &map_q, c * 64, 0, token + s * p.by_group(kTaM),
                          x.h, x.r, bar(S::B_QF + st));
        }
        __syncwarp();
        qn = w.active + 1;
      } else {  // by asynchronous copies
        const int rows = x.wide ? 2 * kTaM : kTaM;
        auto place = [&](int e) {
          const int qr = e / (DP / 8), ch = e % (DP / 8);
          return S::Q + (2 * st + (qr >> 7)) * S::QT + (ch >> 3) * kTaPanel + (qr & 127) * 128 + (((ch & 7) ^ (qr & 7)) << 4);
        };
        for (int r0 = 0; r0 < rows; r0 += 32) {  // each lane knows one row's address
          const long long mine = r0 + lane < x.nq ? query_offset(p, p.q, x.r, x.h, x.i0 + r0 + lane) : 0;
          for (int e = r0 * (DP / 8) + lane; e < (r0 + 32) * (DP / 8); e += 32) {
            const int qr = e / (DP / 8), ch = e % (DP / 8);
            const long long off = __shfl_sync(~0u, mine, qr - r0);
            const bool there = qr < x.nq && ch * 8 < p.dim;
            cp_async16_fill(base + place(e), there ? p.q.data + off + ch * 16 : p.q.data, there ? 16 : 0);
          }
        }
        cp_async_commit();
        cp_async_wait<0>();
        if (p.negate) {  // a negative scale: the queries' signs, each lane the vectors it copied
          for (int e = lane; e < rows * (DP / 8); e += 32) {
            uint4* v = reinterpret_cast<uint4*>(gbase + place(e));
            *v = make_uint4(v->x ^ 0x80008000u, v->y ^ 0x80008000u, v->z ^ 0x80008000u, v->w ^ 0x80008000u);
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::B_QF + st));
      }
      for (int t = 1; t < x.nt && ok; ++t) {
        ok = load(w, t, S::K, S::B_KF, S::B_KE, &map_k, &map_dk);
        if (ok) kn = w.tile + t + 1;
      }
    }
    drain(kn, NST, S::B_KF);
    drain(qn, NQB, S::B_QF);
  } else if (warp == 9) {
    // ---------------------------------------------------------------- scores
    const uint64_t q0 = desc_k(base + S::Q), k0 = desc_k(base + S::K);
    bool ok = true;
    TcWalk<N> w;
    for (w.begin(p); w.valid && ok; w.next(p)) {
      const TcItem<N>& x = w.x;
      const int qs = w.active % NQB;
      if (!(ok = wait_all(S::B_QF + qs, w.active / NQB))) break;
      for (int j = 0; j < x.jobs; ++j) {
        const int g = w.job + j, b = g % NSB, t = w.tile + x.tile(j), st = t % NST, s = j & 1;
        // the buffer's last weights have been multiplied
        if (g >= NSB && !(ok = wait_all(S::B_SE + b, g / NSB - 1))) break;
        if (!(ok = wait_all(S::B_KF + st, t / NST))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = q0 + (2 * qs + (x.wide ? s : 0)) * (S::QT >> 4), bd = k0 + st * (S::TILE >> 4);
          const uint32_t d = tmem + b * N;
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {  // elements past the head size are zero
            const uint32_t in = 2u * (k & 3);
            umma_f16(d, a + (k >> 2) * (kTaPanel >> 4) + in, bd + (k >> 2) * (S::PANEL >> 4) + in, id_s, k != 0);
          }
          umma_commit(bar(S::B_S + b));
          if (!x.wide || s == 1) umma_commit(bar(S::B_KE + st));
          if (j + 1 == x.jobs) umma_commit(bar(S::B_QE + qs));
        }
        __syncwarp();
      }
    }
    if (elect_one()) umma_commit(bar(S::B_DONE));
    __syncwarp();
    mbar_wait_bounded(bar(S::B_DONE), 0u, kTaDrainNs);
  } else if (warp == 10) {
    // ---------------------------------------------------------------- values
    const uint64_t v0 = desc_mn(base + S::V, S::PANEL);
    bool ok = true;
    TcWalk<N> w;
    for (w.begin(p); w.valid && ok; w.next(p)) {
      const TcItem<N>& x = w.x;
      // the last item's sums are read before the first product of this one replaces them
      if (w.active > 0 && !(ok = wait_all(S::B_OE, w.active - 1))) break;
      for (int j = 0; j < x.jobs && ok; ++j) {
        const int g = w.job + j, b = g % NSB, t = w.tile + x.tile(j), st = t % NST, s = j & 1;
        if (!(ok = wait_all(S::B_VF + st, t / NST))) break;
        const int steps = (x.keys(x.tile(j), p.nodes) + 15) / 16;
        const uint64_t bd = v0 + st * (S::TILE >> 4);
        const uint32_t d = tmem + S::O + s * DP, a = tmem + b * N;
        if (!(ok = wait_all(S::B_P + b, g / NSB))) break;
        tc_fence_after();
        if (elect_one()) {
          if (steps == N / 16) {
#pragma unroll
            for (int k = 0; k < N / 16; ++k) umma_f16_ts(d, a + 8u * k, bd + (uint64_t)k * (2048 >> 4), id_o, j >= 2 || k > 0);
          } else {
            for (int k = 0; k < steps; ++k) umma_f16_ts(d, a + 8u * k, bd + (uint64_t)k * (2048 >> 4), id_o, j >= 2 || k > 0);
          }
          umma_commit(bar(S::B_SE + b));
          if (!x.wide || s == 1) umma_commit(bar(S::B_VE + st));
          if (j + 2 >= x.jobs) umma_commit(bar(S::B_O + s));  // the slot's last product of the item
        }
        __syncwarp();
      }
    }
    if (elect_one()) umma_commit(bar(S::B_DONE + 1));
    __syncwarp();
    mbar_wait_bounded(bar(S::B_DONE + 1), 0u, kTaDrainNs);
  } else {
    // ---------------------------------------------------------------- trees and values
    TcWalk<N> w;
    bool ok = true;
    int vn = 0;
    for (w.begin(p); w.valid && ok; w.next(p)) {
      const TcItem<N>& x = w.x;
      if (p.nodes) {
        const int turn = w.active & 1;
        if (w.active >= 2 && !(ok = wait_all(S::B_TE + turn, w.active / 2 - 1))) break;
        if (tree_seen(tree_at(trees[turn], kAtMaxNodes), p.parent + (long long)x.r * p.nodes, p.nodes, lane, 32,
                      [] { __syncwarp(); }))
          atomicOr(p.status, kDevInternal);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::B_T + turn));
      }
      for (int t = 0; t < x.nt && ok; ++t) {
        ok = load(w, t, S::V, S::B_VF, S::B_VE, &map_v, &map_dv);
        if (ok) vn = w.tile + t + 1;
      }
    }
    drain(vn, NST, S::B_VF);
  }
  }
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTaCols);
  }
}

template <bool BF, int DP>
cudaError_t run_tc(const CUtensorMap (&maps)[5], const AttendParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(attend_tc_kernel<BF, DP>, (int)TcShape<DP>::BYTES, allowed);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(p.items < kAtSms ? p.items : kAtSms);
  attend_tc_kernel<BF, DP><<<grid, kTaThreads, TcShape<DP>::BYTES, stream>>>(maps[0], maps[1], maps[2], maps[3], maps[4], p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_tc(const CUtensorMap (&maps)[5], const AttendParams& p, int dtype, cudaStream_t stream) {
  if (dtype == DT_BF16) return p.dim <= 64 ? run_tc<true, 64>(maps, p, stream) : run_tc<true, 128>(maps, p, stream);
  return p.dim <= 64 ? run_tc<false, 64>(maps, p, stream) : run_tc<false, 128>(maps, p, stream);
}

}  // namespace lsb
