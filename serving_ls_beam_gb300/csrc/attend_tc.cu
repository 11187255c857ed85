// Attention of many queries over a row's keys (f16 / bf16, head size up to 128) on the 5th
// generation tensor cores: forced prefixes and scored targets of a cross attention, trees of
// drafts whose nodes share their key heads.
//
//   S = Q K^T,  P = exp2(c S - max),  O = O * correction + P V,  out = O / sum P
//
// with the running maximum and sum of the softmax (Milakov and Gimelshein, 2018).  One CTA per
// SM, ten warps, tiles of 128 keys:
//   warp 0     TMA producer: two rings of swizzled key and value tiles (64-element panels of
//              128-byte rows); a tile's second 64 keys are not fetched when the row ends before;
//   warp 1     owns the 512 tensor-memory columns; one lane issues S = Q K^T (Q and K from
//              shared memory, M 128, N 128) and O += P V (P from tensor memory, V read as the
//              transposed operand from the same [key][element] tile);
//   warps 2-5, 6-9  the softmax of slot 0 and slot 1: a thread has one query (one lane of tensor
//              memory), reads its 128 scores, and writes its weights over them as 16-bit
//              values (rounded to the tensors' type; sums are of the unrounded f32 weights).
// While one slot's softmax runs, the tensor cores work for the other.  With more than 128
// queries the slots are two tiles of queries over the same key tiles (each tile is fetched once
// for 256 queries); with fewer they are the even and the odd key tiles of the same queries,
// joined through shared memory at the end.
//
// The accumulator is rescaled only when a query's maximum has grown by more than 2^8 since the
// last time: until then its weights are at most 2^8 instead of 1, which f32 sums and the 16-bit
// types hold without loss.  Every wait is bounded: one that runs out sets the timeout bit of the
// status word, and the CTA lets its copies and products finish, frees its tensor memory and
// returns.
#include <cuda.h>

#include "ls_device.cuh"
#include "ls_dtype.cuh"
#include "ls_tc.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

constexpr int kTaThreads = 320;
constexpr int kTaM = 128;   // queries of a slot
constexpr int kTaN = 128;   // keys of a tile
constexpr uint32_t kTaPanel = 128 * 128;  // 128 rows of 64 16-bit elements
constexpr uint32_t kTaCols = 512;
constexpr uint32_t kTaO = 256;            // tensor-memory columns: S of the slots at 0 and 128, O from here
constexpr long long kTaDrainNs = 2000000000LL;
constexpr float kTaLazy = 8.0f;           // growth of the maximum (log2) that is let pass

template <int DP>
struct TcShape {
  static constexpr int PANELS = DP / 64;
  static constexpr int NST = DP == 64 ? 4 : 2;                 // stages of either ring
  static constexpr uint32_t TILE = PANELS * kTaPanel;          // 128 vectors of DP elements
  static constexpr uint32_t Q = 0, K = 2 * TILE, V = K + NST * TILE, BAR = V + NST * TILE;
  static constexpr int NBAR = 4 * NST + 1 + 2 + 4 + 2 + 1;     // full / empty x K / V, q, s, p x halves, o, done
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
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(kTaPanel >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
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
__device__ __forceinline__ void softmax_warps_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

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
      if (mbar_test_wait(bar, parity)) return true;
      if ((n & 255u) == 0) {  // the timer and the flag are slow to read
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

template <bool BF, int DP>
__global__ void __launch_bounds__(kTaThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ CUtensorMap map_dk, const __grid_constant__ CUtensorMap map_dv,
                     const AttendParams p) {
  using S = TcShape<DP>;
  constexpr int NST = S::NST, DT = BF ? DT_BF16 : DT_F16;
  extern __shared__ unsigned char ta_raw[];
  __shared__ unsigned long long tree_raw[kAtMaxNodes * 12 / 8];
  const TreeSeen tree = tree_at(tree_raw, kAtMaxNodes);
  __shared__ float2 join_ml[kTaM];
  const uint32_t raw = smem_addr(ta_raw), base = (raw + 1023u) & ~1023u;
  unsigned char* gbase = ta_raw + (base - raw);
  const uint32_t bars = base + S::BAR;
  auto kfull = [&](int s) { return bars + 8u * s; };
  auto kempty = [&](int s) { return bars + 8u * (NST + s); };
  auto vfull = [&](int s) { return bars + 8u * (2 * NST + s); };
  auto vempty = [&](int s) { return bars + 8u * (3 * NST + s); };
  const uint32_t qfull = bars + 8u * (4 * NST);
  auto sfull = [&](int s) { return bars + 8u * (4 * NST + 1 + s); };
  auto pfull = [&](int s, int half) { return bars + 8u * (4 * NST + 3 + 2 * s + half); };  // 64 keys each
  auto ofull = [&](int s) { return bars + 8u * (4 * NST + 7 + s); };
  const uint32_t done = bars + 8u * (4 * NST + 9);
  volatile uint32_t* tmem_at = reinterpret_cast<volatile uint32_t*>(gbase + S::WORDS);
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + S::WORDS + 4);
  volatile int* bad_values = reinterpret_cast<volatile int*>(gbase + S::WORDS + 8);

  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const int it = (int)blockIdx.x, ia = p.by_split(it), split = it - ia * p.splits, ib = p.by_tile(ia);
  const int i0 = (ia - ib * p.m_tiles) * (2 * kTaM), r = p.by_head(ib), h = ib - r * p.kv_heads;
  const int nq = min(2 * kTaM, p.m - i0);
  const bool wide = nq > kTaM;  // two tiles of queries; otherwise the slots share one
  const int len = __shfl_sync(~0u, row_keys(p, r, tid == 0), 0);  // one value, known to be one
  const int nb = (len + kTaN - 1) / kTaN, nbt = nb + (p.nodes ? 1 : 0);
  const int per = (nbt + p.splits - 1) / p.splits;
  const int t_lo = min(split * per, nbt), nt = min(per, nbt - t_lo);  // this CTA's tiles
  const int jobs0 = wide ? nt : (nt + 1) / 2, jobs1 = wide ? nt : nt / 2;
  auto tile_of = [&](int s, int i) { return wide ? i : 2 * i + s; };
  auto keys_of = [&](int t) { return t_lo + t < nb ? min(kTaN, len - (t_lo + t) * kTaN) : p.nodes; };
  const int kd = (p.dim + 15) / 16;

  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(kfull(s), 1);
      mbar_init(kempty(s), 1);
      mbar_init(vfull(s), 1);
      mbar_init(vempty(s), 1);
    }
    mbar_init(qfull, 8);
    for (int s = 0; s < 2; ++s) {
      mbar_init(sfull(s), 1);
      mbar_init(pfull(s, 0), 4);
      mbar_init(pfull(s, 1), 4);
      mbar_init(ofull(s), 1);
    }
    mbar_init(done, 1);
    *abort = 0;
    *bad_values = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(base + S::WORDS, kTaCols);
    tmem_relinquish();
  }
  if (p.nodes) {
    if (tree_seen(tree, p.parent + (long long)r * p.nodes, p.nodes, tid, kTaThreads, [] { __syncthreads(); }))
      atomicOr(p.status, kDevInternal);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(~0u, *tmem_at, 0);
  const Waits wait{abort, p.status, p.spin_limit_ns};

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------------- producer
      int kn = 0, vn = 0;
      bool ok = true;
      auto load = [&](int t, uint32_t ring, uint32_t full, uint32_t empty, const CUtensorMap* map, const CUtensorMap* dmap,
                      int* count) {
        const int st = t % NST;
        if (t >= NST && !wait(empty, (uint32_t)(t / NST - 1) & 1u)) {
          ok = false;
          return;
        }
        const bool draft = t_lo + t >= nb;
        const int halves = draft || keys_of(t) <= 64 ? 1 : 2;
        mbar_arrive_expect_tx(full, (uint32_t)(halves * S::PANELS) * (kTaPanel / 2));
        for (int c = 0; c < S::PANELS; ++c)
          for (int hf = 0; hf < halves; ++hf) {
            const uint32_t dst = ring + st * S::TILE + c * kTaPanel + hf * (kTaPanel / 2);
            if (draft)
              tma_load_4d(dst, dmap, c * 64, 0, h, r, full);
            else
              tma_load_4d(dst, map, c * 64, (t_lo + t) * kTaN + hf * 64, p.kv_head_one ? 0 : h, p.kv_row_one ? 0 : r, full);
          }
        *count = t + 1;
      };
      for (int t = -1; t < nt && ok; ++t) {
        if (t + 1 < nt) load(t + 1, base + S::K, kfull((t + 1) % NST), kempty((t + 1) % NST), &map_k, &map_dk, &kn);
        if (t >= 0 && ok) load(t, base + S::V, vfull(t % NST), vempty(t % NST), &map_v, &map_dv, &vn);
      }
      if (*abort) {  // every copy issued lands before the CTA may exit
        for (int t = max(0, kn - NST); t < kn; ++t) mbar_wait_bounded(kfull(t % NST), (uint32_t)(t / NST) & 1u, kTaDrainNs);
        for (int t = max(0, vn - NST); t < vn; ++t) mbar_wait_bounded(vfull(t % NST), (uint32_t)(t / NST) & 1u, kTaDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (nt > 0) {
      // ---------------------------------------------------------------- products
      // The whole warp walks the tiles, so that the compiler sees one path and keeps the operands
      // of the products in uniform registers; one elected lane issues them.  (With one lane alone
      // in the loop each product took some 90 cycles to issue, twice what it takes to run.)
      constexpr uint32_t ab = BF ? 1u : 0u;
      constexpr uint32_t id0 = (1u << 4) | (ab << 7) | (ab << 10) | ((uint32_t)(kTaM >> 4) << 24);
      constexpr uint32_t id_s = id0 | ((uint32_t)(kTaN >> 3) << 17);
      const uint32_t id_o = id0 | (1u << 16) | ((uint32_t)(kd * 2) << 17);  // N = the head size; B is MN-major
      const uint64_t q0 = desc_k(base + S::Q), k0 = desc_k(base + S::K), v0 = desc_mn(base + S::V);
      bool ok = wait(qfull, 0);
      auto scores = [&](int s, int i) {
        const int t = tile_of(s, i), st = t % NST;
        if (!(ok = ok && __all_sync(~0u, wait(kfull(st), (uint32_t)(t / NST) & 1u)))) return;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = q0 + (wide ? s : 0) * (S::TILE >> 4), b = k0 + st * (S::TILE >> 4);
          const uint32_t d = tmem + s * kTaN;
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {  // elements past the head size are zero
            const uint32_t off = (uint32_t)(k >> 2) * (kTaPanel >> 4) + 2u * (k & 3);
            umma_f16(d, a + off, b + off, id_s, k != 0);
          }
          umma_commit(sfull(s));
          if (!wide || s == 1) umma_commit(kempty(st));
        }
        __syncwarp();
      };
      auto values = [&](int s, int i, bool last) {
        const int t = tile_of(s, i), st = t % NST;
        if (!(ok = ok && __all_sync(~0u, wait(vfull(st), (uint32_t)(t / NST) & 1u)))) return;
        const int steps = (keys_of(t) + 15) / 16;
        const uint64_t b = v0 + st * (S::TILE >> 4);
        const uint32_t d = tmem + kTaO + s * kTaM, a = tmem + s * kTaN;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // the weights of 64 keys at a time, as they are written
          if (!(ok = ok && __all_sync(~0u, wait(pfull(s, half), (uint32_t)i & 1u)))) return;
          tc_fence_after();
          if (elect_one()) {
            if (steps >= 4 * half + 4) {
#pragma unroll
              for (int k = 4 * half; k < 4 * half + 4; ++k)
                umma_f16_ts(d, a + 8u * k, b + (uint64_t)k * (2048 >> 4), id_o, (i | k) != 0);
            } else {
              for (int k = 4 * half; k < steps; ++k)
                umma_f16_ts(d, a + 8u * k, b + (uint64_t)k * (2048 >> 4), id_o, (i | k) != 0);
            }
            if (half == 1) {
              if (!wide || s == 1) umma_commit(vempty(st));
              if (last) umma_commit(ofull(s));
            }
          }
          __syncwarp();
        }
      };
      scores(0, 0);
      if (ok && jobs1 > 0) scores(1, 0);
      for (int i = 0; i < jobs0 && ok; ++i) {
        values(0, i, i + 1 == jobs0);
        if (ok && i + 1 < jobs0) scores(0, i + 1);
        if (i < jobs1) {
          if (ok) values(1, i, i + 1 == jobs1);
          if (ok && i + 1 < jobs1) scores(1, i + 1);
        }
      }
      if (elect_one()) umma_commit(done);
      __syncwarp();
      mbar_wait_bounded(done, 0u, kTaDrainNs);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax
    const int slot = (warp - 2) >> 2, quarter = warp & 3, row = quarter * 32 + lane, wg = tid - 64 - slot * 128;
    const int qn = wide ? min(kTaM, nq - slot * kTaM) : nq;  // queries of the slot
    const int qi = i0 + (wide ? slot * kTaM : 0) + row;
    const bool mine = row < qn;
    const bool warp_live = quarter * 32 < qn;
    const unsigned long long sees = mine && p.nodes ? tree.mask[p.by_group(qi)] : 0ull;
    const bool alive = mine && (!p.nodes || sees != 0);
    const bool dead_any = __any_sync(~0u, !alive);
    const int njobs = slot ? jobs1 : jobs0;
    bool ok = true;
    if (nt > 0) {
      // the slot's queries into shared memory (half of them each when the slots share a tile)
      // by asynchronous copies, all under way at once
      const int rows = wide ? kTaM : kTaM / 2, r0 = wide ? 0 : slot * (kTaM / 2);
      const uint32_t q_s = base + S::Q + (wide ? slot : 0) * S::TILE;
      for (int e = wg; e < rows * (DP / 8); e += 128) {
        const int qr = r0 + e / (DP / 8), c = e % (DP / 8);
        const bool there = qr < qn && c * 8 < p.dim;
        const unsigned char* src = there ? p.q.data + query_offset(p, p.q, r, h, i0 + (wide ? slot * kTaM : 0) + qr) + c * 16 : p.q.data;
        cp_async16_fill(q_s + (c >> 3) * kTaPanel + qr * 128 + (((c & 7) ^ (qr & 7)) << 4), src, there ? 16 : 0);
      }
      cp_async_commit();
      cp_async_wait<0>();
      if (p.negate) {  // a negative scale: the queries' signs, each thread the vectors it copied
        for (int e = wg; e < rows * (DP / 8); e += 128) {
          const int qr = r0 + e / (DP / 8), c = e % (DP / 8);
          uint4* v = reinterpret_cast<uint4*>(gbase + (q_s - base) + (c >> 3) * kTaPanel + qr * 128 + (((c & 7) ^ (qr & 7)) << 4));
          *v = make_uint4(v->x ^ 0x80008000u, v->y ^ 0x80008000u, v->z ^ 0x80008000u, v->w ^ 0x80008000u);
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
    }
    const uint32_t ts = tmem + ((uint32_t)(quarter * 32) << 16) + slot * kTaN;
    const uint32_t to = tmem + ((uint32_t)(quarter * 32) << 16) + kTaO + slot * kTaM;
    float m_run = -INFINITY, l_run = 0.0f;
    const float c = p.scale_log2;  // not negative: a negative scale is in Q's sign
    // the weights of half a tile (and the fixed-up values) are there for the products
    auto hand_over = [&](int half) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull(slot, half));
    };
    for (int i = 0; i < njobs; ++i) {
      const int t = tile_of(slot, i), n = keys_of(t);
      const bool draft = t_lo + t >= nb;
      if (!__all_sync(~0u, wait(sfull(slot), (uint32_t)i & 1u))) {
        ok = false;
        break;
      }
      tc_fence_after();
      // (only after the scores' wait: it says that the ring's slot has been through its last tile)
      // values of the tile's last 16 keys that lie past the row's end, and infinite and NaN
      // values of drafted tokens, must not meet weights of 0: they are made zero (the latter
      // are added back at the end to the queries that see them)
      if ((n & 15 || (draft && p.nodes > 1)) && (!wide || slot == 0)) {
        if (!__all_sync(~0u, wait(vfull(t % NST), (uint32_t)(t / NST) & 1u))) {
          ok = false;
          break;
        }
        unsigned char* v = gbase + S::V + (t % NST) * S::TILE;
        const int fill = (16 - (n & 15)) & 15;
        for (int e = wg; e < fill * (DP / 8); e += 128) {
          const int key = n + e / (DP / 8), x = e % (DP / 8);
          *reinterpret_cast<uint4*>(v + (x >> 3) * kTaPanel + key * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (draft && p.nodes > 1) {
          for (int e = wg; e < n * (DP / 8); e += 128) {
            const int key = e / (DP / 8), x = e % (DP / 8);
            uint32_t* at = reinterpret_cast<uint32_t*>(v + (x >> 3) * kTaPanel + key * 128 + (x & 7) * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              constexpr uint32_t E = BF ? 0x7f80u : 0x7c00u;
              const uint32_t w = at[j];
              const bool lo = (w & E) == E, hi = (w >> 16 & E) == E;
              if (lo || hi) {
                at[j] = w & (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
                *bad_values = 1;
              }
            }
          }
        }
        fence_async_shared();
      }
      __syncwarp();
      if (warp_live) {
        uint32_t s[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld32_issue(ts + k * 32, s[k]);
        tmem_wait_ld();
        if (n < kTaN || dead_any || draft) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            unsigned see = draft ? (k < 2 ? (unsigned)(sees >> (32 * k)) : 0u) : ~0u;
            if (!alive) see = 0u;
            const int left = n - 32 * k;
            if (left < 32) see &= left <= 0 ? 0u : (1u << left) - 1u;
#pragma unroll
            for (int j = 0; j < 32; ++j) s[k][j] = (see >> j) & 1u ? s[k][j] : 0xff800000u;
          }
        }
        float m4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float a = max3(__uint_as_float(s[k][0]), __uint_as_float(s[k][1]), __uint_as_float(s[k][2]));
          float b = max3(__uint_as_float(s[k][3]), __uint_as_float(s[k][4]), __uint_as_float(s[k][5]));
#pragma unroll
          for (int j = 6; j < 30; j += 4) {
            a = max3(a, __uint_as_float(s[k][j]), __uint_as_float(s[k][j + 1]));
            b = max3(b, __uint_as_float(s[k][j + 2]), __uint_as_float(s[k][j + 3]));
          }
          m4[k] = max3(a, b, fmaxf(__uint_as_float(s[k][30]), __uint_as_float(s[k][31])));
        }
        const float mn = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
        const bool grow = mn > m_run + kTaLazy;  // from -inf at the first finite score
        if (__any_sync(~0u, grow)) {
          const float to_m = fmaxf(m_run, mn), sub = to_m == -INFINITY ? 0.0f : to_m;
          const float f = fast_exp2(m_run - sub);
          m_run = to_m;
          l_run *= f;
          if (i > 0) {
#pragma unroll 1
            for (int k = 0; k < kd * 16; k += 32) {
              uint32_t o[32];
              tmem_ld32_issue(to + k, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st32(to + k, o);
            }
            tmem_wait_st();
          }
        }
        const float sub = m_run == -INFINITY ? 0.0f : m_run;
        const float2 c2 = make_float2(c, c), b2 = make_float2(-sub, -sub);
        float2 l0 = make_float2(0.0f, 0.0f), l1 = l0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 x = make_float2(__uint_as_float(s[k][2 * j]), __uint_as_float(s[k][2 * j + 1]));
            float2 e = __ffma2_rn(x, c2, b2);
            e.x = fast_exp2(e.x);
            e.y = fast_exp2(e.y);
            if (j & 1)
              l1 = __fadd2_rn(l1, e);
            else
              l0 = __fadd2_rn(l0, e);
            w[j] = pack_pair<BF>(e.x, e.y);
          }
          tmem_st16(ts + k * 16, w);
          if (k == 1) {
            tmem_wait_st();
            hand_over(0);
          }
        }
        l_run += (l0.x + l1.x) + (l0.y + l1.y);
        tmem_wait_st();
      } else {
        hand_over(0);
      }
      hand_over(1);
    }
    if (ok && njobs > 0) ok = __all_sync(~0u, wait(ofull(slot), 0u));
    if (!wide && nt > 0) {
      // both slots hold parts of the same queries: slot 1 hands its own over in the key ring
      // (free: both slots' products have ended)
      ok = ok && __all_sync(~0u, wait(ofull(0), 0u));
      float* acc = reinterpret_cast<float*>(gbase + S::K);
      tc_fence_after();
      if (slot == 1 && warp_live) {
        join_ml[row] = make_float2(m_run, l_run);
        if (ok && jobs1 > 0) {
#pragma unroll 1
          for (int k = 0; k < kd * 16; k += 32) {
            uint32_t o[32];
            tmem_ld32_issue(to + k, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (k + j < DP) acc[(k + j) * kTaM + row] = __uint_as_float(o[j]);
          }
        }
      }
      softmax_warps_sync();
    }
    tc_fence_after();
    ok = ok && !*abort;
    if (ok && warp_live && (wide || slot == 0)) {
      float f0 = 1.0f, f1 = 0.0f;
      if (!wide && jobs1 > 0) {
        const float2 other = join_ml[row];
        const float M = fmaxf(m_run, other.x), sub = M == -INFINITY ? 0.0f : M;
        f0 = fast_exp2(m_run - sub);
        f1 = fast_exp2(other.x - sub);
        l_run = f0 * l_run + f1 * other.y;
        m_run = M;
      }
      const float inv = p.splits > 1 ? 1.0f : (l_run == 0.0f ? 0.0f : 1.0f / l_run);
      const bool zero = l_run == 0.0f;
      const float* acc = reinterpret_cast<const float*>(gbase + S::K);
      const AtView& vv = p.dvalue;
      const unsigned char* dv = vv.data + (long long)r * vv.row + (long long)h * vv.head;
      const long long pr = ((((long long)r * p.kv_heads + h) * p.m + qi) * p.splits) + split;
      // a tile of output rows: in the key ring, which no product reads any more once slot 0's last
      // one has ended (all scores were issued before it); joined slots, whose sums lie there, use
      // the value ring
      unsigned char* stage = gbase + (wide ? S::K + slot * S::TILE : S::V);
      if (mine && p.splits > 1) p.part_ml[pr] = make_float2(m_run, l_run);
#pragma unroll 1
      for (int k = 0; k < p.dim; k += 32) {
        uint32_t o[32];
        __syncwarp();  // the loads are warp-wide
        if (nt > 0) {
          tmem_ld32_issue(to + k, o);
          tmem_wait_ld();
        }
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          x[j] = zero ? 0.0f : __uint_as_float(o[j]) * f0;
          if (!wide && jobs1 > 0 && f1 != 0.0f && k + j < DP) x[j] = fmaf(f1, acc[(k + j) * kTaM + row], x[j]);
          x[j] *= inv;
        }
        if (*bad_values) {
          for (int nd = 0; nd < p.nodes; ++nd)
            if ((sees >> nd) & 1ull)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (k + j < p.dim) {
                  const float v = load_elem<DT>(dv + nd * vv.pos + (k + j) * 2);
                  if (!isfinite(v)) x[j] += v;
                }
        }
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          if (p.splits > 1) {
            if (mine && k + j < p.dim) {
              float4* dst = reinterpret_cast<float4*>(p.part_o + pr * p.dim + k + j);
              dst[0] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
              dst[1] = make_float4(x[j + 4], x[j + 5], x[j + 6], x[j + 7]);
            }
          } else {
            const int v = (k + j) / 8;
            if (v < DP / 8)
              *reinterpret_cast<uint4*>(stage + row * (DP * 2) + ((v ^ (row & 7)) << 4)) =
                  make_uint4(pack_pair<BF>(x[j], x[j + 1]), pack_pair<BF>(x[j + 2], x[j + 3]),
                             pack_pair<BF>(x[j + 4], x[j + 5]), pack_pair<BF>(x[j + 6], x[j + 7]));
          }
        }
      }
      if (p.splits == 1) {  // whole rows at a time, the warp's own 32
        __syncwarp();
        const int vecs = p.dim / 8;
        for (int e = lane; e < 32 * (DP / 8); e += 32) {
          const int rr = quarter * 32 + e / (DP / 8), v = e % (DP / 8);
          if (rr < qn && v < vecs)
            *reinterpret_cast<uint4*>(p.out.data + query_offset(p, p.out, r, h, i0 + (wide ? slot * kTaM : 0) + rr) + v * 16) =
                *reinterpret_cast<const uint4*>(stage + rr * (DP * 2) + ((v ^ (rr & 7)) << 4));
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTaCols);
  }
}

template <bool BF, int DP>
cudaError_t run_tc(const CUtensorMap (&maps)[4], const AttendParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(attend_tc_kernel<BF, DP>, (int)TcShape<DP>::BYTES, allowed);
  if (e != cudaSuccess) return e;
  attend_tc_kernel<BF, DP><<<(unsigned)p.items, kTaThreads, TcShape<DP>::BYTES, stream>>>(maps[0], maps[1], maps[2], maps[3], p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_tc(const CUtensorMap (&maps)[4], const AttendParams& p, int dtype, cudaStream_t stream) {
  if (dtype == DT_BF16) return p.dim <= 64 ? run_tc<true, 64>(maps, p, stream) : run_tc<true, 128>(maps, p, stream);
  return p.dim <= 64 ? run_tc<false, 64>(maps, p, stream) : run_tc<false, 128>(maps, p, stream);
}

}  // namespace lsb
