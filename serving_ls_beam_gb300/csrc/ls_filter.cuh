// Sampling with temperature, top-k, top-p and min-p, a setting of its own for each row.
//
// With w(x) = 2^((x - M) log2(e) / T), M the row's maximum, every filter keeps a prefix of the tokens in
// the order (x falling, index rising), so that the three together are one cut: the last kept (x, index).
// The token is then found by a prefix sum in the vocabulary's order.
//
// The row's copy lies in the shared memory of one CTA or of a cluster's; of batches of more rows than the GPU
// holds that way, it is read again from L2.  The cut is found without sorting the row:
//   top-k up to 1000: the k-th largest of the threads' (of many: the vectors') maxima bounds the row's k-th
//     largest from below (the hierarchical method's first pass).  What lies above is a short list; it is
//     sorted, its weights are added up, and the draw is from the list itself where up to 256 tokens are kept.
//   larger top-k: counts of x in 2048 equal steps; the step that holds the k-th is the list.
//   top-p: one pass adds the weights, from f32 alone, in coarse whole numbers to 2048 steps, which says between which
//     steps the limit must be passed; a second one sums them exactly, all and by units (of 32 vectors) above those
//     steps, and lists what lies between.
//   A list that overflows (many equal values) is cut again by the bits of x, and equal values by their indices.
// The token is then found by the sums of the units, and in its unit by a prefix sum.
//
// Weights are whole numbers.  A draw near a border between tokens, and a token near the border of the
// nucleus, turn on the last digits of sums over the whole row: with f32 weights and sums some rows in a
// thousand would get another token than in exact arithmetic, and other orders of summation other
// tokens.  Here w is formed to about 2^-28 of its value (a table of 64 powers and a cubic in f32, the
// exponent's argument as an unevaluated pair, two values to an instruction) and rounded to units of 2^-44 of the
// largest; sums of whole numbers are exact in any order, so one CTA and eight give the same bits.
//
// What bounds it: with a short list the chain of a row's phases (load, bound, list, sort, draw; some 20000 clocks)
// over the four rows that an SM has at once: 1024 rows of 40000 f16, top-k 64, top-p 0.95: 37 us, 0.32 of the copy
// rate (with the row in shared memory, two rows per SM, 57; 512 threads per row 45).  Without top-k the weights: some
// 36 instructions each, once for temperature alone (86 us), and for the nucleus a dozen more and an atomic each (153
// us; formed exactly twice 200, added to the steps in 64 bits one by one 254; 64 rows of 120000 bf16 60 us).  4 rows of
// 40000 f32, eight CTAs each: 10 us.
#pragma once

#include <cooperative_groups.h>

#include "ls_attend.h"
#include "ls_device.cuh"
#include "ls_dtype.cuh"
#include "ls_filter.h"

namespace lsb {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kSfWarps = kSfThreads / 32;
constexpr int kSfBins = 2048;
constexpr int kSfList = 2048;        // entries of the list, in the histogram's place
constexpr int kSfRank = kSfThreads;  // lists up to this are ranked and drawn from; longer ones sorted by exchanges
constexpr int kSfCoarse = kSfThreads;  // steps of the histogram of maxima, one per thread
// The largest top-k that goes by a list alone: more overflow the list too often.  By the list and by the counts, us: of 1024
// rows of 40000 top-k 64 36 and 159, 400 90 and 210, 1000 166 and 223, 2000 233 both (it overflows); 64 rows of 120000
// top-k 1000 62 and 85, 2000 104 and 83; 4 rows of 40000 f32 1000 37 and 43, 2000 52 and 44.
constexpr int kSfListed = 1000;
constexpr int kSfSteps = 64;         // steps of an octave in the table of powers
constexpr float kSfMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number in the low bits
constexpr uint32_t kSfMagicBits = 0x4b400000u;

// 2^(-j / 64) in units of 2^-29, from the exponential's series.
struct PowerTable {
  uint32_t whole[kSfSteps];
  float value[kSfSteps];
};
constexpr double power_of(int j) {
  const double z = -0.693147180559945309417232 * j / kSfSteps;
  double term = 1.0, sum = 1.0;
  for (int i = 1; i < 24; ++i) {
    term *= z / i;
    sum += term;
  }
  return sum * 536870912.0;
}
constexpr PowerTable make_powers() {
  PowerTable t{};
  for (int j = 0; j < kSfSteps; ++j) {
    t.whole[j] = (uint32_t)(power_of(j) + 0.5);
    t.value[j] = (float)power_of(j);
  }
  return t;
}
__device__ const PowerTable c_powers = make_powers();

// What a row's weights are made from.
struct RowScale {
  float top;         // M
  float hi, lo;      // 64 log2(e) / T as a pair
  float t_end;       // from here on a weight is 0
  float per_bin;     // steps of the histogram per 1/64 octave
};

// A cut: tokens with x > value, and those with x == value up to index.
struct Cut {
  float value;
  int index;
  __device__ __forceinline__ bool keeps(float x, int i) const { return x > value || (x == value && i <= index); }
};
__device__ __forceinline__ Cut cut_none() { return Cut{-INFINITY, -1}; }  // (-inf itself is never kept)

// What of a row a pass is about: the steps [lo, hi] of the histogram and the keys [from, to].
struct Range {
  int lo, hi;
  uint32_t from, to;
};

struct Shared {  // fixed part of a CTA's shared memory
  uint2 powers[kSfSteps];   // (less the magic number's bits, which the correction brings along)
  u64 warp_sum[2][kSfWarps];
  float warp_max[kSfWarps];
  u64 publish_sum[4];       // what the cluster's CTAs tell each other, a place per purpose
  float publish_max;
  uint32_t publish_key[2];
  u64 before, limit;        // of the crossing step
  int crossing;
  unsigned listed;          // entries of the list (the first CTA's)
  unsigned threads;         // of this CTA with elements for it
  Cut cut;
  int drawn;                // the list gave the token
  float2 min_cut;           // T ln(min_p), as a pair
  int found, kept, token;
  u64 rest;
};

template <int DT, bool BIAS, bool CL>
struct Sampler {
  static constexpr int E = Traits<DT>::kVec, B = Traits<DT>::kBytes;
  static constexpr int SV = BIAS ? E * 4 : 16;  // bytes of a stored vector
  const FilterParams& p;
  Shared& s;
  unsigned char* store;   // the CTA's share of the row
  u64* unit_sum;          // [units]
  u64* hist;              // [kSfBins], then the list
  u64* sorted;            // [kSfRank], then as many weights, in the order of the tokens
  uint32_t* ranks;        // [kSfRank]
  unsigned short* index_rank;  // [kSfRank]: of the sorted list's entries, their place in the order of the tokens
  int row, rank, lead, vectors, first_vec;
  const unsigned char* base;  // the row's first 16-byte vector
  RowScale sc;
  int tid, warp, lane, flip, turn;

  __device__ __forceinline__ void sync() const {
    if constexpr (CL)
      cg::this_cluster().sync();
    else
      __syncthreads();
  }
  template <class T>
  __device__ __forceinline__ T* at(T* local, int cta) const {
    if constexpr (CL)
      return cg::this_cluster().map_shared_rank(local, cta);
    else
      return local;
  }
  __device__ __forceinline__ int ctas() const { return CL ? p.cluster : 1; }

  // vector v of the CTA's share, from memory: -inf outside the row
  __device__ __forceinline__ uint4 fetch(int v) const {
    const int g = first_vec + v;
    uint4 d = make_uint4(Traits<DT>::kNegInfWord, Traits<DT>::kNegInfWord, Traits<DT>::kNegInfWord, Traits<DT>::kNegInfWord);
    if (g < vectors) {
      d = __ldg(reinterpret_cast<const uint4*>(base) + g);
      if (g == 0 || g == vectors - 1) trim(d, g);
    }
    return d;
  }
  // -inf in what of the row's vector g lies outside the row
  __device__ __forceinline__ void trim(uint4& d, int g) const {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = g * E + e - lead;
      if (i < 0 || i >= p.vocab) set_neg_inf<DT>(d, e);
    }
  }
  __device__ __forceinline__ int index_of(int v, int e) const { return (first_vec + v) * E + e - lead; }
  // A vector as it is kept: its bits, or with a bias the sums as f32.  (NaN needs no care: no comparison
  // holds for it, and a maximum passes it over.)
  struct Vec {
    uint4 d[SV / 16];
  };
  __device__ __forceinline__ Vec with_bias(const uint4& raw, int v) const {
    Vec y;
    if constexpr (!BIAS) {
      y.d[0] = raw;
    } else {
      float x[E];
      unpack<DT>(raw, x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = index_of(v, e);
        if (i >= 0 && i < p.vocab) x[e] += __ldg(p.bias + i);
      }
#pragma unroll
      for (int j = 0; j < E / 4; ++j)
        y.d[j] = make_uint4(__float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]), __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3]));
    }
    return y;
  }
  __device__ __forceinline__ Vec get(int v) const {
    if (!p.resident) return with_bias(fetch(v), v);
    Vec y;
#pragma unroll
    for (int j = 0; j < SV / 16; ++j) y.d[j] = reinterpret_cast<const uint4*>(store + (size_t)v * SV)[j];
    return y;
  }
  __device__ __forceinline__ static void values_of(const Vec& y, float (&x)[E]) {
    if constexpr (!BIAS) {
      unpack<DT>(y.d[0], x);
    } else {
#pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        x[4 * j] = __uint_as_float(y.d[j].x);
        x[4 * j + 1] = __uint_as_float(y.d[j].y);
        x[4 * j + 2] = __uint_as_float(y.d[j].z);
        x[4 * j + 3] = __uint_as_float(y.d[j].w);
      }
    }
  }
  __device__ __forceinline__ static float max_of(const Vec& y) {
    if constexpr (!BIAS && DT == DT_F16) {
      const __half2* h = reinterpret_cast<const __half2*>(&y.d[0]);
      const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
      return fmaxf(-INFINITY, fmaxf(__low2float(m), __high2float(m)));
    } else if constexpr (!BIAS && DT == DT_BF16) {
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&y.d[0]);
      const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
      return fmaxf(-INFINITY, fmaxf(__low2float(m), __high2float(m)));
    } else {
      float x[E], m = -INFINITY;
      values_of(y, x);
#pragma unroll
      for (int e = 0; e < E; ++e) m = fmaxf(m, x[e]);
      return m;
    }
  }

  // ---- weights
  __device__ __forceinline__ float steps_below(float x) const { return __fmul_rn(__fsub_rn(sc.top, x), sc.hi); }
  __device__ __forceinline__ int bin_of(float t) const {  // (to the nearest; rising with t, which is all that counts)
    return (int)(__float_as_uint(__fadd_rn(fminf(t * sc.per_bin, (float)(kSfBins - 1)), kSfMagic)) - kSfMagicBits);
  }
  // The weights of a pair, and its steps below the maximum negated; two values to an instruction where f32 has it.
  __device__ __forceinline__ void weigh(float2 x, u64 (&w)[2], float2& below) const {
    const auto both = [](float a) { return make_float2(a, a); };
    const float2 one = both(-1.0f), top = both(sc.top);
    const float2 d = __ffma2_rn(x, one, top);
    const float2 nt = __fmul2_rn(d, both(-sc.hi));
    // top - x = d + err exactly (Knuth's two-sum), times the pair
    const float2 bb = __fadd2_rn(d, both(-sc.top));
    const float2 err = __ffma2_rn(__fadd2_rn(x, bb), one, __ffma2_rn(__ffma2_rn(bb, one, d), one, top));
    const float2 tl = __fadd2_rn(__ffma2_rn(d, both(sc.hi), nt), __ffma2_rn(d, both(sc.lo), __fmul2_rn(err, both(sc.hi))));
    const float2 nf = __ffma2_rn(nt, one, both(kSfMagic));
    const float2 r = __ffma2_rn(tl, one, __fadd2_rn(__fadd2_rn(nf, both(-kSfMagic)), nt));
    constexpr double ln2 = 0.693147180559945309417232 / kSfSteps;
    const float2 q = __fmul2_rn(r, __ffma2_rn(r, __ffma2_rn(r, both((float)(ln2 * ln2 * ln2 / 6)), both((float)(ln2 * ln2 / 2))), both((float)ln2)));
    const uint32_t n0 = __float_as_uint(nf.x), n1 = __float_as_uint(nf.y);  // (the whole number in the low bits)
    const uint2 p0 = s.powers[n0 & (kSfSteps - 1)], p1 = s.powers[n1 & (kSfSteps - 1)];
    const float2 v = __ffma2_rn(make_float2(__uint_as_float(p0.y), __uint_as_float(p1.y)), q, both(kSfMagic));  // 2^(r / 64) - 1, times the power
    w[0] = placed(p0.x + __float_as_uint(v.x), n0, nt.x);
    w[1] = placed(p1.x + __float_as_uint(v.y), n1, nt.y);
    below = nt;
  }
  __device__ __forceinline__ u64 placed(uint32_t f, uint32_t n, float nt) const {
    const int down = (int)(n / kSfSteps) - (int)(kSfMagicBits / kSfSteps) - p.shift;
    f = nt > -sc.t_end ? f >> max(down, 0) : 0u;
    return (u64)f * (1u << max(-down, 0));
  }
  __device__ __forceinline__ u64 weight(float x) const {
    u64 w[2];
    float2 below;
    weigh(make_float2(x, x), w, below);
    return w[0];
  }

  // ---- sums over the CTA and the cluster; every thread gets the result
  __device__ __forceinline__ static u64 warp_total(u64 v) {  // in pieces whose sums 32 bits hold
    constexpr uint32_t PIECE = (1u << 26) - 1;
    const u64 low = __reduce_add_sync(~0u, (uint32_t)v & PIECE), mid = __reduce_add_sync(~0u, (uint32_t)(v >> 26) & PIECE);
    return low + (mid << 26) + ((u64)__reduce_add_sync(~0u, (uint32_t)(v >> 52)) << 52);
  }
  // inclusive prefix over the CTA's threads
  __device__ __forceinline__ u64 scan(u64 v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 t = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += t;
    }
    u64* sums = s.warp_sum[flip];
    flip ^= 1;  // (two in turn: one barrier each)
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    return v + warp_total(lane < warp ? sums[lane & (kSfWarps - 1)] : 0);
  }
  __device__ __forceinline__ u64 block_total(u64 v) {
    v = warp_total(v);
    u64* sums = s.warp_sum[flip];
    flip ^= 1;
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    return warp_total(lane < kSfWarps ? sums[lane & (kSfWarps - 1)] : 0);
  }
  // the cluster's sum of the CTAs' sums `here` (each the same in all of its threads)
  __device__ __forceinline__ u64 row_sum_of(u64 here) {
    if constexpr (!CL) return here;
    turn ^= 1;  // (two places in turn: whoever writes one again has passed the barrier behind the reads of it)
    if (tid == 0) s.publish_sum[turn] = here;
    sync();
    u64 all = 0;
    for (int c = 0; c < ctas(); ++c) all += *at(&s.publish_sum[turn], c);
    return all;
  }

  // ---- passes over the share: f(v, x) for the vectors of the warp's units, 32 at a time, where one of them
  // holds a value that is `worth` it; done(unit) after each
  template <class Worth, class F, class Done>
  __device__ __forceinline__ void each_unit(Worth worth, F f, Done done) const {
    for (int un = warp; un < p.units; un += kSfWarps) {
      for (int i = 0; i < p.unit_vecs; ++i) {
        const int v = (un * p.unit_vecs + i) * 32 + lane;
        const Vec y = get(v);
        if (!__any_sync(~0u, worth(max_of(y)))) continue;
        float x[E];
        values_of(y, x);
        f(v, x);
      }
      done(un);
    }
  }

  // The row into shared memory, in the order of each_unit; the thread's maximum.  `meanwhile` runs with loads under way.
  template <class F>
  __device__ __forceinline__ float load_row(F meanwhile) {
    float mine = -INFINITY;
    if (!BIAS && p.resident) {  // all of it under way at once
      for (int un = warp; un < p.units; un += kSfWarps)
        for (int i = 0; i < p.unit_vecs; ++i) {
          const int v = (un * p.unit_vecs + i) * 32 + lane, g = first_vec + v;
          if (g < vectors)
            cp_async16_fill(smem_addr(store + (size_t)v * 16), base + (size_t)g * 16, 16);
          else
            reinterpret_cast<uint4*>(store)[v] = make_uint4(Traits<DT>::kNegInfWord, Traits<DT>::kNegInfWord, Traits<DT>::kNegInfWord, Traits<DT>::kNegInfWord);
        }
      cp_async_commit();
      meanwhile();
      cp_async_wait<0>();
      for (int un = warp; un < p.units; un += kSfWarps)
        for (int i = 0; i < p.unit_vecs; ++i) {
          const int v = (un * p.unit_vecs + i) * 32 + lane, g = first_vec + v;
          uint4 d = reinterpret_cast<const uint4*>(store)[v];
          if (g == 0 || g == vectors - 1) {
            trim(d, g);
            reinterpret_cast<uint4*>(store)[v] = d;
          }
          mine = fmaxf(mine, max_of(with_bias(d, v)));
        }
      return mine;
    }
    constexpr int AHEAD = 5;
    bool first = true;
    int un = warp, i = 0;  // of the next group of 32 vectors
    while (un < p.units) {
      uint4 d[AHEAD];
      int v[AHEAD];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        v[a] = un < p.units ? (un * p.unit_vecs + i) * 32 + lane : -1;
        if (un < p.units) d[a] = fetch(v[a]);
        if (++i == p.unit_vecs) {
          i = 0;
          un += kSfWarps;
        }
      }
      if (first) meanwhile();
      first = false;
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        if (v[a] < 0) break;
        const Vec y = with_bias(d[a], v[a]);
        mine = fmaxf(mine, max_of(y));
        if (p.resident) {
#pragma unroll
          for (int j = 0; j < SV / 16; ++j) reinterpret_cast<uint4*>(store + (size_t)v[a] * SV)[j] = y.d[j];
        }
      }
    }
    if (first) meanwhile();  // (no unit of the row is the warp's)
    return mine;
  }

  // ---- the histogram
  __device__ __forceinline__ void clear_hist() {
    for (int i = tid; i < kSfBins; i += kSfThreads) hist[i] = 0;
    __syncthreads();
  }
  __device__ __forceinline__ void add_to(int bin, u64 v) {  // two 32-bit halves, the carry by hand
    uint32_t* h = reinterpret_cast<uint32_t*>(hist + bin);
    const uint32_t low = (uint32_t)v, old = atomicAdd(h, low);
    const uint32_t high = (uint32_t)(v >> 32) + (old + low < old);
    if (high) atomicAdd(h + 1, high);
  }
  // The first step at which `base` and the steps up to it reach `limit` (or the last), and the sum before it.
  __device__ __forceinline__ void cross(u64 base_sum, u64 limit, int& bin, u64& before) {
    sync();
    if (rank == 0) {
      constexpr int PER = kSfBins / kSfThreads;
      u64 h[PER], mine = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) h[i] = 0;
      for (int c = 0; c < ctas(); ++c) {
        const u64* from = at(hist, c) + tid * PER;
#pragma unroll
        for (int i = 0; i < PER; ++i) h[i] += from[i];
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) mine += h[i];
      const u64 upto = scan(mine) + base_sum, from = upto - mine;
      if (tid == kSfThreads - 1 && upto < limit) {  // not reached: the last step
        s.crossing = kSfBins - 1;
        s.before = upto - h[PER - 1];
      }
      if (upto >= limit && from < limit) {
        u64 run = from;
        int b = tid * PER;
        for (int i = 0; i < PER; ++i) {
          if (run + h[i] >= limit) {
            b = tid * PER + i;
            break;
          }
          run += h[i];
        }
        s.crossing = b;
        s.before = run;
      }
    }
    sync();
    bin = *at(&s.crossing, 0);
    before = *at(&s.before, 0);
    sync();  // (the steps are read; the list may take their place)
  }

  // ---- the list, in the first CTA's shared memory
  __device__ __forceinline__ bool in_range(float x, int i, const Range& g, const Cut& within) const {
    const float t = steps_below(x);
    if (!(t < sc.t_end)) return false;
    const int b = bin_of(t);
    const uint32_t key = float_ord(x);
    return b >= g.lo && b <= g.hi && key >= g.from && key <= g.to && within.keeps(x, i);
  }
  __device__ __forceinline__ static u64 list_key(float x, int i) { return (u64)~float_ord(x) << 32 | (uint32_t)i; }
  __device__ __forceinline__ static float list_x(u64 key) { return ord_float(~(uint32_t)(key >> 32)); }
  // The elements that `hit` says, of the vectors with a maximum `worth` it; their number (which may be more than the
  // list holds) is in the first CTA's `listed` after a barrier.
  template <class Worth, class Hit>
  __device__ __forceinline__ void gather(Worth worth, Hit hit) {
    u64* list = at(hist, 0);
    unsigned* listed = at(&s.listed, 0);
    each_unit(
        worth,
        [&](int v, const float(&x)[E]) {
          unsigned hits = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) hits |= (hit(x[e], index_of(v, e)) ? 1u : 0u) << e;
          if (hits) {
            unsigned to = atomicAdd(listed, (unsigned)__popc(hits));
#pragma unroll
            for (int e = 0; e < E; ++e)
              if ((hits >> e) & 1u) {
                if (to < kSfList) list[to] = list_key(x[e], index_of(v, e));
                ++to;
              }
          }
        },
        [](int) {});
  }

  // The elements from `bound` on: the threads with such a maximum are put in a row, and their vectors shared out.
  __device__ __forceinline__ unsigned gather_from(float bound, float mine) {
    u64* list = at(hist, 0);
    unsigned* listed = at(&s.listed, 0);
    const unsigned has = __ballot_sync(~0u, mine >= bound);
    unsigned to = 0;
    if (lane == 0 && has) to = atomicAdd(&s.threads, (unsigned)__popc(has));
    to = __shfl_sync(~0u, to, 0) + __popc(has & ((1u << lane) - 1u));
    if (mine >= bound) ranks[to] = tid;
    __syncthreads();
    const unsigned per = p.thread_vecs, all = s.threads * per;
    constexpr int AHEAD = BIAS ? 2 : 3;  // (where the row is not in shared memory, loads from L2)
    for (unsigned n0 = tid; n0 < all; n0 += kSfThreads * AHEAD) {
      Vec y[AHEAD];
      int v[AHEAD];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const unsigned n = n0 + a * kSfThreads;
        v[a] = -1;
        if (n >= all) continue;
        const unsigned who = fast_div(n, p.thread_magic, p.thread_shift), k = n - who * per, of = ranks[who];
        unsigned un = of / 32 + k * kSfWarps, i = 0;
        if (p.unit_vecs > 1) {
          un = of / 32 + k / p.unit_vecs * kSfWarps;
          i = k % p.unit_vecs;
        }
        if (un < (unsigned)p.units) {
          v[a] = (int)(un * p.unit_vecs + i) * 32 + (int)(of & 31);
          y[a] = get(v[a]);
        }
      }
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        if (v[a] < 0 || !(max_of(y[a]) >= bound)) continue;
        float x[E];
        values_of(y[a], x);
        unsigned hits = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) hits |= (x[e] >= bound && x[e] > -INFINITY ? 1u : 0u) << e;
        unsigned put = hits ? atomicAdd(listed, (unsigned)__popc(hits)) : 0u;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((hits >> e) & 1u) {
            if (put < kSfList) list[put] = list_key(x[e], index_of(v[a], e));
            ++put;
          }
      }
    }
    sync();
    return *listed;
  }

  // The list in order, by the first CTA: where it lies then.
  __device__ __forceinline__ const u64* sort_list(unsigned n) {
    if (n <= kSfRank) {  // ranked: several threads to an entry, each counting those before it in a part of the list
      unsigned wide = 32;  // entries, to a power of two
      while (wide < n) wide <<= 1;
      const unsigned i = tid & (wide - 1), parts = kSfThreads / wide, part = tid / wide, step = (n + parts - 1) / parts;
      if (tid < n) ranks[tid] = 0;
      __syncthreads();
      if (i < n) {
        const u64 mine = hist[i];
        unsigned by_value = 0, by_index = 0;
        const unsigned last = min((part + 1) * step, n);
#pragma unroll 4
        for (unsigned j = part * step; j < last; ++j) {
          const u64 other = hist[j];
          by_value += other < mine;
          by_index += (uint32_t)other < (uint32_t)mine;
        }
        if (by_value | by_index) atomicAdd(&ranks[i], by_value << 16 | by_index);
      }
      __syncthreads();
      if (tid < n) {
        sorted[ranks[tid] >> 16] = hist[tid];
        index_rank[ranks[tid] >> 16] = (unsigned short)ranks[tid];
      }
      __syncthreads();
      return sorted;
    }
    unsigned most = kSfRank;
    while (most < n) most <<= 1;
    for (unsigned i = n + tid; i < most; i += kSfThreads) hist[i] = ~0ull;  // last
    __syncthreads();
    for (unsigned size = 2; size <= most; size <<= 1)  // bitonic
      for (unsigned gap = size >> 1; gap; gap >>= 1) {
        for (unsigned t = tid; t < most / 2; t += kSfThreads) {
          const unsigned i = 2 * t - (t & (gap - 1)), j = i + gap;
          const u64 a = hist[i], b = hist[j];
          if ((a > b) == ((i & size) == 0)) {
            hist[i] = b;
            hist[j] = a;
          }
        }
        __syncthreads();
      }
    return hist;
  }
  static constexpr int kPer = kSfList / kSfThreads;
  // A thread's entries of the sorted list: one, or kPer next to each other.
  __device__ __forceinline__ static unsigned entries(unsigned n) { return n <= kSfRank ? 1 : kPer; }

  // The list's first entry at which the count reaches k or the weight `limit`, as the cut.
  __device__ __forceinline__ Cut finish_list(unsigned n, u64 base_count, u64 k, u64 base_sum, u64 limit) {
    if (rank == 0) {
      const u64* keys = sort_list(n);
      const unsigned per = entries(n), first = tid * per;
      u64 w[kPer], mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        w[i] = i < per && first + i < n && limit != ~0ull ? weight(list_x(keys[first + i])) : 0;
        mine += w[i];
      }
      if (tid == 0) s.found = (int)n - 1;
      u64 run = scan(mine) + base_sum - mine;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        run += w[i];
        if (i < per && first + i < n && (base_count + first + i + 1 >= k || run >= limit)) {
          atomicMin(&s.found, (int)(first + i));
          break;
        }
      }
      __syncthreads();
      if (tid == 0) {
        const u64 key = keys[max(s.found, 0)];
        s.cut = n ? Cut{list_x(key), (int)(uint32_t)key} : cut_none();
      }
    }
    sync();
    const Cut c = *at(&s.cut, 0);
    sync();
    return c;
  }

  // A kept token's weight to the sum of its unit.
  __device__ __forceinline__ void add_to_unit(uint32_t index, u64 w) const {
    const int vec = (int)((index + (unsigned)lead) / E), share = p.units * p.unit_vecs * 32, cta = CL ? vec / share : 0;
    atomicAdd(at(unit_sum, cta) + (vec - cta * share) / (32 * p.unit_vecs), w);
  }
  __device__ __forceinline__ void clear_units() const {
    for (int i = tid; i < p.units; i += kSfThreads) unit_sum[i] = 0;
  }
  // All filters on a list that holds the row's first k tokens: true where few are kept, with the token drawn; otherwise
  // the cut, and the units' sums (zero before) of what is kept.
  __device__ __forceinline__ bool draw_list(unsigned n, unsigned k, float top_p, float least, float u, Cut& cut) {
    if (rank == 0) {
      const u64* keys = sort_list(n);
      const unsigned per = entries(n), first = tid * per;
      n = min(n, k);
      u64 w[kPer], mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        w[i] = i < per && first + i < n ? weight(list_x(keys[first + i])) : 0;
        mine += w[i];
      }
      u64* weights = sorted + kSfRank;
      if (per == 1) weights[tid] = 0;
      if (tid == 0) s.kept = 0;
      const u64 upto = scan(mine);
      if (tid == kSfThreads - 1) s.limit = top_p < 1.0f ? share_of(top_p, upto) : ~0ull;
      __syncthreads();
      const u64 limit = s.limit;
      u64 run = upto - mine;
      unsigned keep = 0;  // this thread's kept entries: those that begin before the limit is reached
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (i < per && first + i < n && run < limit && list_x(keys[first + i]) >= least) ++keep;
        run += w[i];
      }
      keep = __reduce_add_sync(~0u, keep);
      if (lane == 0 && keep) atomicAdd(&s.kept, (int)keep);
      __syncthreads();
      const unsigned kept = s.kept;
      if (kept <= kSfRank && per == 1) {
        // the kept weights in the order of the tokens, and the first sum past the target
        if (tid < kept) {
          weights[index_rank[tid]] = mine;
          ranks[index_rank[tid]] = (uint32_t)keys[tid];
        }
        if (tid == kept - 1) s.rest = upto;
        __syncthreads();
        const u64 all = s.rest, here = weights[tid], up = scan(here);
        bool cut_off;
        const u64 target = min(part_of(u, all, cut_off), all - 1);
        if (up > target && up - here <= target) write((int)ranks[tid], here, all);
        if (tid == 0) s.drawn = 1;
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i < per && first + i < kept && w[i]) add_to_unit((uint32_t)keys[first + i], w[i]);
        if (tid == 0) {
          const u64 key = keys[max((int)kept - 1, 0)];
          s.cut = Cut{list_x(key), (int)(uint32_t)key};
          s.drawn = 0;
        }
      }
    }
    sync();
    const bool drawn = *at(&s.drawn, 0);
    cut = *at(&s.cut, 0);
    if (CL && drawn) sync();  // (the first CTA stays until this is read)
    return drawn;
  }
  __device__ __forceinline__ void write(int token, u64 w, u64 all) const {
    p.out_token[row] = token;
    // (near 1 from what is missing; f32 quotients of the exact sums, three roundings: 2^-22 absolute with the logarithm's own)
    if (p.out_logprob) p.out_logprob[row] = w > all / 2 ? log1pf(-((float)(all - w) / (float)all)) : logf((float)w / (float)all);
  }
  // f * all, f in [0, 1], rounded down to a whole number; rest: whether anything was cut off.  (f is a whole
  // number of 24 bits times a power of two: the product is exact, and FP64 is slow on this part.)
  __device__ __forceinline__ static u64 part_of(float f, u64 all, bool& rest) {
    const uint32_t bits = __float_as_uint(f), exponent = bits >> 23;
    const u64 whole = exponent ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const int down = 150 - (int)max(exponent, 1u);  // f = whole / 2^down, 23 <= down <= 149
    const u64 high = __umul64hi(all, whole), low = all * whole;
    if (down >= 128) {
      rest = (high | low) != 0;
      return 0;
    }
    if (down >= 64) {
      rest = low != 0 || (high & ((1ull << (down - 64)) - 1)) != 0;
      return high >> (down - 64);
    }
    rest = (low & ((1ull << down) - 1)) != 0;
    return high << (64 - down) | low >> down;
  }
  __device__ __forceinline__ static u64 share_of(float f, u64 all) {  // the least whole number >= f * all, 1 at least
    bool rest;
    const u64 n = part_of(f, all, rest) + rest;
    return min(max(n, 1ull), all);
  }

  // ---- the first token, in the vocabulary's order, at which the sum of f passes `target` (below the sum of all);
  // unit_sum holds the units' sums, `mine` this CTA's.  Every thread gets the token, and its f in value.
  template <class F>
  __device__ __forceinline__ int locate(F f, u64 mine, u64 target, u64& value) {
    __syncthreads();
    if (tid == 0) {
      s.publish_sum[2] = mine;
      s.found = -1;
      s.token = -1;
    }
    sync();
    u64 before = 0;
    int owner = 0;
    for (int c = 0; c < ctas(); ++c) {
      const u64 here = *at(&s.publish_sum[2], c);
      owner = c;
      if (before + here > target || c == ctas() - 1) break;
      before += here;
    }
    if (owner == rank) {
      // each thread a run of units
      const int per = (p.units + kSfThreads - 1) / kSfThreads, u0 = tid * per, u1 = min(u0 + per, p.units);
      u64 sum = 0;
      for (int i = u0; i < u1; ++i) sum += unit_sum[i];
      const u64 upto = scan(sum) + before;
      if (upto > target && upto - sum <= target) {
        u64 run = upto - sum;
        int i = u0;
        while (i < u1 - 1 && run + unit_sum[i] <= target) run += unit_sum[i++];
        s.found = i;
        s.rest = target - run;
      }
      __syncthreads();
      const int un = s.found;
      if (warp == 0 && un >= 0) {
        u64 rest = s.rest;
        for (int i = 0; i < p.unit_vecs; ++i) {
          const int v = (un * p.unit_vecs + i) * 32 + lane;
          float x[E];
          values_of(get(v), x);
          u64 w[E], sum2 = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            w[e] = f(x[e], index_of(v, e));
            sum2 += w[e];
          }
          u64 up = sum2;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const u64 t = __shfl_up_sync(~0u, up, o);
            if (lane >= o) up += t;
          }
          const u64 all = __shfl_sync(~0u, up, 31);
          if (all > rest) {
            if (up > rest && up - sum2 <= rest) {
              u64 run = up - sum2;
#pragma unroll
              for (int e = 0; e < E; ++e) {
                if (run <= rest && run + w[e] > rest) {
                  s.publish_sum[3] = w[e];
                  s.token = index_of(v, e);
                }
                run += w[e];
              }
            }
            break;
          }
          rest -= all;
        }
      }
    }
    sync();
    const int token = *at(&s.token, owner);
    value = *at(&s.publish_sum[3], owner);
    sync();
    return token;
  }

  // The units' sums of what f says of their vectors; the CTA's sum for every thread.
  template <class Worth, class F>
  __device__ __forceinline__ u64 sum_units(Worth worth, F f) {
    u64 run = 0, all = 0;
    each_unit(
        worth,
        [&](int v, const float(&x)[E]) { run += f(v, x); },
        [&](int un) {
          const u64 t = __any_sync(~0u, run != 0) ? warp_total(run) : 0;
          if (lane == 0) unit_sum[un] = t;
          all += t;
          run = 0;
        });
    return block_total(lane == 0 ? all : 0);
  }

  // Of a long list only the entries among which the sum from `base_sum` on reaches `limit` are left (their number is
  // returned, with base_sum what lies before them); the weights of those before go to their units.  By steps of the
  // keys' bits, one per thread; the first CTA's threads.
  __device__ __forceinline__ unsigned narrow_list(unsigned n, u64 limit, u64& base_sum) {
    constexpr int STEPS = kSfThreads, MINE = kSfList / kSfThreads, PIECE = 21;
    static_assert(3 * STEPS * 4 <= 2 * kSfRank * 8 && kSfList <= 1 << (32 - PIECE), "the sums' pieces");
    auto* sums = reinterpret_cast<uint32_t*>(sorted);  // [3][STEPS], of 21 bits each: whole words are added natively
    uint32_t least = ~0u, most = 0;
    u64 mine[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const unsigned at_n = i * kSfThreads + tid;
      mine[i] = at_n < n ? hist[at_n] : ~0ull;
      if (at_n < n) {
        least = min(least, (uint32_t)(mine[i] >> 32));
        most = max(most, (uint32_t)(mine[i] >> 32));
      }
    }
    least = __reduce_min_sync(~0u, least);
    most = __reduce_max_sync(~0u, most);
    if (tid == 0) {
      s.publish_key[0] = ~0u;
      s.publish_key[1] = 0;
      s.crossing = STEPS - 1;
      s.kept = 0;
    }
    for (int i = tid; i < 3 * STEPS; i += kSfThreads) sums[i] = 0;
    __syncthreads();
    if (lane == 0) {
      atomicMin(&s.publish_key[0], least);
      atomicMax(&s.publish_key[1], most);
    }
    __syncthreads();
    least = s.publish_key[0];
    const uint32_t wide = s.publish_key[1] - least;
    int down = 0;
    while (wide >> down >= (uint32_t)STEPS) ++down;
    // (the keys rise as x falls)
#pragma unroll
    for (int i = 0; i < MINE; ++i)
      if (i * kSfThreads + tid < n) {
        const u64 w = weight(list_x(mine[i]));
        uint32_t* to = sums + (((uint32_t)(mine[i] >> 32) - least) >> down);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const uint32_t piece = (uint32_t)(w >> (k * PIECE)) & ((1u << PIECE) - 1);
          if (piece) atomicAdd(to + k * STEPS, piece);
        }
      }
    __syncthreads();
    const u64 here = sums[tid] + ((u64)sums[STEPS + tid] << PIECE) + ((u64)sums[2 * STEPS + tid] << (2 * PIECE));
    const u64 run = scan(here) - here + base_sum;
    if (run < limit && run + here >= limit) {
      s.crossing = tid;
      s.rest = run;
    }
    if (tid == kSfThreads - 1 && run + here < limit) s.rest = run;  // not reached: the last step
    __syncthreads();
    const uint32_t crossing = s.crossing;
    base_sum = s.rest;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      if (i * kSfThreads + tid >= n) continue;
      const uint32_t step = ((uint32_t)(mine[i] >> 32) - least) >> down;
      if (step < crossing) {
        const u64 w = weight(list_x(mine[i]));
        if (w) add_to_unit((uint32_t)mine[i], w);
      } else if (step == crossing) {
        hist[atomicAdd(&s.kept, 1)] = mine[i];
      }
    }
    __syncthreads();
    return s.kept;
  }

  // The nucleus of the tokens `within`: the cut, and the units' sums of what is kept.  False where equal values are so
  // many that it takes select(), which gives the cut alone.
  //
  // One pass counts the weights in coarse whole numbers in the histogram's steps (2^-31 of an upper bound of the sum).
  // They are formed in f32 alone: t carries four roundings (64 log2(e), its quotient by T, the difference, the product),
  // of up to 32 octaves 4 * 2^-24 * 32 = 2^-17 octaves; the exponent below 32 one more of 2^-20; the power is good to
  // 2^-22: (2^-17 + 2^-20) ln 2 + 2^-22 = 0.9 * 2^-17 of a weight.  And cut to a whole number each loses less than one.
  // So the steps between which the limit must be passed are known, few of them.  A second pass sums the weights exactly, of
  // everything and of the units above those steps, and lists what lies in them.
  template <bool ALL>  // within is everything
  __device__ __forceinline__ bool nucleus(float top_p, const Cut& within, Cut& cut) {
    auto* steps = reinterpret_cast<uint32_t*>(hist);
    for (int i = tid; i < kSfBins; i += kSfThreads) steps[i] = 0;
    // a vector's elements weigh at most its maximum each
    float most = 0.0f;
    for (int un = warp; un < p.units; un += kSfWarps)
      for (int i = 0; i < p.unit_vecs; ++i)
        most += fast_exp2(-fminf(steps_below(max_of(get((un * p.unit_vecs + i) * 32 + lane))), sc.t_end) * (1.0f / kSfSteps));
    // (2^12 to one, rounded up, so that whole numbers can be added up)
    const u64 bound = row_sum_of(block_total((u64)(most * 4096.0f) + 1)) * E;
    const int down = max(64 - __clzll((long long)bound) - 12 + 29 + p.shift - 31, 0);
    const float unit = (float)(29 + p.shift - down);  // a weight of 1 in coarse whole numbers is 2^unit
    each_unit([&](float top) { return top >= within.value && steps_below(top) < sc.t_end; },
              [&](int v, const float(&x)[E]) {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                  const auto both = [](float y) { return make_float2(y, y); };
                  const float2 t = __fmul2_rn(__ffma2_rn(make_float2(x[e], x[e + 1]), both(-1.0f), both(sc.top)), both(sc.hi));
                  const float2 y = __ffma2_rn(t, both(-1.0f / kSfSteps), both(unit));
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    if (!ALL && !within.keeps(x[e + k], index_of(v, e + k))) continue;
                    const uint32_t coarse = __float2uint_rz(fast_exp2(k ? y.y : y.x));  // (NaN: 0)
                    if (coarse) atomicAdd(steps + bin_of(k ? t.y : t.x), coarse);
                  }
                }
              },
              [](int) {});
    if (tid == 0) s.listed = 0;
    sync();
    if (rank == 0) {
      constexpr int PER = kSfBins / kSfThreads;
      u64 h[PER], here = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) h[i] = 0;
      for (int c = 0; c < ctas(); ++c) {
        const uint4* from = reinterpret_cast<const uint4*>(at(steps, c) + tid * PER);
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
          const uint4 y = from[i];
          h[4 * i] += y.x;
          h[4 * i + 1] += y.y;
          h[4 * i + 2] += y.z;
          h[4 * i + 3] += y.w;
        }
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) here += h[i];
      if (tid == 0) {
        s.found = kSfBins - 1;
        s.kept = kSfBins - 1;
      }
      u64 run = scan(here) - here;
      // what the whole numbers' sum is at least and at most where the coarse one's is c
      const auto at_least = [&](u64 c) { return (u64)max((long long)(c - (c >> 17)) - (p.vocab >> down) - 1, 0ll); };
      const auto at_most = [&](u64 c) { return c + (c >> 17) + p.vocab + (p.vocab >> 17) + 2; };  // (what was cut off is as uncertain)
      const u64 all = block_total(here);
      bool cut_off;
      const u64 maybe = part_of(top_p, at_least(all), cut_off), sure = part_of(top_p, at_most(all), cut_off) + 2;
#pragma unroll
      for (int i = 0; i < PER; ++i) {  // passed at this step: possibly, certainly
        run += h[i];
        if (at_most(run) >= maybe) atomicMin(&s.found, tid * PER + i);
        if (at_least(run) >= sure) atomicMin(&s.kept, tid * PER + i);
      }
    }
    sync();
    const int lo = *at(&s.found, 0), hi = *at(&s.kept, 0);
    // as bounds of t, a little wider: what lies above is above in the steps too, what lies below below
    const float t_lo = lo > 0 ? __fdiv_rn((float)lo - 0.5f, sc.per_bin) * (1.0f - 0x1p-20f) : -1.0f;
    const float t_hi = hi < kSfBins - 1 ? __fdiv_rn((float)hi + 0.5f, sc.per_bin) * (1.0f + 0x1p-20f) : INFINITY;
    u64* list = hist;  // (in the place of the steps, which the first CTA has read)
    unsigned* listed = &s.listed;
    u64 run = 0, all = 0, total = 0;
    each_unit(
        [&](float top) { return top >= within.value && steps_below(top) < sc.t_end; },
        [&](int v, const float(&x)[E]) {
          unsigned hits = 0;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            u64 w[2];
            float2 below;
            weigh(make_float2(x[e], x[e + 1]), w, below);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float t = -(k ? below.y : below.x);
              if (!(t < sc.t_end) || (!ALL && !within.keeps(x[e + k], index_of(v, e + k)))) continue;
              total += w[k];
              if (t < t_lo)
                run += w[k];
              else if (t <= t_hi)
                hits |= 1u << (e + k);
            }
          }
          if (hits) {
            unsigned to = atomicAdd(listed, (unsigned)__popc(hits));
#pragma unroll
            for (int e = 0; e < E; ++e)
              if ((hits >> e) & 1u) {
                if (to < kSfList) list[to] = list_key(x[e], index_of(v, e));
                ++to;
              }
          }
        },
        [&](int un) {
          const u64 t = __any_sync(~0u, run != 0) ? warp_total(run) : 0;
          if (lane == 0) unit_sum[un] = t;
          all += t;
          run = 0;
        });
    all = block_total(lane == 0 ? all : 0);
    if (CL && rank != 0) {  // each CTA's list behind the first's (entry by entry, every one would wait for the other SM)
      const unsigned n = *listed;
      if (tid == 0) s.kept = (int)atomicAdd(at(&s.listed, 0), n);
      __syncthreads();
      const unsigned to = s.kept;
      for (unsigned i = tid; i < min(n, (unsigned)kSfList) && to + i < kSfList; i += kSfThreads) at(hist, 0)[to + i] = list[i];
    }
    const u64 above = row_sum_of(all);
    const u64 limit = share_of(top_p, row_sum_of(block_total(total)));
    if constexpr (!CL) __syncthreads();  // (in a cluster the sum has had its barrier)
    const unsigned n = *at(&s.listed, 0);
    if (n > kSfList) {
      sync();
      cut = select<true>(limit, within);
      return false;
    }
    if (rank == 0) {
      u64 base_sum = above;
      const unsigned left = n > kSfRank ? narrow_list(n, limit, base_sum) : n;
      const u64* keys = sort_list(left);
      const unsigned per = entries(left), first = tid * per;
      u64 w[kPer], here = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        w[i] = i < per && first + i < left ? weight(list_x(keys[first + i])) : 0;
        here += w[i];
      }
      if (tid == 0) s.found = (int)left - 1;
      u64 up = scan(here) - here + base_sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (i < per && first + i < left && up < limit) {  // kept
          if (w[i]) add_to_unit((uint32_t)keys[first + i], w[i]);
          if (up + w[i] >= limit) s.found = (int)(first + i);
        }
        up += w[i];
      }
      __syncthreads();
      if (tid == 0) {
        const u64 key = keys[max(s.found, 0)];
        s.cut = left ? Cut{list_x(key), (int)(uint32_t)key} : cut_none();
      }
    }
    sync();
    cut = *at(&s.cut, 0);
    return true;
  }

  // The cut at which the count (MASS: the weights' sum) over the tokens `within` reaches `limit`.
  template <bool MASS>
  __device__ __forceinline__ Cut select(u64 limit, const Cut& within) {
    auto value = [&](float x) -> u64 { return MASS ? weight(x) : 1ull; };
    auto worth = [&](float top) { return top >= within.value && steps_below(top) < sc.t_end; };
    clear_hist();
    each_unit(worth,
              [&](int v, const float(&x)[E]) {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                  u64 w[2];
                  float2 below;
                  if constexpr (MASS) weigh(make_float2(x[e], x[e + 1]), w, below);
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    const float t = MASS ? -(k ? below.y : below.x) : steps_below(x[e + k]);
                    if (t < sc.t_end && within.keeps(x[e + k], index_of(v, e + k))) {
                      if constexpr (MASS)
                        add_to(bin_of(t), w[k]);
                      else
                        atomicAdd(reinterpret_cast<uint32_t*>(hist + bin_of(t)), 1u);
                    }
                  }
                }
              },
              [](int) {});
    int bin;
    u64 before;
    cross(0, limit, bin, before);
    Range g{bin, bin, 0u, ~0u};
    // (each round divides the keys by 2048: three end it)
    for (int round = 0; round < 5; ++round) {
      if (rank == 0 && tid == 0) s.listed = 0;
      sync();
      gather([&](float top) { return worth(top) && bin_of(steps_below(top)) <= g.hi && float_ord(top) >= g.from; },
             [&](float x, int i) { return in_range(x, i, g, within); });
      sync();
      const unsigned n = *at(&s.listed, 0);
      sync();
      if (n <= kSfList) return MASS ? finish_list(n, 0, ~0ull, before, limit) : finish_list(n, before, limit, 0, ~0ull);
      // too many: by the bits of x
      uint32_t least = ~0u, most = 0;
      each_unit(worth,
                [&](int v, const float(&x)[E]) {
#pragma unroll
                  for (int e = 0; e < E; ++e)
                    if (in_range(x[e], index_of(v, e), g, within)) {
                      least = min(least, float_ord(x[e]));
                      most = max(most, float_ord(x[e]));
                    }
                },
                [](int) {});
      least = __reduce_min_sync(~0u, least);
      most = __reduce_max_sync(~0u, most);
      if (tid == 0) {
        s.publish_key[0] = ~0u;
        s.publish_key[1] = 0;
      }
      __syncthreads();
      if (lane == 0) {
        atomicMin(&s.publish_key[0], least);
        atomicMax(&s.publish_key[1], most);
      }
      sync();
      for (int c = 0; c < ctas(); ++c) {
        least = min(least, *at(&s.publish_key[0], c));
        most = max(most, *at(&s.publish_key[1], c));
      }
      sync();
      if (least == most) {  // equal values: by their indices
        const float x0 = ord_float(least);
        const u64 w0 = MASS ? value(x0) : 1ull, need = limit > before ? limit - before : 0;
        const u64 rank_of = w0 ? max((need + w0 - 1) / w0, 1ull) : 1ull;
        auto one = [&](float x, int i) -> u64 { return in_range(x, i, g, within) ? 1ull : 0ull; };
        const u64 here = sum_units(worth, [&](int v, const float(&x)[E]) {
          u64 n = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) n += one(x[e], index_of(v, e));
          return n;
        });
        const u64 all = row_sum_of(here);
        u64 w;
        const int i = locate(one, here, min(rank_of, all) - 1, w);
        return Cut{x0, i};
      }
      int down = 0;
      while ((most - least) >> down >= (uint32_t)kSfBins) ++down;
      clear_hist();
      each_unit(worth,
                [&](int v, const float(&x)[E]) {
#pragma unroll
                  for (int e = 0; e < E; ++e)
                    if (in_range(x[e], index_of(v, e), g, within)) add_to((int)((most - float_ord(x[e])) >> down), value(x[e]));
                },
                [](int) {});
      const u64 base_sum = before;
      cross(base_sum, limit, bin, before);
      g.to = most - ((uint32_t)bin << down);
      const uint32_t wide = (1u << down) - 1u;
      g.from = g.to > wide ? g.to - wide : 0u;
    }
    return within;
  }
  __device__ __forceinline__ void run() {
    // the row's settings (used when the row's loads are under way) and the table
    float temp = p.temperature ? __ldg(p.temperature + row) : 1.0f, top_p = p.top_p ? __ldg(p.top_p + row) : 1.0f;
    float min_p = p.min_p ? __ldg(p.min_p + row) : 0.0f, u = __ldg(p.u + row);
    int top_k = p.top_k ? __ldg(p.top_k + row) : 0;
    uint2 power = make_uint2(0u, 0u);
    if (tid < kSfSteps) power = make_uint2(__ldg(&c_powers.whole[tid]), __float_as_uint(__ldg(&c_powers.value[tid])));
    const float mine = load_row([&]() {
      if (tid < kSfSteps) s.powers[tid] = make_uint2(power.x - kSfMagicBits, power.y);
      for (int i = tid; i < kSfCoarse / 2; i += kSfThreads) hist[i] = 0;  // (a cluster's CTAs count in the first's)
      clear_units();
      if (tid == 0) s.threads = 0;
      if (min_p > 0.0f && tid == kSfThreads - 1) {  // (once: FP64 is slow)
        // (an infinite temperature keeps everything: infinity times log(1) would be NaN)
        const double cut = temp < INFINITY ? (double)temp * log((double)min_p) : -INFINITY;
        const float high = (float)cut;
        s.min_cut = make_float2(high, isfinite(high) ? (float)(cut - (double)high) : 0.0f);
      }
    });
    bool bad = false;
    if (!(temp >= 0.0f)) bad = true, temp = 0.0f;
    if (top_k < 0) bad = true, top_k = 0;
    if (!(top_p > 0.0f && top_p <= 1.0f)) bad = true, top_p = 1.0f;
    if (!(min_p >= 0.0f && min_p <= 1.0f)) bad = true, min_p = 0.0f;
    if (!(u >= 0.0f && u < 1.0f)) bad = true, u = u >= 1.0f ? 1.0f : 0.0f;
    if (bad && rank == 0 && tid == 0 && p.status) atomicOr(p.status, kDevInternal);
    if (temp == 0.0f) top_k = 1, top_p = 1.0f, min_p = 0.0f, temp = 1.0f;
    if (top_k >= p.vocab) top_k = 0;
    // the row's maximum
    float m = mine;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    if (lane == 0) s.warp_max[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSfWarps; ++w) m = fmaxf(m, s.warp_max[w]);
    if constexpr (CL) {
      if (tid == 0) s.publish_max = m;
      sync();
      for (int c = 0; c < ctas(); ++c) m = fmaxf(m, *at(&s.publish_max, c));
    }
    if (!(fabsf(m) < INFINITY)) {  // nothing to draw (or +inf, which is not supported)
      if (rank == 0 && tid == 0) {
        p.out_token[row] = -1;
        if (p.out_logprob) p.out_logprob[row] = -INFINITY;
      }
      if constexpr (CL) sync();
      return;
    }
    sc.top = m;
    // 64 log2(e) / T as a pair: the quotient, and what it leaves
    constexpr double kSteps = kSfSteps * 1.4426950408889634073599;
    constexpr float kStepsHi = (float)kSteps, kStepsLo = (float)(kSteps - (double)kStepsHi);
    sc.hi = fminf(__fdiv_rn(kStepsHi, temp), 1e30f);
    sc.lo = sc.hi < 1e30f && temp < INFINITY ? __fdiv_rn(__fadd_rn(__fmaf_rn(-sc.hi, temp, kStepsHi), kStepsLo), temp) : 0.0f;
    float least = -INFINITY;  // the smallest x with w >= min_p: M + T ln(min_p), rounded up
    if (min_p > 0.0f) {
      const float2 sum = two_sum(m, s.min_cut.x);
      least = sum.x;
      if (__fadd_rn(sum.y, s.min_cut.y) > 0.0f) least = ord_float(float_ord(least) + 1);
    }
    sc.t_end = (float)(kSfSteps * (p.shift + 31));
    sc.per_bin = (float)kSfBins / fminf(sc.t_end, 48.0f * sc.hi);
    Cut cut = cut_none();
    bool open = true;     // the list has not done it
    bool summed = false;  // the units' sums of what is kept are there
    if (top_k > 0 && top_k <= kSfListed && (top_k <= kSfThreads * ctas() / 4 || top_k <= vectors / 4)) {
      // The k-th largest of the threads' maxima, or of the vectors', by coarse steps: at least k tokens lie there
      // or above, and not many more.  The threads' are at hand, and good enough while k is few of them: by the threads' and
      // by the vectors', us, 1024 rows of 40000 top-k 30 30 and 41, 64 36 and 46; 64 rows of 120000 over four CTAs top-k 200 27
      // and 31.  (Up to half of the threads they would be still, by less: top-k 100 45 and 50, 500 36 and 45.)
      const float per_step = (float)kSfCoarse / fminf(sc.t_end, 48.0f * sc.hi);
      auto* steps = reinterpret_cast<uint32_t*>(at(hist, 0));
      auto count = [&](float top) {
        const float t = steps_below(top);
        if (t < sc.t_end) atomicAdd(steps + (int)fminf(t * per_step, (float)(kSfCoarse - 1)), 1u);
      };
      if (top_k <= kSfThreads * ctas() / 4)
        count(mine);
      else
        for (int v = tid; v < p.units * p.unit_vecs * 32; v += kSfThreads) count(max_of(get(v)));
      sync();
      if (rank == 0) {
        if (warp == 0) {  // 32 steps at a time, one per lane
          const uint32_t* h = reinterpret_cast<const uint32_t*>(hist);
          constexpr int ROUNDS = kSfCoarse / 32;
          uint32_t part[ROUNDS], before = 0;
#pragma unroll
          for (int i = 0; i < ROUNDS; ++i) part[i] = h[i * 32 + lane];
          int crossing = -1;
#pragma unroll
          for (int i = 0; i < ROUNDS; ++i) {
            const uint32_t sum = __reduce_add_sync(~0u, part[i]);
            if (crossing < 0 && before + sum >= (uint32_t)top_k) {
              uint32_t upto = part[i];
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                const uint32_t t = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += t;
              }
              crossing = i * 32 + __ffs(__ballot_sync(~0u, before + upto >= (uint32_t)top_k)) - 1;
            }
            before += sum;
          }
          if (lane == 0) {
            s.crossing = crossing;
            s.listed = 0;
          }
        }
      }
      sync();
      const int step = *at(&s.crossing, 0);
      // (a little below the step: a lower bound is all it has to be; the last one holds all that has a weight)
      const bool last = step >= kSfCoarse - 1;
      const float deep = __fdiv_rn((last ? sc.t_end : (float)(step + 1)) * 1.001f, last ? sc.hi : per_step * sc.hi);
      float bound = __fsub_rd(m, deep);
      if (step < 0 || !(bound <= m)) bound = -INFINITY;
      const unsigned n = gather_from(bound, mine);
      if (n <= kSfList) {
        open = false;
        summed = true;
        if (draw_list(n, top_k, top_p, least, u, cut)) return;
      }
    }
    if (open) {
      if (top_k > 0) cut = select<false>(top_k, cut);
      if (top_p < 1.0f) {
        const Cut by_k = cut;
        summed = top_k > 0 ? nucleus<false>(top_p, by_k, cut) : nucleus<true>(top_p, by_k, cut);
      }
      if (least > cut.value) {
        cut = Cut{least, 0x7fffffff};
        summed = false;
      }
    }
    auto kept = [&](float x, int i) -> u64 { return cut.keeps(x, i) ? weight(x) : 0ull; };
    u64 here = 0;
    if (summed) {
      for (int i = tid; i < p.units; i += kSfThreads) here += unit_sum[i];
      here = block_total(here);
    } else {
      here = sum_units([&](float top) { return top >= cut.value; }, [&](int v, const float(&x)[E]) {
        u64 sum = 0;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          u64 w[2];
          float2 below;
          weigh(make_float2(x[e], x[e + 1]), w, below);
          sum += (cut.keeps(x[e], index_of(v, e)) ? w[0] : 0) + (cut.keeps(x[e + 1], index_of(v, e + 1)) ? w[1] : 0);
        }
        return sum;
      });
    }
    const u64 all = row_sum_of(here);
    bool cut_off;
    const u64 target = min(part_of(u, all, cut_off), all - 1);
    u64 w;
    const int token = locate(kept, here, target, w);
    if (rank == 0 && tid == 0) write(token, w, all);
  }
};

template <int DT, bool BIAS, bool CL>
__global__ void __launch_bounds__(kSfThreads, 1024 / kSfThreads) sample_filter_kernel(const __grid_constant__ FilterParams p) {
  extern __shared__ __align__(16) unsigned char sf_raw[];
  __shared__ Shared shared;
  using S = Sampler<DT, BIAS, CL>;
  const int c = CL ? p.cluster : 1, row = blockIdx.x / c, rank = blockIdx.x - row * c;
  const size_t stored = p.resident ? (size_t)p.units * p.unit_vecs * 32 * S::SV : 0;
  unsigned char* after = sf_raw + stored;
  u64* hist = reinterpret_cast<u64*>(after);
  u64* sorted = hist + kSfBins;
  uint32_t* ranks = reinterpret_cast<uint32_t*>(sorted + 2 * kSfRank);
  unsigned short* index_rank = reinterpret_cast<unsigned short*>(ranks + kSfRank);
  u64* unit_sum = reinterpret_cast<u64*>(index_rank + kSfRank);
  const unsigned char* at = p.logits + (long long)row * p.row_bytes;
  const unsigned lead_bytes = (unsigned)(reinterpret_cast<uintptr_t>(at) & 15);
  const int lead = (int)(lead_bytes / S::B);
  S s{p, shared, sf_raw, unit_sum, hist, sorted, ranks, index_rank, row, rank, lead, (int)(((long long)lead + p.vocab + S::E - 1) / S::E),
      rank * p.units * p.unit_vecs * 32, at - lead_bytes, RowScale{}, (int)threadIdx.x, (int)threadIdx.x >> 5,
      (int)threadIdx.x & 31, 0, 0};
  s.run();
}

size_t filter_smem(const FilterParams& p, int stored_vector) {
  return (p.resident ? (size_t)p.units * p.unit_vecs * 32 * stored_vector : 0) + (kSfBins + 2 * kSfRank + (size_t)p.units) * 8 + kSfRank * 6;
}

template <int DT, bool BIAS, bool CL>
cudaError_t run_filter(const FilterParams& p, size_t bytes, cudaStream_t stream) {
  auto kernel = sample_filter_kernel<DT, BIAS, CL>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_shared(kernel, 226 * 1024 - (int)sizeof(Shared), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.rows * p.cluster));
  cfg.blockDim = dim3(kSfThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int DT, bool BIAS>
cudaError_t plan_filter(FilterParams p, cudaStream_t stream) {
  constexpr int E = Traits<DT>::kVec, SV = BIAS ? E * 4 : 16;
  constexpr size_t kMost = 226 * 1024 - sizeof(Shared) - 1024;  // what one CTA may have
  constexpr long long kFew = 2 * kAtSms;
  const long long groups = ((long long)p.vocab + E - 1 + E - 1 + 32 * E - 1) / (32 * E);  // of 32 vectors
  auto share = [&](int c) {
    const long long n = (groups + c - 1) / c;
    p.cluster = c;
    p.unit_vecs = (int)((n + kSfMaxUnits - 1) / kSfMaxUnits);
    p.units = (int)((n + p.unit_vecs - 1) / p.unit_vecs);
    p.resident = 1;
    p.thread_vecs = (p.units + kSfWarps - 1) / kSfWarps * p.unit_vecs;
    make_divisor((uint32_t)p.thread_vecs, &p.thread_magic, &p.thread_shift);
    return filter_smem(p, SV);
  };
  // CTAs of a row: as many as the GPU holds at once, and at least as many as keep the row in shared memory
  int c = p.cluster == 2 || p.cluster == 4 || p.cluster == 8 ? p.cluster : 1;
  const bool forced = p.cluster != 0;
  while (!forced && c < kSfMaxCluster && (long long)p.rows * c * 2 <= kFew && groups >= 16 * c) c *= 2;
  // More rows than CTAs with a row in shared memory fit the GPU: four CTAs per SM without it, and what is read again
  // comes from L2.
  const bool many = (long long)p.rows * c > kFew;
  while (!many && !forced && c < kSfMaxCluster && share(c) > kMost) c *= 2;
  size_t bytes = share(c);
  if (bytes > kMost || many) {
    p.resident = 0;
    bytes = filter_smem(p, SV);
  }
  return c > 1 ? run_filter<DT, BIAS, true>(p, bytes, stream) : run_filter<DT, BIAS, false>(p, bytes, stream);
}

}  // namespace
}  // namespace lsb
