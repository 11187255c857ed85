// Sampling with temperature, top-k, top-p and min-p, a setting of its own for each row.
//
// With w(x) = 2^((x - M) log2(e) / T), M the row's maximum, every filter keeps a prefix of the tokens in
// the order (x falling, index rising), so that the three together are one cut: the last kept (x, index).
// The token is then found by a prefix sum in the vocabulary's order.
//
// The row is read once, into the shared memory of one CTA or of a cluster's; what follows runs on
// that copy.  The cut is found without sorting the row:
//   top-k up to a quarter of the threads: the k-th largest of the threads' maxima bounds the row's
//     k-th largest from below (the hierarchical method's first pass); what lies above is a short list.
//   otherwise a histogram of x in 2048 equal steps, of counts for top-k, of weights for top-p; the step
//     in which the limit is passed is the list.  A list that overflows (many equal values) is cut again by
//     the bits of x, and equal values by their indices.
// The list is sorted, its weights are added up, and that gives the cut.
//
// Weights are whole numbers.  A draw near a border between tokens, and a token near the border of the
// nucleus, turn on the last digits of sums over the whole row: with f32 weights and sums some rows in a
// thousand would get another token than in exact arithmetic, and other orders of summation other
// tokens.  Here w is formed to about 2^-30 of its value (a table of 64 powers and a cubic in f32, the
// exponent's argument as an unevaluated pair) and rounded to units of 2^-44 of the largest; sums of whole
// numbers are exact in any order.
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
constexpr int kSfRank = 512;         // lists up to this are ranked, longer ones sorted by exchanges; the fewest kept
                                     // tokens that are drawn by a pass over the row
constexpr int kSfCoarse = kSfThreads;  // steps of the histogram of maxima, one per thread
constexpr int kSfListed = 1000;      // the largest top-k that goes by a list alone
constexpr int kSfSteps = 64;         // steps of an octave in the table of powers
constexpr float kSfMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number in the low bits

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
__constant__ PowerTable c_powers = make_powers();

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
  uint2 powers[kSfSteps];
  u64 warp_sum[2][kSfWarps];
  float warp_max[kSfWarps];
  u64 publish_sum[4];       // what the cluster's CTAs tell each other, a place per purpose
  float publish_max;
  uint32_t publish_key[2];
  u64 before, limit;        // of the crossing step
  int crossing;
  unsigned listed;          // entries of the list (the first CTA's)
  Cut cut;
  int drawn;                // the list gave the token
  double min_cut;           // T ln(min_p)
  float least;              // the smallest x with w >= min_p
  int found, kept;
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
  u64* sorted;            // [kSfRank], then as many weights
  int row, rank, lead, vectors, first_vec;
  const unsigned char* base;  // the row's first 16-byte vector
  RowScale sc;
  int tid, warp, lane, flip;

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
      if (g == 0 || g == vectors - 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int i = g * E + e - lead;
          if (i < 0 || i >= p.vocab) set_neg_inf<DT>(d, e);
        }
      }
    }
    return d;
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
  __device__ __forceinline__ int bin_of(float t) const { return (int)fminf(t * sc.per_bin, (float)(kSfBins - 1)); }
  __device__ __forceinline__ u64 weight(float x) const {
    const float d = __fsub_rn(sc.top, x);
    const float t = __fmul_rn(d, sc.hi);
    if (!(t < sc.t_end)) return 0;
    // top - x = d + err exactly (Knuth's two-sum), times the pair
    const float bb = __fsub_rn(d, sc.top);
    const float err = __fsub_rn(__fsub_rn(sc.top, __fsub_rn(d, bb)), __fadd_rn(x, bb));
    const float tl = __fadd_rn(__fmaf_rn(d, sc.hi, -t), __fmaf_rn(d, sc.lo, __fmul_rn(err, sc.hi)));
    const float nf = __fadd_rn(t, kSfMagic);
    const float r = __fsub_rn(__fsub_rn(__fsub_rn(nf, kSfMagic), t), tl);
    constexpr float k1 = (float)(0.693147180559945309417232 / kSfSteps), k2 = (float)(0.693147180559945309417232 / kSfSteps * 0.693147180559945309417232 / kSfSteps / 2),
                    k3 = (float)(0.693147180559945309417232 / kSfSteps * 0.693147180559945309417232 / kSfSteps * 0.693147180559945309417232 / kSfSteps / 6);
    const float q = r * fmaf(r, fmaf(r, k3, k2), k1);  // 2^(r / 64) - 1
    const uint32_t n = __float_as_uint(nf) & 0x3fffffu;
    const uint2 pw = s.powers[n & (kSfSteps - 1)];
    const uint32_t f = pw.x + (__float_as_uint(__fmaf_rn(__uint_as_float(pw.y), q, kSfMagic)) - 0x4b400000u);
    const int down = (int)(n / kSfSteps) - p.shift;
    return (u64)(f >> max(down, 0)) << max(-down, 0);
  }

  // ---- sums over the CTA and the cluster; every thread gets the result
  __device__ __forceinline__ static u64 warp_total(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
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
    if (tid == 0) s.publish_sum[1] = here;
    sync();
    u64 all = 0;
    for (int c = 0; c < ctas(); ++c) all += *at(&s.publish_sum[1], c);
    sync();
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

  __device__ __forceinline__ float load_row() {
    float mine = -INFINITY;
    const int n = p.units * p.unit_vecs;  // groups of 32 vectors
    constexpr int AHEAD = 5;
    for (int g0 = warp; g0 < n; g0 += kSfWarps * AHEAD) {
      uint4 d[AHEAD];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int g = g0 + a * kSfWarps;
        if (g < n) d[a] = fetch(g * 32 + lane);
      }
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int g = g0 + a * kSfWarps;
        if (g >= n) break;
        const int v = g * 32 + lane;
        const Vec y = with_bias(d[a], v);
        mine = fmaxf(mine, max_of(y));
        if (p.resident) {
#pragma unroll
          for (int j = 0; j < SV / 16; ++j) reinterpret_cast<uint4*>(store + (size_t)v * SV)[j] = y.d[j];
        }
      }
    }
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
  // top_p below 1: the limit is that share of the steps' sum and `more`, of all CTAs.
  __device__ __forceinline__ void cross(u64 base_sum, u64& limit, int& bin, u64& before, float top_p = 1.0f, u64 more = 0) {
    if (top_p < 1.0f) {
      more = block_total(more);
      if (tid == 0) s.publish_sum[0] = more;
    }
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
      if (top_p < 1.0f) {
        if (tid == kSfThreads - 1) {
          u64 all = upto;
          for (int c = 0; c < ctas(); ++c) all += *at(&s.publish_sum[0], c);
          s.limit = share_of(top_p, all);
        }
        __syncthreads();
        limit = s.limit;
      }
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
    if (top_p < 1.0f) limit = *at(&s.limit, 0);
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
  // list holds).
  template <class Worth, class Hit>
  __device__ __forceinline__ unsigned gather(Worth worth, Hit hit) {
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
    sync();
    return *listed;
  }

  // The list in order, by the first CTA: where it lies then.
  __device__ __forceinline__ const u64* sort_list(unsigned n) {
    if (n <= kSfRank) {  // a warp to an entry: how many come before it
      for (unsigned i = warp; i < n; i += kSfWarps) {
        const u64 mine = hist[i];
        unsigned before = 0;
        for (unsigned j = lane; j < n; j += 32) before += hist[j] < mine;
        before = __reduce_add_sync(~0u, before);
        if (lane == 0) sorted[before] = mine;
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

  // All filters on a list that holds the row's first k tokens: the draw itself where few are kept, or the cut.
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
      if (per == 1 && first < n) weights[tid] = mine;
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
        if (tid == kept - 1) s.rest = upto;
        __syncthreads();
        const u64 all = s.rest;
        bool cut_off;
        const u64 target = min(part_of(u, all, cut_off), all - 1);
        for (unsigned i = warp; i < kept; i += kSfWarps) {
          const uint32_t index = (uint32_t)keys[i];
          u64 up = 0;
          for (unsigned j = lane; j < kept; j += 32)
            if ((uint32_t)keys[j] <= index) up += weights[j];
          up = warp_total(up);
          if (lane == 0 && up > target && up - weights[i] <= target) write(index, weights[i], all);
        }
        if (tid == 0) s.drawn = 1;
      } else if (tid == 0) {
        const u64 key = keys[max((int)kept - 1, 0)];
        s.cut = Cut{list_x(key), (int)(uint32_t)key};
        s.drawn = 0;
      }
    }
    sync();
    const bool drawn = *at(&s.drawn, 0);
    cut = *at(&s.cut, 0);
    sync();
    return drawn;
  }
  __device__ __forceinline__ void write(int token, u64 w, u64 all) const {
    p.out_token[row] = token;
    // (near 1 from what is missing)
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
      s.cut.index = -1;
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
                  s.cut.index = index_of(v, e);
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
    const int token = *at(&s.cut.index, owner);
    value = *at(&s.publish_sum[3], owner);
    sync();
    return token;
  }

  // The units' sums of f; the CTA's sum for every thread.
  template <class Worth, class F>
  __device__ __forceinline__ u64 sum_units(Worth worth, F f) {
    u64 run = 0, all = 0;
    each_unit(
        worth,
        [&](int v, const float(&x)[E]) {
#pragma unroll
          for (int e = 0; e < E; ++e) run += f(x[e], index_of(v, e));
        },
        [&](int un) {
          const u64 t = __any_sync(~0u, run != 0) ? warp_total(run) : 0;
          if (lane == 0) unit_sum[un] = t;
          all += t;
          run = 0;
        });
    return block_total(lane == 0 ? all : 0);
  }

  // The cut at which the count (MASS: the weights' sum) over the tokens `within` reaches `limit` (top_p of their sum).
  template <bool MASS>
  __device__ __forceinline__ Cut select(u64 limit, float top_p, const Cut& within, float thread_max) {
    auto value = [&](float x) -> u64 { return MASS ? weight(x) : 1ull; };
    auto worth = [&](float top) { return top >= within.value && steps_below(top) < sc.t_end; };
    clear_hist();
    u64 small = 0, border = 0;
    if constexpr (MASS) {
      // Weights under (1 - top_p) / vocab of the sum are together under 1 - top_p of it: the limit is passed before
      // them, and they need no steps.  The sum is at least that of the threads' maxima, where all are within.
      if (within.value == -INFINITY) {
        const u64 some = row_sum_of(block_total(weight(thread_max)));
        border = (u64)((1.0f - top_p) * 0.99f * (float)some / (float)p.vocab);
      }
    }
    each_unit(worth,
              [&](int v, const float(&x)[E]) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                  const float t = steps_below(x[e]);
                  if (t < sc.t_end && within.keeps(x[e], index_of(v, e))) {
                    if constexpr (MASS) {
                      const u64 w = weight(x[e]);
                      if (w < border)
                        small += w;
                      else
                        add_to(bin_of(t), w);
                    } else {
                      atomicAdd(reinterpret_cast<uint32_t*>(hist + bin_of(t)), 1u);
                    }
                  }
                }
              },
              [](int) {});
    int bin;
    u64 before;
    cross(0, limit, bin, before, MASS ? top_p : 1.0f, small);
    Range g{bin, bin, 0u, ~0u};
    // (each round divides the keys by 2048: three end it)
    for (int round = 0; round < 5; ++round) {
      if (rank == 0 && tid == 0) s.listed = 0;
      sync();
      const unsigned n = gather([&](float top) { return worth(top) && bin_of(steps_below(top)) <= g.hi && float_ord(top) >= g.from; },
                                [&](float x, int i) { return in_range(x, i, g, within); });
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
        const u64 here = sum_units(worth, one);
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
    for (int j = tid; j < kSfSteps; j += kSfThreads) s.powers[j] = make_uint2(c_powers.whole[j], __float_as_uint(c_powers.value[j]));
    // the row's settings
    float temp = p.temperature ? __ldg(p.temperature + row) : 1.0f, top_p = p.top_p ? __ldg(p.top_p + row) : 1.0f;
    float min_p = p.min_p ? __ldg(p.min_p + row) : 0.0f, u = __ldg(p.u + row);
    int top_k = p.top_k ? __ldg(p.top_k + row) : 0;
    bool bad = false;
    if (!(temp >= 0.0f)) bad = true, temp = 0.0f;
    if (top_k < 0) bad = true, top_k = 0;
    if (!(top_p > 0.0f && top_p <= 1.0f)) bad = true, top_p = 1.0f;
    if (!(min_p >= 0.0f && min_p <= 1.0f)) bad = true, min_p = 0.0f;
    if (!(u >= 0.0f && u < 1.0f)) bad = true, u = u >= 1.0f ? 1.0f : 0.0f;
    if (bad && rank == 0 && tid == 0 && p.status) atomicOr(p.status, kDevInternal);
    if (temp == 0.0f) top_k = 1, top_p = 1.0f, min_p = 0.0f, temp = 1.0f;
    if (top_k >= p.vocab) top_k = 0;
    if (min_p > 0.0f && tid == kSfThreads - 1) s.min_cut = (double)temp * log((double)min_p);  // (once: FP64 is slow)
    for (int i = tid; i < kSfCoarse / 2; i += kSfThreads) hist[i] = 0;  // (a cluster's CTAs count in the first's)
    const float mine = load_row();
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
    sc.lo = sc.hi < 1e30f ? __fdiv_rn(__fadd_rn(__fmaf_rn(-sc.hi, temp, kStepsHi), kStepsLo), temp) : 0.0f;
    if (min_p > 0.0f) {
      if (tid == 0) s.least = __double2float_ru((double)m + s.min_cut);
      __syncthreads();
    }
    sc.t_end = (float)(kSfSteps * (p.shift + 31));
    sc.per_bin = (float)kSfBins / fminf(sc.t_end, 48.0f * sc.hi);
    Cut cut = cut_none();
    bool open = true;  // the list has not done it
    if (top_k > 0 && top_k <= kSfListed && (top_k <= kSfThreads * ctas() / 4 || top_k <= vectors / 4)) {
      // The k-th largest of the threads' maxima, or of the vectors', by coarse steps: at least k tokens lie there
      // or above, and not many more.
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
        const u64 here = reinterpret_cast<const uint32_t*>(hist)[tid], upto = scan(here);
        if (upto >= top_k && upto - here < top_k) s.crossing = tid;
        if (tid == kSfThreads - 1 && upto < top_k) s.crossing = -1;
        if (tid == 0) s.listed = 0;
      }
      sync();
      const int step = *at(&s.crossing, 0);
      // (a little below the step: a lower bound is all it has to be)
      float bound = __fsub_rd(m, __fdiv_rn((float)(step + 1) * 1.001f, per_step * sc.hi));
      if (step < 0 || !(bound <= m)) bound = -INFINITY;
      const unsigned n = gather([&](float top) { return top >= bound; }, [&](float x, int) { return x >= bound && x > -INFINITY; });
      if constexpr (CL) sync();  // (the first CTA's counter has been read)
      if (n <= kSfList) {
        open = false;
        if (draw_list(n, top_k, top_p, min_p > 0.0f ? s.least : -INFINITY, u, cut)) return;
      }
    }
    if (open && top_k > 0) cut = select<false>(top_k, 1.0f, cut, mine);
    if (open && top_p < 1.0f) cut = select<true>(0, top_p, cut, mine);
    if (min_p > 0.0f && s.least > cut.value) cut = Cut{s.least, 0x7fffffff};
    auto kept = [&](float x, int i) -> u64 { return cut.keeps(x, i) ? weight(x) : 0ull; };
    const u64 here = sum_units([&](float top) { return top >= cut.value; }, kept);
    const u64 all = row_sum_of(here);
    bool cut_off;
    const u64 target = min(part_of(u, all, cut_off), all - 1);
    u64 w;
    const int token = locate(kept, here, target, w);
    if (rank == 0 && tid == 0) write(token, w, all);
  }
};

template <int DT, bool BIAS, bool CL>
__global__ void __launch_bounds__(kSfThreads, 2) sample_filter_kernel(const __grid_constant__ FilterParams p) {
  extern __shared__ __align__(16) unsigned char sf_raw[];
  __shared__ Shared shared;
  using S = Sampler<DT, BIAS, CL>;
  const int c = CL ? p.cluster : 1, row = blockIdx.x / c, rank = blockIdx.x - row * c;
  const size_t stored = p.resident ? (size_t)p.units * p.unit_vecs * 32 * S::SV : 0;
  unsigned char* after = sf_raw + stored;
  u64* hist = reinterpret_cast<u64*>(after);
  u64* sorted = hist + kSfBins;
  u64* unit_sum = sorted + 2 * kSfRank;
  const unsigned char* at = p.logits + (long long)row * p.row_bytes;
  const unsigned lead_bytes = (unsigned)(reinterpret_cast<uintptr_t>(at) & 15);
  const int lead = (int)(lead_bytes / S::B);
  S s{p, shared, sf_raw, unit_sum, hist, sorted, row, rank, lead, (int)(((long long)lead + p.vocab + S::E - 1) / S::E),
      rank * p.units * p.unit_vecs * 32, at - lead_bytes, RowScale{}, (int)threadIdx.x, (int)threadIdx.x >> 5,
      (int)threadIdx.x & 31, 0};
  s.run();
}

size_t filter_smem(const FilterParams& p, int stored_vector) {
  return (p.resident ? (size_t)p.units * p.unit_vecs * 32 * stored_vector : 0) + (kSfBins + 2 * kSfRank + (size_t)p.units) * 8;
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
  const long long groups = ((long long)p.vocab + E - 1 + E - 1 + 32 * E - 1) / (32 * E);  // of 32 vectors
  auto share = [&](int c) {
    const long long n = (groups + c - 1) / c;
    p.cluster = c;
    p.unit_vecs = (int)((n + kSfMaxUnits - 1) / kSfMaxUnits);
    p.units = (int)((n + p.unit_vecs - 1) / p.unit_vecs);
    p.resident = 1;
    return filter_smem(p, SV);
  };
  // CTAs of a row: as many as the GPU holds at once, and at least as many as keep the row in shared memory
  int c = p.cluster == 2 || p.cluster == 4 || p.cluster == 8 ? p.cluster : 1;
  while (p.cluster == 0 && c < kSfMaxCluster && ((long long)p.rows * c * 2 <= 2 * 152 && groups >= 16 * c)) c *= 2;
  while (c < kSfMaxCluster && share(c) > kMost) c *= 2;
  size_t bytes = share(c);
  if (bytes > kMost) {
    p.resident = 0;
    bytes = filter_smem(p, SV);
  }
  return c > 1 ? run_filter<DT, BIAS, true>(p, bytes, stream) : run_filter<DT, BIAS, false>(p, bytes, stream);
}

}  // namespace

cudaError_t launch_sample_filter(FilterParams p, int dtype, cudaStream_t stream) {
  if (dtype == DT_F32) return p.bias ? plan_filter<DT_F32, true>(p, stream) : plan_filter<DT_F32, false>(p, stream);
  if (dtype == DT_F16) return p.bias ? plan_filter<DT_F16, true>(p, stream) : plan_filter<DT_F16, false>(p, stream);
  return p.bias ? plan_filter<DT_BF16, true>(p, stream) : plan_filter<DT_BF16, false>(p, stream);
}

}  // namespace lsb
