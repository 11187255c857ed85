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
constexpr int kSfRank = 512;         // lists up to this are ranked, longer ones sorted by exchanges
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
  u64 warp_sum[kSfWarps];
  float warp_max[kSfWarps];
  u64 publish_sum[4];       // what the cluster's CTAs tell each other, a place per purpose
  float publish_max;
  uint32_t publish_key[2];
  u64 before;               // of the crossing step
  int crossing;
  unsigned listed;          // entries of the list (the first CTA's)
  Cut cut;
  int found;
  u64 rest;
};

template <int DT, bool BIAS, bool CL>
struct Sampler {
  static constexpr int E = Traits<DT>::kVec, B = Traits<DT>::kBytes;
  static constexpr int SV = BIAS ? E * 4 : 16;  // bytes of a stored vector
  const FilterParams& p;
  Shared& s;
  unsigned char* store;   // the CTA's share of the row
  float* unit_max;        // [units]
  u64* unit_sum;          // [units]
  u64* hist;              // [kSfBins], then the list
  u64* sorted;            // [kSfRank]
  int row, rank, lead, vectors, first_vec;
  const unsigned char* base;  // the row's first 16-byte vector
  RowScale sc;
  int tid, warp, lane;

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
  __device__ __forceinline__ void values_of(const uint4& d, int v, float (&x)[E]) const {
    unpack<DT>(d, x);
    if constexpr (BIAS) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = index_of(v, e);
        if (i >= 0 && i < p.vocab) x[e] += __ldg(p.bias + i);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = x[e] == x[e] ? x[e] : -INFINITY;
  }
  __device__ __forceinline__ void get(int v, float (&x)[E]) const {
    if (!p.resident) {
      values_of(fetch(v), v, x);
    } else if constexpr (BIAS) {
      const float4* from = reinterpret_cast<const float4*>(store + (size_t)v * SV);
#pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        const float4 y = from[j];
        x[4 * j] = y.x;
        x[4 * j + 1] = y.y;
        x[4 * j + 2] = y.z;
        x[4 * j + 3] = y.w;
      }
    } else {
      unpack<DT>(*reinterpret_cast<const uint4*>(store + (size_t)v * SV), x);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = x[e] == x[e] ? x[e] : -INFINITY;
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
    __syncthreads();
    if (lane == 31) s.warp_sum[warp] = v;
    __syncthreads();
    u64 before = 0;
    for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
    return v + before;
  }
  __device__ __forceinline__ u64 block_total(u64 v) {
    v = warp_total(v);
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int w = 0; w < kSfWarps; ++w) t += s.warp_sum[w];
    return t;
  }
  __device__ __forceinline__ u64 row_total(u64 v, int place) {
    const u64 t = block_total(v);
    if constexpr (!CL) return t;
    if (tid == 0) s.publish_sum[place] = t;
    sync();
    u64 all = 0;
    for (int c = 0; c < ctas(); ++c) all += *at(&s.publish_sum[place], c);
    sync();
    return all;
  }

  // ---- passes over the share: f(v, x) for every vector of the units whose maximum passes `worth`
  template <class Worth, class F, class Done>
  __device__ __forceinline__ void each_unit(Worth worth, F f, Done done) {
    for (int un = warp; un < p.units; un += kSfWarps) {
      if (!worth(unit_max[un])) {
        done(un, false);
        continue;
      }
      for (int i = 0; i < p.unit_vecs; ++i) {
        const int v = (un * p.unit_vecs + i) * 32 + lane;
        float x[E];
        get(v, x);
        f(v, x);
      }
      done(un, true);
    }
  }

  __device__ __forceinline__ float load_row() {
    float mine = -INFINITY;
    const int n = p.units * p.unit_vecs;  // groups of 32 vectors
    constexpr int AHEAD = 4;
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
        float x[E], m = -INFINITY;
        values_of(d[a], v, x);
#pragma unroll
        for (int e = 0; e < E; ++e) m = fmaxf(m, x[e]);
        if (p.resident) {
          if constexpr (BIAS) {
#pragma unroll
            for (int j = 0; j < E / 4; ++j)
              reinterpret_cast<float4*>(store + (size_t)v * SV)[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
          } else {
            *reinterpret_cast<uint4*>(store + (size_t)v * SV) = d[a];
          }
        }
        mine = fmaxf(mine, m);
        if (p.unit_vecs == 1) {
#pragma unroll
          for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
          if (lane == 0) unit_max[g] = m;
        }
      }
    }
    if (p.unit_vecs > 1) {
      __syncthreads();
      for (int un = warp; un < p.units; un += kSfWarps) {
        float m = -INFINITY;
        for (int i = 0; i < p.unit_vecs; ++i) {
          float x[E];
          get((un * p.unit_vecs + i) * 32 + lane, x);
#pragma unroll
          for (int e = 0; e < E; ++e) m = fmaxf(m, x[e]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if (lane == 0) unit_max[un] = m;
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
  __device__ __forceinline__ unsigned gather(const Range& g, const Cut& within) {
    if (rank == 0 && tid == 0) s.listed = 0;
    sync();
    u64* list = at(hist, 0);
    unsigned* listed = at(&s.listed, 0);
    each_unit(
        [&](float top) {
          const float t = steps_below(top);
          return t < sc.t_end && bin_of(t) <= g.hi && top >= within.value && float_ord(top) >= g.from;
        },
        [&](int v, const float(&x)[E]) {
          unsigned hits = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) hits |= (in_range(x[e], index_of(v, e), g, within) ? 1u : 0u) << e;
          if (!__any_sync(~0u, hits != 0)) return;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const bool hit = (hits >> e) & 1u;
            const unsigned mask = __ballot_sync(~0u, hit);
            if (!mask) continue;
            unsigned from = 0;
            if (lane == __ffs(mask) - 1) from = atomicAdd(listed, (unsigned)__popc(mask));
            from = __shfl_sync(~0u, from, __ffs(mask) - 1) + __popc(mask & ((1u << lane) - 1u));
            if (hit && from < kSfList) list[from] = (u64)~float_ord(x[e]) << 32 | (uint32_t)index_of(v, e);
          }
        },
        [](int, bool) {});
    sync();
    const unsigned n = *listed;
    sync();
    return n;
  }
  __device__ __forceinline__ static float list_x(u64 key) { return ord_float(~(uint32_t)(key >> 32)); }

  // The list's first entry at which the count reaches k or the weight `limit`; top_p (below 1) instead of a limit:
  // of the weight of the list's first k.  The first CTA works it out, every thread gets the cut.
  __device__ __forceinline__ Cut finish_list(unsigned n, u64 base_count, u64 k, u64 base_sum, u64 limit, float top_p) {
    if (rank == 0) {
      const u64* keys = hist;
      if (n <= kSfRank) {
        for (unsigned i = tid; i < n; i += kSfThreads) {
          const u64 mine = hist[i];
          unsigned before = 0;
          for (unsigned j = 0; j < n; ++j) before += hist[j] < mine;
          sorted[before] = mine;
        }
        keys = sorted;
        __syncthreads();
      } else {  // bitonic, the places past the list last
        for (unsigned i = n + tid; i < kSfList; i += kSfThreads) hist[i] = ~0ull;
        __syncthreads();
        for (unsigned size = 2; size <= kSfList; size <<= 1)
          for (unsigned gap = size >> 1; gap; gap >>= 1) {
            for (unsigned t = tid; t < kSfList / 2; t += kSfThreads) {
              const unsigned i = 2 * t - (t & (gap - 1)), j = i + gap;
              const u64 a = hist[i], b = hist[j];
              if ((a > b) == ((i & size) == 0)) {
                hist[i] = b;
                hist[j] = a;
              }
            }
            __syncthreads();
          }
      }
      constexpr int PER = kSfList / kSfThreads;
      const unsigned first = tid * PER;
      u64 w[PER], mine = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        w[i] = first + i < n && base_count + first + i < k ? weight(list_x(keys[first + i])) : 0;
        mine += w[i];
      }
      const u64 upto = scan(mine);
      if (top_p < 1.0f) {
        if (tid == kSfThreads - 1) s.rest = upto;
        __syncthreads();
        limit = share_of(top_p, s.rest);
      }
      if (tid == 0) s.found = (int)n - 1;
      __syncthreads();
      u64 run = base_sum + upto - mine;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        run += w[i];
        if (first + i < n && (base_count + first + i + 1 >= k || run >= limit)) {
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
  __device__ __forceinline__ static u64 share_of(float f, u64 all) {  // the least whole number >= f * all
    const u64 n = (u64)ceil((double)f * (double)all);
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
          get(v, x);
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

  // The units' sums of f (over units whose maximum passes `worth`); the CTA's sum for every thread.
  template <class Worth, class F>
  __device__ __forceinline__ u64 sum_units(Worth worth, F f) {
    u64 run = 0, all = 0;
    each_unit(
        worth,
        [&](int v, const float(&x)[E]) {
#pragma unroll
          for (int e = 0; e < E; ++e) run += f(x[e], index_of(v, e));
        },
        [&](int un, bool any) {
          const u64 t = any ? warp_total(run) : 0;
          if (lane == 0) unit_sum[un] = t;
          all += t;
          run = 0;
        });
    return block_total(lane == 0 ? all : 0);
  }

  // The cut at which the count (by weight: the weights' sum) over the tokens `within` reaches `limit`.
  template <bool MASS>
  __device__ __forceinline__ Cut select(u64 limit, const Cut& within) {
    auto value = [&](float x) -> u64 { return MASS ? weight(x) : 1ull; };
    clear_hist();
    each_unit([&](float top) { return top >= within.value && steps_below(top) < sc.t_end; },
              [&](int v, const float(&x)[E]) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                  const float t = steps_below(x[e]);
                  if (t < sc.t_end && within.keeps(x[e], index_of(v, e))) {
                    if constexpr (MASS)
                      add_to(bin_of(t), weight(x[e]));
                    else
                      atomicAdd(reinterpret_cast<uint32_t*>(hist + bin_of(t)), 1u);
                  }
                }
              },
              [](int, bool) {});
    int bin;
    u64 before;
    cross(0, limit, bin, before);
    Range g{bin, bin, 0u, ~0u};
    // (each round divides the keys by 2048: three end it)
    for (int round = 0; round < 5; ++round) {
      const unsigned n = gather(g, within);
      if (n <= kSfList)
        return MASS ? finish_list(n, 0, ~0ull, before, limit, 1.0f) : finish_list(n, before, limit, 0, ~0ull, 1.0f);
      // too many: by the bits of x
      uint32_t least = ~0u, most = 0;
      auto worth = [&](float top) { return top >= within.value && steps_below(top) < sc.t_end; };
      each_unit(worth,
                [&](int v, const float(&x)[E]) {
#pragma unroll
                  for (int e = 0; e < E; ++e)
                    if (in_range(x[e], index_of(v, e), g, within)) {
                      least = min(least, float_ord(x[e]));
                      most = max(most, float_ord(x[e]));
                    }
                },
                [](int, bool) {});
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
                [](int, bool) {});
      const u64 base_sum = before;
      cross(base_sum, limit, bin, before);
      g.to = most - ((uint32_t)bin << down);
      const uint32_t wide = (1u << down) - 1u;
      g.from = g.to > wide ? g.to - wide : 0u;
    }
    return within;
  }
  // the cluster's sum of the CTAs' sums `here` (the same in all of a CTA's threads)
  __device__ __forceinline__ u64 row_sum_of(u64 here) {
    if constexpr (!CL) return here;
    if (tid == 0) s.publish_sum[1] = here;
    sync();
    u64 all = 0;
    for (int c = 0; c < ctas(); ++c) all += *at(&s.publish_sum[1], c);
    sync();
    return all;
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
    if (m == -INFINITY) {
      if (rank == 0 && tid == 0) {
        p.out_token[row] = -1;
        if (p.out_logprob) p.out_logprob[row] = -INFINITY;
      }
      if constexpr (CL) sync();
      return;
    }
    sc.top = m;
    const double c = fmin(92.33248261893502 / (double)temp, 1e30);  // 64 log2(e) / T
    sc.hi = (float)c;
    sc.lo = (float)(c - (double)sc.hi);
    sc.t_end = (float)(kSfSteps * (p.shift + 31));
    sc.per_bin = (float)kSfBins / fminf(sc.t_end, 48.0f * sc.hi);
    Cut cut = cut_none();
    bool open = true;  // top-p still to do
    if (top_k > 0 && top_k <= kSfThreads * ctas() / 4) {
      // the k-th largest of the threads' maxima, by the histogram's steps
      clear_hist();
      const float t = steps_below(mine);
      if (t < sc.t_end) atomicAdd(reinterpret_cast<uint32_t*>(hist + bin_of(t)), 1u);
      int bin;
      u64 before;
      cross(0, top_k, bin, before);
      const unsigned n = gather(Range{0, bin, 0u, ~0u}, cut);
      if (n <= kSfList) {
        cut = finish_list(n, 0, top_k, 0, ~0ull, top_p);
        open = false;
      }
    }
    if (open && top_k > 0) cut = select<false>(top_k, cut);
    if (open && top_p < 1.0f) {
      const Cut by_k = cut;
      const u64 here = sum_units([&](float top) { return top >= by_k.value; },
                                 [&](float x, int i) -> u64 { return by_k.keeps(x, i) ? weight(x) : 0ull; });
      cut = select<true>(share_of(top_p, row_sum_of(here)), by_k);
    }
    if (min_p > 0.0f) {
      const float least = __double2float_ru((double)m + (double)temp * log((double)min_p));
      if (least > cut.value) cut = Cut{least, 0x7fffffff};
    }
    auto kept = [&](float x, int i) -> u64 { return cut.keeps(x, i) ? weight(x) : 0ull; };
    const u64 here = sum_units([&](float top) { return top >= cut.value; }, kept);
    const u64 all = row_sum_of(here);
    u64 target = (u64)((double)u * (double)all);
    target = min(target, all - 1);
    u64 w;
    const int token = locate(kept, here, target, w);
    if (rank == 0 && tid == 0) {
      p.out_token[row] = token;
      if (p.out_logprob) {
        // near 1 from what is missing
        p.out_logprob[row] = w > all / 2 ? log1pf(-((float)(all - w) / (float)all)) : logf((float)w / (float)all);
      }
    }
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
  u64* unit_sum = sorted + kSfRank;
  float* unit_max = reinterpret_cast<float*>(unit_sum + p.units);
  const unsigned char* at = p.logits + (long long)row * p.row_bytes;
  const unsigned lead_bytes = (unsigned)(reinterpret_cast<uintptr_t>(at) & 15);
  const int lead = (int)(lead_bytes / S::B);
  S s{p, shared, sf_raw, unit_max, unit_sum, hist, sorted, row, rank, lead, (int)(((long long)lead + p.vocab + S::E - 1) / S::E),
      rank * p.units * p.unit_vecs * 32, at - lead_bytes, RowScale{}, (int)threadIdx.x, (int)threadIdx.x >> 5,
      (int)threadIdx.x & 31};
  s.run();
}

size_t filter_smem(const FilterParams& p, int stored_vector) {
  return (p.resident ? (size_t)p.units * p.unit_vecs * 32 * stored_vector : 0) + (kSfBins + kSfRank) * 8 + (size_t)p.units * 12;
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
