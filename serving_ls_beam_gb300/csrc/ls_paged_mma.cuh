// Attention of one new token per row over a paged cache with 16-bit queries: up to 16 query heads share a
// key head, far too few for the tensor cores to be the limit, so the kernel is built around the stream of
// pages from memory and uses the warp-level matrix instructions (m16n8k16, f32 accumulators in registers).
//
//   S^T = K Q^T,  P = exp2(S - max),  O^T = O^T * correction + V^T P^T,  out = O / sum P
//
// in one pass with the running maximum and sum of the softmax (Milakov and Gimelshein, 2018), transposed so
// that keys and head elements are an instruction's 16 rows and the queries its 8 columns.
//
// Pages go straight from memory into registers in the instructions' own layout, 16 bytes per lane and load,
// through no shared memory: the order of the head's elements within a product's contraction is free as
// long as the queries have the same one, so lane (g, t) takes 16 bytes t, t + 4, .. of keys g and g + 8, and
// of the values 16 bytes g, g + 8, .. of keys 2t, 2t + 1, 2t + 8, 2t + 9, whose pairs it puts together itself.  A load
// instruction covers 64 (keys) or 128 bytes (values) of a head vector in a row, whatever the page size.  Where 16
// positions lie in one page (TILES) the lanes share its number and keep their places; otherwise lane n looks up key
// n's page.  Numbers are looked up two blocks ahead; keys are loaded again as soon as a block's scores are formed,
// values as soon as its sums are; a worker's next part has its queries and its first page numbers under way while
// the one before is at work.
//
// 8-bit codes become f16, exactly, in registers; a key's scale multiplies its scores.  A value's scale
// cannot go into its f16 elements nor, by itself, into an f16 weight (a key with nearly all the weight may have
// values 2^-20 of the others'), so the weights of the second product are 2^(score + log2 scale - reference) with a
// reference of their own, the largest such exponent, apart from the maximum that the sum is taken with.
//
// A weight goes into that product in two pieces (REST), rounded and what the rounding left: in f16 together good to 2^-22,
// in bf16 to 2^-16 of it.  The sum takes it as it is, in f32.  With the first piece alone the weights' rounding would count
// as much as the result's (relative errors against 64 bits, one piece and two: bf16 2.3e-3 and 1.7e-3, f16 over int8 2.9e-4
// and 2.1e-4, f16 1.07e-4 and 0.93e-4); the second costs a product per fragment (131000 bf16 positions 90.2 -> 90.3 us,
// int8 36.0 -> 36.7, 1024 short f16 rows 54.8 -> 55.6).  With bf16 queries over codes one f16 piece is 2^-11 of a weight
// beside a result rounded to 2^-8 of its value (1.67e-3 and 1.66e-3; 219 and 227 us), and is all there is.
//
// What bounds it: the instructions around the products (some 260 per warp for a block of 4 KB of 16-bit keys and values,
// twice that for codes, whose conversion is the most of it; 750 per part) and the latency that 8 to 16 warps per SM leave.
// 256 rows x 8 key heads of 128 codes, 4 queries, 501 to 4000 positions: 1.22 GB in 219 us, 0.82 of the measured copy rate
// (a CTA's four warps per part 238; page numbers through shuffles for every key 235); one row of 131000 bf16 positions
// 90 us, 0.88 (the parts joined by one thread per element 114); 32 rows of 2000 to 8000 105 us, 0.92; 64 rows x 16 heads of
// 64 int8, 300 to 999 positions: 37 us, 0.37; 1024 rows x 16 heads of 64 f16, 48 to 63 positions: 56 us, 0.62.  Blocks of 32
// keys for 16-bit heads of 64: no faster; a fifth CTA per SM for them spills (int8 36 -> 48 us).
#pragma once

#include "ls_paged.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

enum { KIND_F16 = 0, KIND_BF16 = 1, KIND_E4M3 = 2, KIND_I8 = 3 };

constexpr float kPmLazy = 8.0f;  // growth of a reference (log2) that is let pass
constexpr float kPmLift = 7.0f;  // f16 weights lie up to 2^7 (2^15 with that growth): kAtLift's reason

__device__ __forceinline__ uint4 stream16(const unsigned char* at) {
  uint4 d;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(d.x), "=r"(d.y), "=r"(d.z), "=r"(d.w)
               : "l"(at));
  return d;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint2 stream8(const unsigned char* at) {
  uint2 d;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(d.x), "=r"(d.y) : "l"(at));
  return d;
}

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool BF>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return half2_bits(lo, hi);
  }
}
// What pack_pair's rounding left of a pair of weights, rounded itself.
template <bool BF>
__device__ __forceinline__ uint32_t rest_of(float lo, float hi, uint32_t rounded) {
  if constexpr (BF) {
    return pack_pair<BF>(lo - __uint_as_float(rounded << 16), hi - __uint_as_float(rounded & 0xffff0000u));
  } else {
    const __half2 h = *reinterpret_cast<const __half2*>(&rounded);
    return pack_pair<BF>(lo - __low2float(h), hi - __high2float(h));
  }
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four codes as f16: the lower two and the upper two.
template <int KIND>
__device__ __forceinline__ void codes_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KIND == KIND_E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {  // 0x6400 + b is 1024 + b in f16; b = code + 128
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __floats2half2_rn(1152.0f, 1152.0f);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off), y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

__device__ __forceinline__ float log2_of(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int KIND, int DP, int NQ>
struct PmShape {
  static constexpr bool CODES = KIND >= KIND_E4M3;
  static constexpr int KB = CODES ? 32 : 16;           // keys of a block
  static constexpr int KT = KB / 16;
  static constexpr int KC = CODES ? DP / 64 : DP / 32;  // 16-byte loads of a lane per key
  static constexpr int VB = CODES && DP == 64 ? 8 : 16;  // bytes of a lane's load of a value vector
  static constexpr int VE = CODES ? VB : VB / 2;        // and its elements
  static constexpr int VC = DP / (8 * VE);              // such loads per value vector
  static constexpr int VW = VB / 4;
  static constexpr int CTAS = DP == 64 ? (NQ == 1 ? 4 : 3) : DP == 128 && NQ == 1 ? 3 : 2;  // paged_mma_ctas()
  static constexpr bool QREG = DP <= 128;               // the queries' fragments stay in registers
};

template <int KIND, int DP, int NQ, bool TILES, bool REST>
__global__ void __launch_bounds__(kPgThreads, PmShape<KIND, DP, NQ>::CTAS)
    paged_mma_kernel(const __grid_constant__ PagedParams p, int dtype, int by_warp) {
  using S = PmShape<KIND, DP, NQ>;
  constexpr int KB = S::KB, KT = S::KT, KC = S::KC, VC = S::VC, VW = S::VW, VE = S::VE;
  constexpr bool CODES = S::CODES, BF = KIND == KIND_BF16;
  constexpr float LIFT = BF ? 0.0f : kPmLift;
  constexpr int RING = 2;                // parts known at once: the one at work and the next
  constexpr int QROW = DP * 2 + 16;      // bytes of a query, padded: eight queries' vectors in distinct banks
  extern __shared__ __align__(16) unsigned char pm_raw[];  // [warp][2][8 NQ] queries; with four warps to a part then [warp][8 NQ][DP] sums
  __shared__ PgShare share;
  __shared__ PgPart ring[kPgWarps][RING];
  __shared__ float wm[kPgWarps][8 * NQ], wl[kPgWarps][8 * NQ];
  __shared__ int flag[kPgWarps];
  __shared__ int32_t first_page[kPgWarps][TILES ? KT : 1][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int W = by_warp ? 1 : kPgWarps, wi = by_warp ? 0 : warp;
  constexpr int CB = CODES ? 1 : 2;      // bytes of a cache element
  constexpr uint32_t ALL = KB == 32 ? ~0u : 0xffffu;
  const int line = p.dim * CB;
  const bool exact = p.dim == DP;
  bool bad = false;
  unsigned char* my_q = pm_raw + warp * 2 * 8 * NQ * QROW;
  float* acc = reinterpret_cast<float*>(pm_raw + kPgWarps * 2 * 8 * NQ * QROW);

  PgWalk<KB> walk(p, share, by_warp ? blockIdx.x * kPgWarps + warp : blockIdx.x, warp, lane);
  auto next_part = [&](int slot) {
    PgPart y;
    if (!walk.next(y)) return false;
    if (lane == 0) ring[warp][slot] = y;
    __syncwarp();
    return true;
  };

  // ---- the block that is looked up next.  TILES: 16 keys lie in one page.  Otherwise lane n looks up key n.
  constexpr int NP = TILES ? KT : 1;
  int page[NP], place[NP];
  auto look_up = [&](const PgPart& y, int blk) {
    const int hi = y.hi, len = y.len;
    const long long table = (long long)y.r * p.pages.table_row;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      page[k] = -1;
      const int n = blk * KB + (TILES ? 16 * k : lane);
      if ((TILES || lane < KB) && blk < hi) page[k] = pg_page(p, table, n, len, place[k], bad);
    }
  };

  // ---- the block that is fetched, the one looked up before
  uint32_t seen = 0;           // the keys that are there
  float ks = 0.0f, vl = 0.0f;  // of key `lane`: the key's and the value's scale
  uint4 kr[KT][2][KC];
  uint32_t vr[KT][4][VC][VW];
  long long voff[NP];
  auto fetch_keys = [&](const PgPart& y, int blk) {
    const long long h = y.h;
    if constexpr (TILES) {
      const int len = y.len;
      seen = 0;
#pragma unroll
      for (int k = 0; k < KT; ++k)
        if (page[k] >= 0) seen |= (0xffffu >> max(16 - (len - (blk * KB + 16 * k)), 0)) << 16 * k;
    } else {
      seen = __ballot_sync(~0u, page[0] >= 0);
    }
    long long koff[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      koff[k] = voff[k] = 0;
      if (page[k] >= 0) {
        koff[k] = h * p.pages.key.head + (long long)page[k] * p.pages.key.row + (long long)place[k] * p.pages.key.pos;
        voff[k] = h * p.pages.value.head + (long long)page[k] * p.pages.value.row + (long long)place[k] * p.pages.value.pos;
      }
    }
    if constexpr (CODES) {
      ks = vl = 0.0f;
      if ((seen >> lane) & 1u) {
        const bool up = TILES && KT > 1 && lane >= 16;
        const int pg = up ? page[NP - 1] : page[0];
        const long long pl = TILES ? (up ? place[NP - 1] : place[0]) + (lane & 15) : place[0];
        ks = __ldg(reinterpret_cast<const float*>(p.pages.kscale.data + h * p.pages.kscale.head + (long long)pg * p.pages.kscale.row +
                                                  pl * p.pages.kscale.pos));
        vl = __ldg(reinterpret_cast<const float*>(p.pages.vscale.data + h * p.pages.vscale.head + (long long)pg * p.pages.vscale.row +
                                                  pl * p.pages.vscale.pos));
      }
    }
    const bool whole = seen == ALL && exact;
    const unsigned char* base = p.pages.key.data + t * 16 + (TILES ? g * p.pages.key.pos : 0);
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int key = k * 16 + hf * 8 + g;
        const unsigned char* at = base + (TILES ? koff[TILES ? k : 0] + hf * 8 * p.pages.key.pos : __shfl_sync(~0u, koff[0], key));
        const bool ok = (seen >> key) & 1u;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          if (whole)
            kr[k][hf][i] = stream16(at + i * 64);
          else
            kr[k][hf][i] = ok && t * 16 + i * 64 < line ? stream16(at + i * 64) : make_uint4(0u, 0u, 0u, 0u);
        }
      }
  };
  auto fetch_values = [&]() {
    const bool whole = seen == ALL && exact;
    const unsigned char* base = p.pages.value.data + g * S::VB + (TILES ? 2 * t * p.pages.value.pos : 0);
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k * 16 + 2 * t + (j & 1) + (j >> 1) * 8;
        const unsigned char* at =
            base + (TILES ? voff[TILES ? k : 0] + ((j & 1) + (j >> 1) * 8) * p.pages.value.pos : __shfl_sync(~0u, voff[0], key));
        const bool ok = (seen >> key) & 1u;
#pragma unroll
        for (int i = 0; i < VC; ++i) {
          const bool there = whole || (ok && g * S::VB + i * 8 * S::VB < line);
          if constexpr (VW == 4) {
            const uint4 d = there ? stream16(at + i * 8 * S::VB) : make_uint4(0u, 0u, 0u, 0u);
            vr[k][j][i][0] = d.x;
            vr[k][j][i][1] = d.y;
            vr[k][j][i][2] = d.z;
            vr[k][j][i][3] = d.w;
          } else {
            const uint2 d = there ? stream8(at + i * 8 * S::VB) : make_uint2(0u, 0u);
            vr[k][j][i][0] = d.x;
            vr[k][j][i][1] = d.y;
          }
        }
      }
  };
  // the queries of the ring's part `slot` into its half of the warp's buffer
  auto fetch_queries = [&](int slot) {
    const PgPart& y = ring[warp][slot];
    unsigned char* to = my_q + (slot & 1) * 8 * NQ * QROW;
    const unsigned char* from = p.q.data + (long long)y.r * p.q.row + (long long)(y.h * p.group + y.i0) * p.q.head;
    constexpr int CH = DP / 8;  // 16-byte pieces
    const int nq = y.nq;
    for (int n = lane; n < nq * CH; n += 32) {
      const int q = n / CH, c = n % CH;
      const bool there = c * 8 < p.dim;
      cp_async16_fill(smem_addr(to + q * QROW + c * 16), there ? from + (long long)q * p.q.head + c * 16 : p.q.data, there ? 16 : 0);
    }
    cp_async_commit();
  };

  // the page numbers of a part's first block, for take_pages later
  auto fetch_pages = [&](const PgPart& y, int blk) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int n = blk * KB + (TILES ? 16 * k : lane);
      const bool there = (TILES || lane < KB) && blk < y.hi && n < y.len;
      const int32_t* from = p.pages.table + (long long)y.r * p.pages.table_row + (there ? p.pages.by_page(n) : 0);
      if (there) cp_async4(smem_addr(&first_page[warp][k][lane]), from);
    }
    cp_async_commit();
  };
  auto take_pages = [&](const PgPart& y, int blk) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int n = blk * KB + (TILES ? 16 * k : lane);
      page[k] = -1;
      if ((TILES || lane < KB) && blk < y.hi && n < y.len) {
        place[k] = n - p.pages.by_page(n) * p.pages.page_size;
        const int pg = first_page[warp][k][lane];
        if ((unsigned)pg < (unsigned)p.pages.num_pages)
          page[k] = pg;
        else
          bad = true;
      }
    }
  };

  int cp = 0;  // the part at work
  bool work = next_part(0);
  if (work) {
    look_up(ring[warp][0], ring[warp][0].lo + wi);
    fetch_queries(0);
    fetch_keys(ring[warp][0], ring[warp][0].lo + wi);
    fetch_values();
  }

  uint32_t qf[S::QREG ? NQ : 1][S::QREG ? DP / 8 : 1];
  float cs[NQ][2];  // of the lane's columns, query 8 a + 2 t + e: what a product is multiplied by
  float m[NQ][2], z[NQ][2], l[NQ][2], o[DP / 16][NQ][4];
#pragma unroll 1
  while (work) {
    const PgPart& x = ring[warp][cp];
    int b = x.lo + wi;
    uint32_t seen_now = seen;
    float ks_now = ks, vl_now = vl;
    const int x_hi = x.hi;
    look_up(x, b + W);
    // what the next part needs first is under way while this one is at work: its queries and its pages' numbers
    work = next_part(cp ^ 1);
    {
      cp_async_wait<0>();
      __syncwarp();
      if (work) {
        fetch_queries(cp ^ 1);
        fetch_pages(ring[warp][cp ^ 1], ring[warp][cp ^ 1].lo + wi);
      }
      const unsigned char* src = my_q + (cp & 1) * 8 * NQ * QROW + g * QROW;
#pragma unroll
      for (int a = 0; a < NQ; ++a) {
        // lane (g, t): the elements of query 8 a + g that meet the keys' in its registers
        uint32_t f[DP / 8];
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) {
          // 16-bit pages: 16 bytes t + 4 i; codes: 32 bytes t + 4 (i / 2), in halves
          const uint4 d = a * 8 + g < x.nq ? *reinterpret_cast<const uint4*>(src + a * 8 * QROW + (CODES ? (t + 4 * (i / 2)) * 32 + (i % 2) * 16 : (t + 4 * i) * 16))
                                           : make_uint4(0u, 0u, 0u, 0u);
          f[4 * i] = d.x;
          f[4 * i + 1] = d.y;
          f[4 * i + 2] = d.z;
          f[4 * i + 3] = d.w;
        }
        cs[a][0] = cs[a][1] = p.scale_log2;
        if constexpr (CODES) {
          if (dtype == DT_BF16) {  // to f16 by a power of two per query: exact but for what is under 2^-39 of its largest
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) top = max(top, max(f[i] & 0x7fffu, (f[i] >> 16) & 0x7fffu));
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            const int up = min(max(127 + 14 - (int)(top >> 7), -112), 126);  // (bf16's exponent; 2^up is a normal f32)
            const float mul = __uint_as_float((uint32_t)(up + 127) << 23);
#pragma unroll
            for (int i = 0; i < DP / 8; ++i)
              f[i] = half2_bits(__uint_as_float(f[i] << 16) * mul, __uint_as_float(f[i] & 0xffff0000u) * mul);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int u = __shfl_sync(~0u, up, (2 * t + e) * 4);
              cs[a][e] = p.scale_log2 * __uint_as_float((uint32_t)(127 - u) << 23);
            }
          }
        }
        if constexpr (S::QREG) {
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) qf[a][i] = f[i];
        } else {  // (as f16, and zeros past the last query, in place)
          unsigned char* to = my_q + (cp & 1) * 8 * NQ * QROW + (a * 8 + g) * QROW;
#pragma unroll
          for (int i = 0; i < DP / 32; ++i)
            *reinterpret_cast<uint4*>(to + (CODES ? (t + 4 * (i / 2)) * 32 + (i % 2) * 16 : (t + 4 * i) * 16)) =
                make_uint4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        }
        m[a][0] = m[a][1] = z[a][0] = z[a][1] = -INFINITY;
        l[a][0] = l[a][1] = 0.0f;
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) o[j][a][0] = o[j][a][1] = o[j][a][2] = o[j][a][3] = 0.0f;
      }
    }
#pragma unroll 1
    do {
      // S^T = K Q^T
      float s[KT][NQ][4];
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int a = 0; a < NQ; ++a) s[k][a][0] = s[k][a][1] = s[k][a][2] = s[k][a][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        constexpr int PER = CODES ? 4 : 2;  // products of 16 elements per load
#pragma unroll
        for (int y = 0; y < PER; ++y) {
          uint32_t qb[NQ][2];
#pragma unroll
          for (int a = 0; a < NQ; ++a) {
            if constexpr (S::QREG) {
              qb[a][0] = qf[a][(i * PER + y) * 2];
              qb[a][1] = qf[a][(i * PER + y) * 2 + 1];
            } else {
              const int at = CODES ? (t + 4 * i) * 32 + y * 8 : (t + 4 * i) * 16 + y * 8;
              const uint2 d = *reinterpret_cast<const uint2*>(my_q + (cp & 1) * 8 * NQ * QROW + (a * 8 + g) * QROW + at);
              qb[a][0] = d.x;
              qb[a][1] = d.y;
            }
          }
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            const uint4 &u = kr[k][0][i], &v = kr[k][1][i];
            uint32_t a0, a1, a2, a3;
            if constexpr (CODES) {
              const uint32_t uw = y == 0 ? u.x : y == 1 ? u.y : y == 2 ? u.z : u.w, vw = y == 0 ? v.x : y == 1 ? v.y : y == 2 ? v.z : v.w;
              codes_half<KIND>(uw, a0, a2);
              codes_half<KIND>(vw, a1, a3);
            } else {
              a0 = y == 0 ? u.x : u.z;
              a1 = y == 0 ? v.x : v.z;
              a2 = y == 0 ? u.y : u.w;
              a3 = y == 0 ? v.y : v.w;
            }
#pragma unroll
            for (int a = 0; a < NQ; ++a) mma16816<BF>(s[k][a], a0, a1, a2, a3, qb[a][0], qb[a][1]);
          }
        }
      }
      const bool more = b + W < x_hi;
      if (more) fetch_keys(x, b + W);

      // the scores in powers of two
      float lv[KT][2];  // the value scale's logarithm of keys 16 k + 8 hf + g
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float sk = 1.0f;
          if constexpr (CODES) {
            sk = __shfl_sync(~0u, ks_now, k * 16 + hf * 8 + g);
            lv[k][hf] = __shfl_sync(~0u, log2_of(vl_now), k * 16 + hf * 8 + g);
          }
#pragma unroll
          for (int a = 0; a < NQ; ++a)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[k][a][2 * hf + e] *= CODES ? sk * cs[a][e] : cs[a][e];
        }
      if (seen_now != ALL) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            if (!((seen_now >> (k * 16 + hf * 8 + g)) & 1u)) {
              lv[k][hf] = 0.0f;
#pragma unroll
              for (int a = 0; a < NQ; ++a) s[k][a][2 * hf] = s[k][a][2 * hf + 1] = -INFINITY;
            }
      }
      // The references are raised, over all lanes, only when some lane's own largest has grown by more
      // than 2^8; until then weights are at most 2^8 times as large, which the sums and types hold.
      float top[NQ][2], topz[NQ][2];
      bool grown = false;
#pragma unroll
      for (int a = 0; a < NQ; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[a][e] = -INFINITY;
          topz[a][e] = -INFINITY;
#pragma unroll
          for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              top[a][e] = fmaxf(top[a][e], s[k][a][2 * hf + e]);
              if constexpr (CODES) topz[a][e] = fmaxf(topz[a][e], s[k][a][2 * hf + e] + lv[k][hf]);
            }
          if constexpr (CODES)
            grown |= top[a][e] > m[a][e] + kPmLazy || topz[a][e] - LIFT > z[a][e] + kPmLazy;
          else
            grown |= top[a][e] - LIFT > m[a][e] + kPmLazy;
        }
      if (__any_sync(~0u, grown)) {
#pragma unroll
        for (int a = 0; a < NQ; ++a) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) {
              top[a][e] = fmaxf(top[a][e], __shfl_xor_sync(~0u, top[a][e], w));
              if constexpr (CODES) topz[a][e] = fmaxf(topz[a][e], __shfl_xor_sync(~0u, topz[a][e], w));
            }
            const float mn = fmaxf(m[a][e], CODES ? top[a][e] : top[a][e] - LIFT);
            const float fm = fast_exp2(m[a][e] - (mn == -INFINITY ? 0.0f : mn));
            l[a][e] *= fm;
            m[a][e] = mn;
            f[e] = fm;
            if constexpr (CODES) {
              const float zn = fmaxf(z[a][e], topz[a][e] - LIFT);
              f[e] = fast_exp2(z[a][e] - (zn == -INFINITY ? 0.0f : zn));
              z[a][e] = zn;
            }
          }
#pragma unroll
          for (int j = 0; j < DP / 16; ++j) {
            o[j][a][0] *= f[0];
            o[j][a][1] *= f[1];
            o[j][a][2] *= f[0];
            o[j][a][3] *= f[1];
          }
        }
      }
      uint32_t pb[KT][NQ][2], pr[KT][NQ][2];  // the weights, and (REST) their remainders
#pragma unroll
      for (int a = 0; a < NQ; ++a) {
        float sub[2], subz[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sub[e] = m[a][e] == -INFINITY ? 0.0f : m[a][e];
          subz[e] = z[a][e] == -INFINITY ? 0.0f : z[a][e];
        }
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float y = s[k][a][2 * hf + e], w1 = fast_exp2(y - sub[e]);
              l[a][e] += w1;
              w[e] = CODES ? fast_exp2(y + lv[k][hf] - subz[e]) : w1;
            }
            const uint32_t most = pack_pair<BF>(w[0], w[1]);
            pb[k][a][hf] = transpose8(most);
            if constexpr (REST) pr[k][a][hf] = transpose8(rest_of<BF>(w[0], w[1], most));
          }
      }

      // O^T += V^T P^T
#pragma unroll
      for (int i = 0; i < VC; ++i)
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            const uint32_t v0 = vr[k][0][i][w], v1 = vr[k][1][i][w], v2 = vr[k][2][i][w], v3 = vr[k][3][i][w];
            if constexpr (CODES) {
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                uint32_t a0, a1, a2, a3;
                codes_half<KIND>(__byte_perm(v0, v1, hh ? 0x7362 : 0x5140), a0, a1);
                codes_half<KIND>(__byte_perm(v2, v3, hh ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                for (int a = 0; a < NQ; ++a) {
                  mma16816<BF>(o[(i * VW + w) * 2 + hh][a], a0, a1, a2, a3, pb[k][a][0], pb[k][a][1]);
                  if constexpr (REST) mma16816<BF>(o[(i * VW + w) * 2 + hh][a], a0, a1, a2, a3, pr[k][a][0], pr[k][a][1]);
                }
              }
            } else {
              const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
              const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
#pragma unroll
              for (int a = 0; a < NQ; ++a) {
                mma16816<BF>(o[i * VW + w][a], a0, a1, a2, a3, pb[k][a][0], pb[k][a][1]);
                if constexpr (REST) mma16816<BF>(o[i * VW + w][a], a0, a1, a2, a3, pr[k][a][0], pr[k][a][1]);
              }
            }
          }
      if (more) {
        fetch_values();
        seen_now = seen;
        ks_now = ks;
        vl_now = vl;
        look_up(x, b + 2 * W);
      }
      b += W;
    } while (b < x_hi);
    if (work) {
      cp_async_wait<0>();
      __syncwarp();
      const PgPart& y = ring[warp][cp ^ 1];
      take_pages(y, y.lo + wi);
      fetch_keys(y, y.lo + wi);
      fetch_values();
    }

    // the lanes' sums; weighted values in units of 2^-m
#pragma unroll
    for (int a = 0; a < NQ; ++a) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[a][e] += __shfl_xor_sync(~0u, l[a][e], w);
        f[e] = m[a][e] == -INFINITY ? 0.0f : fast_exp2(z[a][e] - m[a][e]);
      }
      if constexpr (CODES) {
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
          o[j][a][0] *= f[0];
          o[j][a][1] *= f[1];
          o[j][a][2] *= f[0];
          o[j][a][3] *= f[1];
        }
      }
    }
    const bool out_bf = CODES ? dtype == DT_BF16 : BF;
    if (by_warp) {
#pragma unroll
      for (int a = 0; a < NQ; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int q = a * 8 + 2 * t + e;
          if (q >= x.nq) continue;
          const float inv = l[a][e] == 0.0f ? 0.0f : 1.0f / l[a][e];
          const long long row = x.parts == 1 ? 0 : (long long)pg_slot(x.base, x.part) * p.tile + q;
          if (x.parts > 1 && g == 0) p.part_ml[row] = make_float2(m[a][e], l[a][e]);
#pragma unroll
          for (int i = 0; i < VC; ++i) {
            const int d = (g + 8 * i) * VE;
            if (d >= p.dim) continue;
#pragma unroll
            for (int w = 0; w < VE; w += 8) {
              float y[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] = o[(i * VE + w + j) / 2][a][(j & 1) * 2 + e];
              if (x.parts == 1) {
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  h[j] = out_bf ? pack_pair<true>(y[2 * j] * inv, y[2 * j + 1] * inv) : pack_pair<false>(y[2 * j] * inv, y[2 * j + 1] * inv);
                *reinterpret_cast<uint4*>(pg_out(p, x, q) + (d + w) * 2) = make_uint4(h[0], h[1], h[2], h[3]);
              } else {
                float4* to = reinterpret_cast<float4*>(p.part_o + row * p.dim + d + w);
                to[0] = make_float4(y[0], y[1], y[2], y[3]);
                to[1] = make_float4(y[4], y[5], y[6], y[7]);
              }
            }
          }
        }
      if (x.parts > 1 && pg_last(p, x, lane, &flag[warp], [] { __syncwarp(); })) pg_join(p, x, dtype, 0, 1, lane);
    } else {
#pragma unroll
      for (int a = 0; a < NQ; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int q = a * 8 + 2 * t + e;
          if (g == 0) {
            wm[warp][q] = m[a][e];
            wl[warp][q] = l[a][e];
          }
          if (q >= x.nq) continue;
#pragma unroll
          for (int i = 0; i < VC; ++i)
#pragma unroll
            for (int w = 0; w < VE; w += 4)
              *reinterpret_cast<float4*>(acc + (warp * 8 * NQ + q) * DP + (g + 8 * i) * VE + w) =
                  make_float4(o[(i * VE + w) / 2][a][e], o[(i * VE + w) / 2][a][2 + e], o[(i * VE + w) / 2 + 1][a][e],
                              o[(i * VE + w) / 2 + 1][a][2 + e]);
        }
      __syncthreads();
      const int quads = p.dim / 4;
      for (int n = threadIdx.x; n < x.nq * quads; n += kPgThreads) {
        const int q = n / quads, d = (n - q * quads) * 4;
        float M = wm[0][q];
#pragma unroll
        for (int w = 1; w < kPgWarps; ++w) M = fmaxf(M, wm[w][q]);
        const float sub = M == -INFINITY ? 0.0f : M;
        float L = 0.0f;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kPgWarps; ++w) {
          const float f = fast_exp2(wm[w][q] - sub);
          const float4 v = *reinterpret_cast<const float4*>(acc + (w * 8 * NQ + q) * DP + d);
          L = fmaf(f, wl[w][q], L);
          y.x = fmaf(f, v.x, y.x);
          y.y = fmaf(f, v.y, y.y);
          y.z = fmaf(f, v.z, y.z);
          y.w = fmaf(f, v.w, y.w);
        }
        if (x.parts == 1) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          uint2 h;
          h.x = out_bf ? pack_pair<true>(y.x * inv, y.y * inv) : pack_pair<false>(y.x * inv, y.y * inv);
          h.y = out_bf ? pack_pair<true>(y.z * inv, y.w * inv) : pack_pair<false>(y.z * inv, y.w * inv);
          *reinterpret_cast<uint2*>(pg_out(p, x, q) + d * 2) = h;
        } else {
          const long long row = (long long)pg_slot(x.base, x.part) * p.tile + q;
          *reinterpret_cast<float4*>(p.part_o + row * p.dim + d) = y;
          if (d == 0) p.part_ml[row] = make_float2(M, L);
        }
      }
      if (x.parts > 1) {
        if (pg_last(p, x, threadIdx.x, &flag[0], [] { __syncthreads(); })) pg_join(p, x, dtype, warp, kPgWarps, lane);
      }
      __syncthreads();
    }
    cp ^= 1;
  }
  if (bad) atomicOr(p.status, kDevInternal);
  if (blockIdx.x == 0) {  // lengths out of range
    for (int r = threadIdx.x; r < p.rows; r += kPgThreads) {
      const int n = __ldg(p.len + r);
      if (n < 0 || n > p.pages.places) atomicOr(p.status, kDevInternal);
    }
  }
}

template <int KIND, int DP, int NQ, bool REST>
cudaError_t run_paged(const PagedParams& p, int dtype, bool by_warp, cudaStream_t stream) {
  const unsigned grid = (unsigned)(by_warp ? p.workers / kPgWarps : p.workers);
  constexpr int QUERIES = kPgWarps * 2 * 8 * NQ * (DP * 2 + 16), SUMS = kPgWarps * 8 * NQ * DP * 4;
  const int bytes = QUERIES + (by_warp ? 0 : SUMS);
  auto kernel = p.pages.page_size % 16 == 0 ? paged_mma_kernel<KIND, DP, NQ, true, REST> : paged_mma_kernel<KIND, DP, NQ, false, REST>;
  static std::atomic<uint64_t> allowed[2];
  const cudaError_t e = allow_shared(kernel, QUERIES + SUMS, allowed[p.pages.page_size % 16 == 0]);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kPgThreads, bytes, stream>>>(p, dtype, by_warp);
  return cudaGetLastError();
}

template <int KIND, bool REST>
cudaError_t run_paged_dim(const PagedParams& p, int dtype, bool by_warp, cudaStream_t stream) {
  if (p.dim <= 64) return p.tile <= 8 ? run_paged<KIND, 64, 1, REST>(p, dtype, by_warp, stream) : run_paged<KIND, 64, 2, REST>(p, dtype, by_warp, stream);
  if (p.dim <= 128) return p.tile <= 8 ? run_paged<KIND, 128, 1, REST>(p, dtype, by_warp, stream) : run_paged<KIND, 128, 2, REST>(p, dtype, by_warp, stream);
  return run_paged<KIND, 256, 1, REST>(p, dtype, by_warp, stream);
}

}  // namespace
}  // namespace lsb
