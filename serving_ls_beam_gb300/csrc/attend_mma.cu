// Attention of few queries over a row's keys (f16 / bf16): the decode step with shared key
// heads, small trees, the beams of a sentence.  With M queries per key the products take M flops
// per byte of keys and values read, far below what the tensor cores need to be the limit, so this
// kernel is built around the stream of keys and values from memory and uses the warp-level
// matrix instructions (m16n8k16, f32 accumulators in registers).
//
//   S^T = K Q^T,  P = exp2(c S - max),  O^T = O^T * correction + V^T P^T,  out = O / sum P
//
// in one pass with the running maximum and sum of the softmax (Milakov and Gimelshein, 2018).
// The products are taken transposed, keys (and head elements) as the instruction's 16 rows and
// queries as its 8 columns, so that 1 to 8 queries fill what 16 rows would leave empty: half the
// instructions and accumulators.  P is rounded to the tensors' type for the second product (its
// error averages out over the keys like the values' own rounding) and turned into that product's
// operand by an 8 x 8 transpose in registers; the sums use the unrounded f32 weights.
//
// A warp streams blocks of KB keys and their values through a ring of its own in shared memory,
// no CTA barrier in the stream: whole blocks by TMA (one lane, a mbarrier per ring slot, the
// 128-byte swizzle for conflict-free ldmatrix), a row's last block by 16-byte asynchronous
// copies of all lanes into the same layout.  There the drafted tokens follow the row's keys
// without a gap, and zeros fill the block, so that nothing past the row's end reaches a product.
// Two ways to share the work out, by AttendParams::warps:
//   1: a warp takes whole problems, one after the other, and its ring runs ahead into the next
//      problem (its queries and parents come through the ring as well), so that short rows
//      stream without a gap;
//   4: the CTA's four warps take the blocks of one (part of a) problem in turn and merge their
//      results in shared memory.
//
// What bounds it: the instructions around the products (a block's turn takes some 300 per warp for
// 8 KB of keys and values), so the number of warps an SM holds counts (12, by two ring slots each
// and by registers; a third slot in place of the third CTA: 66 against 52 us on the first of these).
// Single-token step of 1024 beams x 16 heads of 64 elements, 48 to 63 positions: 239 MB in 42 us,
// 0.84 of the measured copy rate; 128 trees of 13 nodes over 300 to 999 positions: 354 MB in 68 us,
// 0.77; 64 rows x 8 key heads of 128 elements, 4 queries, 500 to 3000 positions: 460 MB in 86 us,
// 0.79.  With 16 rows of queries in place of 8 columns the first took 98 us.
#include "ls_device.cuh"
#include "ls_dtype.cuh"
#include "ls_tc.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

constexpr int kMmWarps = 4;
constexpr int kMmThreads = kMmWarps * 32;
constexpr long long kMmDrainNs = 2000000000LL;
constexpr float kMmLazy = 8.0f;  // growth of the maximum (log2) that is let pass

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& x) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// The 8 x 8 matrix of 16-bit values whose row g lane (g, t) holds two of, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int DP, int NQ>
struct MmaShape {
  static constexpr int KB = DP == 64 ? 32 : 16;        // keys per block
  static constexpr int NS = 2;                         // blocks in the ring
  static constexpr int PANELS = DP / 64;
  static constexpr int PANEL = KB * 128;               // a block's rows of 64 elements
  static constexpr int STAGE = 2 * PANELS * PANEL;     // keys, then values
  static constexpr bool QREG = NQ * DP <= 256;         // the queries' fragments stay in registers
  // CTAs per SM: three by the rings, 64 KB a CTA (128 KB for heads above 128: one); two by registers from 32
  // queries of 64 elements or 16 of 128 on.  (With four as the cap, which the rings do not allow, eight queries
  // of 64 elements had 128 registers and the first example above took 41.8 us; now 158 registers, 41.6 us.)
  static constexpr int CTAS = DP > 128 ? 1 : NQ * DP <= 128 ? 3 : 2;
  static_assert(CTAS * (kMmWarps * NS * STAGE + 1024) <= 228 * 1024, "what an SM's shared memory holds");
};

// Bytes of one warp's shared memory after its ring, and where the parts begin.  With four warps
// to an item there is one item, otherwise one set of queries and parents per ring slot.
struct MmaSmem {
  int bars, q, q_one, q_row, par, par_one, tree, total;
};
template <int DP, int NQ>
__host__ __device__ inline MmaSmem mma_smem(int m, int nodes, int warps) {
  using S = MmaShape<DP, NQ>;
  const int sets = warps == 1 ? S::NS : 1;
  MmaSmem s;
  s.bars = 0;
  s.q = 16 * ((S::NS * 8 + 15) / 16);
  s.q_row = DP * 2 + 16;  // padded: eight queries' vectors in distinct banks
  s.q_one = (S::QREG && m < 8 * NQ ? m : 8 * NQ) * s.q_row;
  s.par = s.q + sets * s.q_one;
  s.par_one = (nodes + 3) / 4 * 16;
  s.tree = s.par + sets * s.par_one;
  s.total = (s.tree + tree_bytes(nodes) + 15) / 16 * 16;
  return s;
}
template <int DP, int NQ>
inline int mma_smem_bytes(int m, int nodes, int warps) {
  return kMmWarps * (MmaShape<DP, NQ>::NS * MmaShape<DP, NQ>::STAGE + mma_smem<DP, NQ>(m, nodes, warps).total) + 1024;
}

// One item: the problem, the first of its queries, and the blocks b, b + W, .. < b_end of this
// warp over the row's keys and drafted tokens.
struct MmaItem {
  int r, h, i0, nq, split, len, b, b_end;
};

template <int KB, int NQ>
__device__ __forceinline__ MmaItem open_item(const AttendParams& p, int it, int len, int w) {
  MmaItem x;
  const int a = p.by_split(it);
  x.split = it - a * p.splits;
  const int b = p.by_tile(a);
  x.i0 = (a - b * p.m_tiles) * 8 * NQ;
  x.r = p.by_head(b);
  x.h = b - x.r * p.kv_heads;
  x.nq = min(8 * NQ, p.m - x.i0);
  x.len = min(max(len, 0), p.max_len);
  const int nbt = (x.len + p.nodes + KB - 1) / KB;
  const int per = p.splits == 1 ? nbt : (nbt + p.splits - 1) / p.splits;
  const int lo = min(x.split * per, nbt);
  x.b = lo + w;
  x.b_end = min(lo + per, nbt);
  // a warp without a block takes an empty one, so that every item has a stage in the ring
  if (x.b >= x.b_end) x.b = x.b_end = -1;
  return x;
}
__device__ __forceinline__ int item_row(const AttendParams& p, int it) { return p.by_head(p.by_tile(p.by_split(it))); }

template <bool BF, int DP, int NQ>
__global__ void __launch_bounds__(kMmThreads, MmaShape<DP, NQ>::CTAS)
    attend_mma_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const AttendParams p) {
  using S = MmaShape<DP, NQ>;
  constexpr int KB = S::KB, NS = S::NS, KT = KB / 16, DT = BF ? DT_BF16 : DT_F16;
  constexpr int CPR = DP / 8, RPI = 32 / CPR;  // 16-byte vectors of a row; rows per copy instruction
  extern __shared__ unsigned char mm_raw[];
  __shared__ float wm[kMmWarps][8 * NQ], wl[kMmWarps][8 * NQ];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int W = p.warps, wi = W == 1 ? 0 : warp, sets = W == 1 ? NS : 1;
  const MmaSmem sm = mma_smem<DP, NQ>(p.m, p.nodes, W);
  const uint32_t raw = smem_addr(mm_raw), rings = (raw + 1023u) & ~1023u;  // the swizzle's period
  const uint32_t ring = rings + warp * NS * S::STAGE;
  unsigned char* mine = mm_raw + (rings - raw) + kMmWarps * NS * S::STAGE + warp * sm.total;
  const uint32_t base = smem_addr(mine);
  const TreeSeen tree = tree_at(mine + sm.tree, p.nodes);
  const int chunks = p.dim / 8;
  const int kd = (p.dim + 15) / 16;  // 16-element steps of a head
  const float c = p.scale_log2;      // positive: a negative scale is in Q's sign
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(base + sm.bars + 8 * i, 1);
    fence_barrier_init();
  }
  __syncwarp();
  // of a block in panels of 64 elements: byte offset of 16-byte vector c of row r.  The products'
  // operands: a lane's offset for the first 16 elements; later ones differ in two bits of it.
  auto at = [&](int r, int c) { return (uint32_t)((c >> 3) * S::PANEL + r * 128 + (((c & 7) ^ (r & 7)) << 4)); };
  const uint32_t k_lane = at(lane & 15, lane >> 4), v_lane = at((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);
  const uint32_t flip = p.negate ? 0x80008000u : 0u;  // a negative scale: the queries' signs
  // (unsigned: an item's number plus the stride, each below 2^31, may pass it)
  const uint32_t items = (uint32_t)p.items;
  const uint32_t stride = W == 1 ? gridDim.x * kMmWarps : gridDim.x;
  const uint32_t first = W == 1 ? blockIdx.x * kMmWarps + warp : blockIdx.x;

  // ---- the ring's filling side: item `fi` (its length loaded one item ahead), block `fx.b`
  const int fc = lane % CPR, fr = lane / CPR;  // this lane's vector of a row, and its row of a copy
  const bool fcv = fc < chunks;
  const int fsz = fcv ? 16 : 0, fo = fcv ? fc * 16 : 0;
  uint32_t fi = first;
  int f_seq = 0, f_slot = 0;
  bool f_new = true;
  MmaItem fx{};
  int f_len = fi < items ? __ldg(p.len + item_row(p, fi)) : 0;
  bool timed_out = false;
  uint32_t pending = 0;  // bit i: a TMA copy into slot i is under way
  auto fill = [&]() {
    if (fi < items && !timed_out) {
      if (f_new) {
        fx = open_item<KB, NQ>(p, fi, f_len, wi);
        if (fi + stride < items) f_len = __ldg(p.len + item_row(p, fi + stride));
        const uint32_t qd = base + sm.q + f_seq * sm.q_one;
        // (ldmatrix reads all places: those past the last query are zeros, so that their scores, which say
        // when the maximum is reduced, do not depend on what lay there)
        const int places = S::QREG ? fx.nq : 8 * NQ;
        for (int i = fr; i < places; i += RPI) {
          const bool there = i < fx.nq;
          const unsigned char* from = there ? p.q.data + query_offset(p, p.q, fx.r, fx.h, fx.i0 + i) + fo : p.q.data;
          cp_async16_fill(qd + i * sm.q_row + fc * 16, from, there ? fsz : 0);
        }
        for (int i = lane; i < p.nodes; i += 32)
          cp_async4(base + sm.par + f_seq * sm.par_one + i * 4, p.parent + (long long)fx.r * p.nodes + i);
        f_seq = f_seq + 1 == sets ? 0 : f_seq + 1;
        f_new = false;
      }
      const uint32_t kd_ = ring + f_slot * S::STAGE, vd_ = kd_ + S::PANELS * S::PANEL;
      if (fx.b >= 0 && fx.b * KB + KB <= fx.len) {
        pending |= 1u << f_slot;
        if (lane == 0) {
          const uint32_t bar = base + sm.bars + 8 * f_slot;
          const int h = p.kv_head_one ? 0 : fx.h, r = p.kv_row_one ? 0 : fx.r;
          // the slot's last contents may have come by the lanes' own copies and stores
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_arrive_expect_tx(bar, S::STAGE);
#pragma unroll
          for (int c = 0; c < S::PANELS; ++c) {
            tma_load_4d(kd_ + c * S::PANEL, &map_k, c * 64, fx.b * KB, h, r, bar);
            tma_load_4d(vd_ + c * S::PANEL, &map_v, c * 64, fx.b * KB, h, r, bar);
          }
        }
      } else {  // the row's last block: its drafted tokens, then zeros
        const int total = fx.b >= 0 ? fx.len + p.nodes : 0;
        const int j0 = fx.b * KB + fr;
        const unsigned char* fk = p.key.data + (long long)fx.r * p.key.row + (long long)fx.h * p.key.head + fo;
        const unsigned char* fv = p.value.data + (long long)fx.r * p.value.row + (long long)fx.h * p.value.head + fo;
        const unsigned char* dk = p.dkey.data + (long long)fx.r * p.dkey.row + (long long)fx.h * p.dkey.head + fo;
        const unsigned char* dv = p.dvalue.data + (long long)fx.r * p.dvalue.row + (long long)fx.h * p.dvalue.head + fo;
        // the lane's place in the cache and among the drafted tokens, advanced row by row of its copies
        const unsigned char* ck = fk + j0 * p.key.pos;
        const unsigned char* cv = fv + j0 * p.value.pos;
        const unsigned char* nk = dk + (j0 - fx.len) * p.dkey.pos;
        const unsigned char* nv = dv + (j0 - fx.len) * p.dvalue.pos;
        const long long ks = RPI * p.key.pos, vs = RPI * p.value.pos, nks = RPI * p.dkey.pos, nvs = RPI * p.dvalue.pos;
#pragma unroll
        for (int u = 0; u < KB / RPI; ++u) {
          const uint32_t off = at(u * RPI + fr, fc);
          const int j = j0 + u * RPI;
          const bool ok = fcv && j < total && j >= 0, cached = j < fx.len;
          cp_async16_fill(kd_ + off, ok ? (cached ? ck : nk) : p.q.data, ok ? 16 : 0);
          cp_async16_fill(vd_ + off, ok ? (cached ? cv : nv) : p.q.data, ok ? 16 : 0);
          ck += ks;
          cv += vs;
          nk += nks;
          nv += nvs;
        }
      }
      if (fx.b >= 0) fx.b += W;
      if (fx.b < 0 || fx.b >= fx.b_end) {
        fi += stride;
        f_new = true;
      }
    }
    cp_async_commit();
    f_slot = f_slot + 1 == NS ? 0 : f_slot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < NS; ++i) fill();

  int slot = 0, seq = 0;
  uint32_t phases = 0;  // bit i: the parity that slot i's barrier completes next
  int c_len = first < items ? __ldg(p.len + item_row(p, first)) : 0;
#pragma unroll 1
  for (uint32_t it = first; it < items; it += stride) {
    MmaItem x = open_item<KB, NQ>(p, it, c_len, wi);
    if (x.len != c_len && lane == 0) atomicOr(p.status, kDevInternal);
    if (it + stride < items) c_len = __ldg(p.len + item_row(p, it + stride));
    const uint32_t qs = base + sm.q + seq * sm.q_one;
    uint32_t qf[S::QREG ? NQ : 1][DP / 16][2];
    bool bad_values = false, dead_any = false;
    unsigned alive = ~0u;  // bit 2 * a + e: query 8 a + 2 t + e sees something
    float m_run[NQ][2], l_run[NQ][2], o[DP / 16][NQ][4];
#pragma unroll
    for (int a = 0; a < NQ; ++a) {
      m_run[a][0] = m_run[a][1] = -INFINITY;
      l_run[a][0] = l_run[a][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) o[j][a][0] = o[j][a][1] = o[j][a][2] = o[j][a][3] = 0.0f;
    }
    bool open = true;
#pragma unroll 1
    do {
      cp_async_wait<NS - 1>();
      // After a wait that ran out nothing is fetched or waited for any more; the loops just end.  A limit
      // of zero is one that has run out at the first wait, whether or not its copies are there already.
      if (((pending >> slot) & 1u) && !timed_out) {
        const bool there = p.spin_limit_ns > 0 && mbar_wait_bounded(base + sm.bars + 8 * slot, (phases >> slot) & 1u, p.spin_limit_ns);
        if (__all_sync(~0u, there)) {
          phases ^= 1u << slot;
          pending ^= 1u << slot;
        } else {
          timed_out = true;
        }
      }
      __syncwarp();  // every lane's copies of this stage are there
      if (open) {
        open = false;
        if constexpr (S::QREG) {
#pragma unroll
          for (int a = 0; a < NQ; ++a)
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int q = a * 8 + g;
                qf[a][kk][e] = (q < x.nq ? lds32(qs + q * sm.q_row + (2 * kk + e) * 16 + t * 4) : 0u) ^ flip;
              }
        }
        if (p.nodes) {
          const int* par = reinterpret_cast<const int*>(mine + sm.par + seq * sm.par_one);
          if (tree_seen_from(tree, [&](int i) { return par[i]; }, p.nodes, lane, 32, [] { __syncwarp(); }))
            atomicOr(p.status, kDevInternal);
          alive = 0;
#pragma unroll
          for (int a = 0; a < 2 * NQ; ++a) {
            const int q = (a >> 1) * 8 + 2 * t + (a & 1);
            if (q < x.nq && tree.mask[p.by_group(x.i0 + q)]) alive |= 1u << a;
            dead_any |= q < x.nq && !((alive >> a) & 1u);
          }
          dead_any = __any_sync(~0u, dead_any);
        }
        seq = seq + 1 == sets ? 0 : seq + 1;
      }
      const uint32_t ks = ring + slot * S::STAGE, vs = ks + S::PANELS * S::PANEL;
      const int n0 = max(x.b, 0) * KB;
      const int total = x.b < 0 ? 0 : x.len + p.nodes;

      // S^T = K Q^T
      float s[KT][NQ][4];
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int a = 0; a < NQ; ++a) s[k][a][0] = s[k][a][1] = s[k][a][2] = s[k][a][3] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        if (DP == 64 || kk < kd) {
          uint32_t qb[NQ][2];
          if constexpr (S::QREG) {
#pragma unroll
            for (int a = 0; a < NQ; ++a) {
              qb[a][0] = qf[a][kk][0];
              qb[a][1] = qf[a][kk][1];
            }
          } else {
#pragma unroll
            for (int a = 0; a < NQ; a += 2) {
              uint32_t f[4];
              const int q = a * 8 + (lane & 7) + (lane >> 4) * 8, c = 2 * kk + ((lane >> 3) & 1);
              ldsm4(f, qs + q * sm.q_row + c * 16);
              qb[a][0] = f[0] ^ flip;
              qb[a][1] = f[1] ^ flip;
              qb[a + 1][0] = f[2] ^ flip;
              qb[a + 1][1] = f[3] ^ flip;
            }
          }
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            uint32_t f[4];
            ldsm4(f, ((ks + k_lane) ^ ((kk & 3) << 5)) + (kk >> 2) * S::PANEL + k * 2048);
#pragma unroll
            for (int a = 0; a < NQ; ++a) mma16816<BF>(s[k][a], f, qb[a][0], qb[a][1]);
          }
        }
      }

      const bool edge = x.b < 0 || n0 + KB > x.len;
      // values that some queries must not meet: infinite and NaN ones of the drafted tokens are
      // taken out and added back at the end to the queries that see them
      if (edge && p.nodes > 1) {
        bool hit = false;
        const int from = max(x.len - n0, 0), upto = min(total - n0, KB);
        for (int e = from * CPR + lane; e < upto * CPR; e += 32) {
          const uint32_t a = vs + at(e / CPR, e % CPR);
          uint4 v = lds128(a);
          if (clear_non_finite<BF>(v)) {
            sts128(a, v);
            hit = true;
          }
        }
        bad_values |= __any_sync(~0u, hit);
        __syncwarp();
      }

      if (edge || dead_any) {
#pragma unroll
        for (int a = 0; a < NQ; ++a)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int q = a * 8 + 2 * t + e, d = x.len - n0;  // the drafted tokens' first place in the block
            uint32_t sees = (alive >> (2 * a + e)) & 1u ? ~0u : 0u;  // bit i: key i of the block
            if (edge && sees) {
              const unsigned long long see = p.nodes && q < x.nq ? tree.mask[p.by_group(x.i0 + q)] : 0ull;
              sees = x.b < 0 ? 0u : d >= 0 ? ((1u << d) - 1u) | (uint32_t)(see << d) : (uint32_t)(see >> -d);
            }
            sees >>= g;
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                if (!((sees >> (k * 16 + hf * 8)) & 1u)) s[k][a][2 * hf + e] = -INFINITY;
          }
      }
      // The maximum is taken over the lanes, and the sums rescaled, only when some lane's own has
      // grown by more than 2^8: until then weights are at most 2^8 times as large (in f16 2^15, kAtLift),
      // which f32 sums and the 16-bit types hold without loss.
      float top[NQ][2];
      bool grown = false;
#pragma unroll
      for (int a = 0; a < NQ; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[a][e] = fmaxf(s[0][a][e], s[0][a][2 + e]);
#pragma unroll
          for (int k = 1; k < KT; ++k) top[a][e] = fmaxf(top[a][e], fmaxf(s[k][a][e], s[k][a][2 + e]));
          grown |= fmaf(top[a][e], c, -kAtLift<BF>) > m_run[a][e] + kMmLazy;
        }
      if (__any_sync(~0u, grown)) {
#pragma unroll
        for (int a = 0; a < NQ; ++a) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float bm = top[a][e];
            bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, 4));
            bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, 8));
            bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, 16));
            const float mn = fmaxf(m_run[a][e], fmaf(bm, c, -kAtLift<BF>));
            f[e] = fast_exp2(m_run[a][e] - (mn == -INFINITY ? 0.0f : mn));
            m_run[a][e] = mn;
            l_run[a][e] *= f[e];
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
      uint32_t pb[KT][NQ][2];
#pragma unroll
      for (int a = 0; a < NQ; ++a) {
        const float sub[2] = {m_run[a][0] == -INFINITY ? 0.0f : -m_run[a][0], m_run[a][1] == -INFINITY ? 0.0f : -m_run[a][1]};
#pragma unroll
        for (int k = 0; k < KT; ++k) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[k][a][e] = fast_exp2(fmaf(s[k][a][e], c, sub[e & 1]));
          l_run[a][0] += s[k][a][0] + s[k][a][2];
          l_run[a][1] += s[k][a][1] + s[k][a][3];
          pb[k][a][0] = transpose8(pack2<BF>(s[k][a][0], s[k][a][1]));
          pb[k][a][1] = transpose8(pack2<BF>(s[k][a][2], s[k][a][3]));
        }
      }

      // O^T += V^T P^T
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) {
        if (DP == 64 || j < kd) {
#pragma unroll
          for (int k = 0; k < KT; ++k) {
            uint32_t f[4];
            ldsm4_trans(f, ((vs + v_lane) ^ ((j & 3) << 5)) + (j >> 2) * S::PANEL + k * 2048);
#pragma unroll
            for (int a = 0; a < NQ; ++a) mma16816<BF>(o[j][a], f, pb[k][a][0], pb[k][a][1]);
          }
        }
      }
      __syncwarp();  // all lanes are done with this stage
      fill();
      slot = slot + 1 == NS ? 0 : slot + 1;
      if (x.b >= 0) x.b += W;
    } while (x.b >= 0 && x.b < x.b_end);

    if (bad_values) {  // rare: the infinite and NaN values of the drafted tokens
      const unsigned char* dv = p.dvalue.data + (long long)x.r * p.dvalue.row + (long long)x.h * p.dvalue.head;
      for (int nd = 0; nd < p.nodes; ++nd)
#pragma unroll
        for (int a = 0; a < 2 * NQ; ++a) {
          const int q = (a >> 1) * 8 + 2 * t + (a & 1);
          if (q >= x.nq || !((tree.mask[p.by_group(x.i0 + q)] >> nd) & 1ull)) continue;
#pragma unroll
          for (int j = 0; j < DP / 16; ++j)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int d = j * 16 + hf * 8 + g;
              const float v = d < p.dim ? load_elem<DT>(dv + nd * p.dvalue.pos + d * 2) : 0.0f;
              if (!isfinite(v)) o[j][a >> 1][2 * hf + (a & 1)] += v;
            }
        }
      __syncwarp();
    }
#pragma unroll
    for (int a = 0; a < NQ; ++a)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l_run[a][e] += __shfl_xor_sync(~0u, l_run[a][e], 4);
        l_run[a][e] += __shfl_xor_sync(~0u, l_run[a][e], 8);
        l_run[a][e] += __shfl_xor_sync(~0u, l_run[a][e], 16);
      }
    if (W == 1) {  // never split
#pragma unroll
      for (int a = 0; a < NQ; ++a) {
        if (a * 8 >= x.nq) break;
        const int q = a * 8 + g;  // the query whose elements this lane stores after the transpose
        unsigned char* out = p.out.data + query_offset(p, p.out, x.r, x.h, x.i0 + min(q, x.nq - 1)) + t * 4;
        const bool z0 = l_run[a][0] == 0.0f, z1 = l_run[a][1] == 0.0f;
        const float i0 = z0 ? 0.0f : 1.0f / l_run[a][0], i1 = z1 ? 0.0f : 1.0f / l_run[a][1];
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
          if (j >= kd) break;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float y0 = z0 ? 0.0f : o[j][a][2 * hf] * i0, y1 = z1 ? 0.0f : o[j][a][2 * hf + 1] * i1;
            const uint32_t y = transpose8(pack2<BF>(y0, y1));
            if (q < x.nq && 2 * j + hf < chunks) *reinterpret_cast<uint32_t*>(out + j * 32 + hf * 16) = y;
          }
        }
      }
    } else {
      // the four warps' results, added in their order
      constexpr int PITCH = DP;
      static_assert(8 * NQ * PITCH * 4 <= NS * S::STAGE, "within the rings: the barriers lie behind them");
      cp_async_wait<0>();
      __syncthreads();
      float* acc = reinterpret_cast<float*>(mm_raw + (rings - raw));
#pragma unroll
      for (int a = 0; a < NQ; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int q = a * 8 + 2 * t + e;
          if (g == 0) {
            wm[warp][q] = m_run[a][e];
            wl[warp][q] = l_run[a][e];
          }
          if (q < x.nq) {
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) {
              acc[(warp * 8 * NQ + q) * PITCH + j * 16 + g] = o[j][a][e];
              acc[(warp * 8 * NQ + q) * PITCH + j * 16 + 8 + g] = o[j][a][2 + e];
            }
          }
        }
      __syncthreads();
      const int half_dim = p.dim / 2;
      const long long prow = (((long long)x.r * p.kv_heads + x.h) * p.m + x.i0) * p.splits + x.split;
      for (int e = threadIdx.x; e < x.nq * half_dim; e += kMmThreads) {
        const int q = e / half_dim, d = (e - q * half_dim) * 2;
        float M = wm[0][q];
#pragma unroll
        for (int w = 1; w < kMmWarps; ++w) M = fmaxf(M, wm[w][q]);
        const float sub = M == -INFINITY ? 0.0f : M;
        float L = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
        for (int w = 0; w < kMmWarps; ++w) {
          const float l = wl[w][q], f = fast_exp2(wm[w][q] - sub);
          L = fmaf(f, l, L);
          const float2 v = *reinterpret_cast<const float2*>(acc + (w * 8 * NQ + q) * PITCH + d);
          o0 = add_part(o0, f, v.x, l);
          o1 = add_part(o1, f, v.y, l);
        }
        if (p.splits == 1) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          *reinterpret_cast<uint32_t*>(p.out.data + query_offset(p, p.out, x.r, x.h, x.i0 + q) + d * 2) =
              pack2<BF>(L == 0.0f ? 0.0f : o0 * inv, L == 0.0f ? 0.0f : o1 * inv);
        } else {
          const long long pr = prow + (long long)q * p.splits;
          *reinterpret_cast<float2*>(p.part_o + pr * p.dim + d) = make_float2(o0, o1);
          if (d == 0) p.part_ml[pr] = make_float2(M, L);
        }
      }
    }
  }
  if (timed_out && lane == 0) atomicOr(p.status, kDevTimeout);
  if (timed_out) {  // every copy lands before the CTA may exit
    for (int i = 0; i < NS; ++i)
      if ((pending >> i) & 1u) mbar_wait_bounded(base + sm.bars + 8 * i, (phases >> i) & 1u, kMmDrainNs);
  }
  cp_async_wait<0>();
}

template <bool BF, int DP, int NQ>
cudaError_t run_mma(const AttendParams& p, int dtype, cudaStream_t stream) {
  using S = MmaShape<DP, NQ>;
  static std::atomic<uint64_t> allowed{0};
  const int most = mma_smem_bytes<DP, NQ>(8 * NQ, kAtMaxNodes, 1);
  const int bytes = mma_smem_bytes<DP, NQ>(p.m, p.nodes, p.warps);
  auto kernel = attend_mma_kernel<BF, DP, NQ>;
  cudaError_t e = allow_shared(kernel, most, allowed);
  if (e != cudaSuccess) return e;
  // without a row of a whole block there is nothing for TMA to read
  CUtensorMap maps[2] = {};
  if (p.max_len >= S::KB && !encode_keys(maps, p, dtype, S::KB)) return cudaErrorInvalidValue;
  long long grid = p.items;
  if (p.warps == 1) {
    static std::atomic<uint64_t> known{0};
    int occ = 0;
    e = resident_ctas(kernel, kMmThreads, bytes, known, &occ);
    if (e != cudaSuccess) return e;
    const long long need = (p.items + kMmWarps - 1) / kMmWarps, fit = (long long)kAtSms * occ;
    grid = need < fit ? need : fit;
  }
  kernel<<<(unsigned)grid, kMmThreads, bytes, stream>>>(maps[0], maps[1], p);
  return cudaGetLastError();
}

template <bool BF, int DP>
cudaError_t run_mma_queries(const AttendParams& p, int dtype, cudaStream_t stream) {
  const int q = attend_mma_queries(p.dim, p.m);
  if (q == 8) return run_mma<BF, DP, 1>(p, dtype, stream);
  if constexpr (DP <= 128) {
    if (q == 32) return run_mma<BF, DP, 4>(p, dtype, stream);
  }
  return run_mma<BF, DP, 2>(p, dtype, stream);
}

template <bool BF>
cudaError_t run_mma_dim(const AttendParams& p, int dtype, cudaStream_t stream) {
  if (p.dim <= 64) return run_mma_queries<BF, 64>(p, dtype, stream);
  if (p.dim <= 128) return run_mma_queries<BF, 128>(p, dtype, stream);
  return run_mma_queries<BF, 256>(p, dtype, stream);
}

}  // namespace

int attend_mma_queries(int dim, int m) { return m <= 8 ? 8 : m <= 16 || dim > 128 ? 16 : 32; }

cudaError_t launch_attend_mma(const AttendParams& p, int dtype, cudaStream_t stream) {
  return dtype == DT_BF16 ? run_mma_dim<true>(p, dtype, stream) : run_mma_dim<false>(p, dtype, stream);
}

}  // namespace lsb
