// Attention of few queries over a row's keys (f16 / bf16): the decode step, small trees, beams
// of a sentence.  With M queries per key the products take M flops per byte of keys and values
// read, far below what the tensor cores need to be the limit, so this kernel is built around
// the stream of keys and values from memory and uses the warp-level matrix instructions
// (m16n8k16, f32 accumulators), whose 16-row operand fits 1 to 16 (or two of them 32) queries
// and whose accumulators stay in registers.
//
//   S = Q K^T,  P = exp2(c S - max),  O = O * correction + P V,  out = O / sum P
//
// in one pass with the running maximum and sum of the softmax (Milakov and Gimelshein, 2018).
// P is rounded to the tensors' type for the second product (its error averages out over the
// keys like the values' own rounding); the sums use the unrounded f32 weights.
//
// A warp streams blocks of KB keys and their values through a ring of its own in shared memory
// by 16-byte asynchronous copies (zero-filled past the row's keys, so nothing there reaches a
// product), rows XOR-swizzled for conflict-free ldmatrix; no CTA barrier in the stream.  Two
// ways to share the work out, by AttendParams::warps:
//   1: a warp takes whole problems, one after the other, and its ring runs ahead into the next
//      problem (its queries and parents come through the ring as well), so that short rows
//      stream without a gap;
//   4: the CTA's four warps take the blocks of one (part of a) problem in turn and merge their
//      results in shared memory.
#include "ls_device.cuh"
#include "ls_dtype.cuh"
#include "ls_tree.cuh"

namespace lsb {
namespace {

constexpr int kMmWarps = 4;
constexpr int kMmThreads = kMmWarps * 32;

__device__ __forceinline__ void cp_async16_fill(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // bytes read; the rest of the 16 are zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
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

// The two 16-bit values of w, zero where they are infinite or NaN; *hit is set for those.
template <bool BF>
__device__ __forceinline__ uint32_t finite2(uint32_t w, bool* hit) {
  constexpr uint32_t E = BF ? 0x7f80u : 0x7c00u;
  if ((w & E) == E) {
    w &= 0xffff0000u;
    *hit = true;
  }
  if ((w & (E << 16)) == E << 16) {
    w &= 0x0000ffffu;
    *hit = true;
  }
  return w;
}

template <int DP, int MT>
struct MmaShape {
  static constexpr int KB = DP == 64 ? 32 : 16;   // keys per block
  static constexpr int NS = DP == 256 ? 2 : 3;    // blocks in the ring
  static constexpr int ROW = DP * 2;              // bytes of a staged vector
  static constexpr int STAGE = 2 * KB * ROW;
  static constexpr bool QREG = MT == 1 && DP <= 128;  // the queries' fragments stay in registers
};

// Bytes of one warp's shared memory, and where its parts begin.
struct MmaSmem {
  int q, q_one, par, tree, total;
};
template <int DP, int MT>
__host__ __device__ inline MmaSmem mma_smem(int m, int nodes) {
  using S = MmaShape<DP, MT>;
  MmaSmem s;
  s.q = S::NS * S::STAGE;
  s.q_one = (S::QREG && m < 16 ? m : 16 * MT) * S::ROW;
  s.par = s.q + S::NS * s.q_one;
  const int np = (nodes + 3) / 4 * 16;
  s.tree = s.par + S::NS * np;
  s.total = (s.tree + (nodes ? (int)sizeof(TreeSeen) : 0) + 127) / 128 * 128;
  return s;
}

// One item: the problem, the first of its queries, and the blocks [b, b_end) (step) of this warp.
struct MmaItem {
  int r, h, i0, nq, split, len, nb, b, b_end;
};

template <int DP, int MT>
__device__ __forceinline__ int item_row(const AttendParams& p, long long it) {
  return (int)(it / ((long long)p.splits * p.m_tiles * p.kv_heads));
}

template <int DP, int MT>
__device__ __forceinline__ MmaItem open_item(const AttendParams& p, long long it, int len, int w) {
  constexpr int KB = MmaShape<DP, MT>::KB;
  MmaItem x;
  x.split = (int)(it % p.splits);
  it /= p.splits;
  x.i0 = (int)(it % p.m_tiles) * 16 * MT;
  it /= p.m_tiles;
  x.h = (int)(it % p.kv_heads);
  x.r = (int)(it / p.kv_heads);
  x.nq = min(16 * MT, p.m - x.i0);
  x.len = min(max(len, 0), p.max_len);
  x.nb = (x.len + KB - 1) / KB;
  const int nbt = x.nb + (p.nodes + KB - 1) / KB;
  const int per = (nbt + p.splits - 1) / p.splits;
  const int lo = min(x.split * per, nbt);
  x.b = lo + w;
  x.b_end = min(lo + per, nbt);
  // a warp without a block takes an empty one, so that every item has a stage in the ring
  if (x.b >= x.b_end) x.b = x.b_end = -1;
  return x;
}

template <bool BF, int DP, int MT>
__global__ void __launch_bounds__(kMmThreads) attend_mma_kernel(const AttendParams p) {
  using S = MmaShape<DP, MT>;
  constexpr int KB = S::KB, NS = S::NS, ROW = S::ROW, NT = KB / 8, DT = BF ? DT_BF16 : DT_F16;
  extern __shared__ unsigned char mm_raw[];
  __shared__ float wm[kMmWarps][16 * MT], wl[kMmWarps][16 * MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const MmaSmem sm = mma_smem<DP, MT>(p.m, p.nodes);
  unsigned char* mine = mm_raw + warp * sm.total;
  const uint32_t base = smem_addr(mine);
  TreeSeen& tree = *reinterpret_cast<TreeSeen*>(mine + sm.tree);
  const int np = (p.nodes + 3) / 4 * 16;
  const int W = p.warps, wi = W == 1 ? 0 : warp;
  const int chunks = p.dim / 8;         // 16-byte vectors of a key
  const int kd = (p.dim + 15) / 16;     // k steps of the first product
  const long long stride = W == 1 ? (long long)gridDim.x * kMmWarps : gridDim.x;
  const long long first = W == 1 ? (long long)blockIdx.x * kMmWarps + warp : blockIdx.x;

  // ---- the ring's filling side: item `fi` (its length loaded one item ahead), block `fx.b`
  long long fi = first;
  int f_seq = 0, f_slot = 0;
  bool f_new = true;
  MmaItem fx{};
  int f_len = fi < p.items ? __ldg(p.len + item_row<DP, MT>(p, fi)) : 0;
  auto fill = [&]() {
    if (fi < p.items) {
      if (f_new) {
        fx = open_item<DP, MT>(p, fi, f_len, wi);
        const long long nx = fi + stride;
        if (nx < p.items) f_len = __ldg(p.len + item_row<DP, MT>(p, nx));
        const uint32_t qd = base + sm.q + f_seq * sm.q_one;
        for (int e = lane; e < fx.nq * (DP / 8); e += 32) {
          const int i = e / (DP / 8), c = e % (DP / 8);
          const unsigned char* src = p.q.data + query_offset(p, p.q, fx.r, fx.h, fx.i0 + i);
          cp_async16_fill(qd + i * ROW + ((c ^ (i & 7)) << 4), src + (c < chunks ? c * 16 : 0), c < chunks);
        }
        for (int i = lane; i < p.nodes; i += 32)
          cp_async4(base + sm.par + f_seq * np + i * 4, p.parent + (long long)fx.r * p.nodes + i);
        f_seq = f_seq + 1 == NS ? 0 : f_seq + 1;
        f_new = false;
      }
      const bool draft = fx.b >= fx.nb;
      const int n0 = fx.b < 0 ? 0 : (draft ? fx.b - fx.nb : fx.b) * KB;
      const int n = fx.b < 0 ? 0 : (draft ? p.nodes : fx.len) - n0;  // keys of the block, if below KB
      const AtView& kv = draft ? p.dkey : p.key;
      const AtView& vv = draft ? p.dvalue : p.value;
      const unsigned char* ks = kv.data + (long long)fx.r * kv.row + (long long)fx.h * kv.head + (long long)n0 * kv.pos;
      const unsigned char* vs = vv.data + (long long)fx.r * vv.row + (long long)fx.h * vv.head + (long long)n0 * vv.pos;
      const uint32_t kd_ = base + f_slot * S::STAGE, vd_ = kd_ + KB * ROW;
      constexpr int CPR = DP / 8;
#pragma unroll
      for (int u = 0; u < KB * CPR / 32; ++u) {
        const int e = u * 32 + lane, row = e / CPR, c = e % CPR;
        const bool ok = row < n && c < chunks;
        const uint32_t off = row * ROW + ((c ^ (row & 7)) << 4);
        cp_async16_fill(kd_ + off, ok ? ks + row * kv.pos + c * 16 : p.q.data, ok);
        cp_async16_fill(vd_ + off, ok ? vs + row * vv.pos + c * 16 : p.q.data, ok);
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
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) fill();

  int slot = 0, seq = 0;
  int c_len = first < p.items ? __ldg(p.len + item_row<DP, MT>(p, first)) : 0;
  for (long long it = first; it < p.items; it += stride) {
    MmaItem x = open_item<DP, MT>(p, it, c_len, wi);
    if (x.len != c_len && lane == 0) atomicOr(p.status, kDevInternal);
    if (it + stride < p.items) c_len = __ldg(p.len + item_row<DP, MT>(p, it + stride));
    const uint32_t qs = base + sm.q + seq * sm.q_one;
    uint32_t qf[S::QREG ? DP / 16 : 1][4];
    bool bad_values = false, dead_any = false;
    unsigned alive = ~0u;  // bit 2 * mt + half: the query sees something
    float m_run[MT][2], l_run[MT][2], o[MT][DP / 8][4];
#pragma unroll
    for (int a = 0; a < MT; ++a) {
      m_run[a][0] = m_run[a][1] = -INFINITY;
      l_run[a][0] = l_run[a][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < DP / 8; ++j) o[a][j][0] = o[a][j][1] = o[a][j][2] = o[a][j][3] = 0.0f;
    }
    bool open = true;
    do {
      cp_async_wait<NS - 2>();
      __syncwarp();  // every lane's copies of this stage are there, and all are done with the last one
      if (open) {
        open = false;
        if constexpr (S::QREG) {
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = g + (e & 1) * 8, c = 2 * kk + (e >> 1);
              qf[kk][e] = row < x.nq ? lds32(qs + row * ROW + ((c ^ (row & 7)) << 4) + t * 4) : 0u;
            }
          }
        }
        if (p.nodes) {
          const int* par = reinterpret_cast<const int*>(mine + sm.par + seq * np);
          if (tree_seen_from(tree, [&](int i) { return par[i]; }, p.nodes, lane, 32, [] { __syncwarp(); }))
            atomicOr(p.status, kDevInternal);
          alive = 0;
#pragma unroll
          for (int a = 0; a < 2 * MT; ++a) {
            const int row = (a >> 1) * 16 + (a & 1) * 8 + g;
            if (row < x.nq && tree.mask[(x.i0 + row) / p.group]) alive |= 1u << a;
            dead_any |= row < x.nq && !((alive >> a) & 1u);
          }
          dead_any = __any_sync(~0u, dead_any);
        }
        seq = seq + 1 == NS ? 0 : seq + 1;
      }
      fill();
      const uint32_t ks = base + slot * S::STAGE, vs = ks + KB * ROW;
      const bool draft = x.b >= x.nb;
      const int n0 = x.b < 0 ? 0 : (draft ? x.b - x.nb : x.b) * KB;
      const int n = x.b < 0 ? 0 : (draft ? p.nodes : x.len) - n0;

      // S = Q K^T
      float s[MT][NT][4];
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int j = 0; j < NT; ++j) s[a][j][0] = s[a][j][1] = s[a][j][2] = s[a][j][3] = 0.0f;
      const int lr = (lane & 7) + ((lane >> 4) << 3), lc = (lane >> 3) & 1;  // K: key within 16, 16-byte half
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        if (kk < kd) {
          uint32_t qa[MT][4];
          if constexpr (S::QREG) {
#pragma unroll
            for (int e = 0; e < 4; ++e) qa[0][e] = qf[kk][e];
          } else {
#pragma unroll
            for (int a = 0; a < MT; ++a) {
              const int row = a * 16 + (lane & 15), c = 2 * kk + (lane >> 4);
              ldsm4(qa[a], qs + row * ROW + ((c ^ (row & 7)) << 4));
            }
          }
#pragma unroll
          for (int j = 0; j < NT; j += 2) {
            uint32_t b[4];
            const int row = j * 8 + lr, c = 2 * kk + lc;
            ldsm4(b, ks + row * ROW + ((c ^ (row & 7)) << 4));
#pragma unroll
            for (int a = 0; a < MT; ++a) {
              mma16816<BF>(s[a][j], qa[a], b[0], b[1]);
              mma16816<BF>(s[a][j + 1], qa[a], b[2], b[3]);
            }
          }
        }
      }

      // values that some queries must not meet: infinite and NaN ones of the drafted tokens are
      // taken out and added back at the end to the queries that see them
      if (draft && p.nodes > 1) {
        bool hit = false;
        for (int e = lane; e < min(n, KB) * (DP / 8); e += 32) {
          const uint32_t at = vs + e * 16;
          uint4 v = lds128(at);
          bool h = false;
          v.x = finite2<BF>(v.x, &h);
          v.y = finite2<BF>(v.y, &h);
          v.z = finite2<BF>(v.z, &h);
          v.w = finite2<BF>(v.w, &h);
          if (h) sts128(at, v);
          hit |= h;
        }
        bad_values |= __any_sync(~0u, hit);
        __syncwarp();
      }

      const bool edge = draft || n < KB || dead_any;
#pragma unroll
      for (int a = 0; a < MT; ++a) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[a][j][e] *= p.scale_log2;
        if (edge) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int row = a * 16 + half * 8 + g;
            unsigned see = ((alive >> (2 * a + half)) & 1u) ? ~0u : 0u;
            if (draft && see && row < x.nq) see = (unsigned)(tree.mask[(x.i0 + row) / p.group] >> n0);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = j * 8 + 2 * t + e;
                if (key >= n || !((see >> key) & 1u)) s[a][j][2 * half + e] = -INFINITY;
              }
          }
        }
        float bm[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          bm[0] = fmaxf(bm[0], fmaxf(s[a][j][0], s[a][j][1]));
          bm[1] = fmaxf(bm[1], fmaxf(s[a][j][2], s[a][j][3]));
        }
        bool moved = false;
        float fct[2], sub[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          bm[half] = fmaxf(bm[half], __shfl_xor_sync(~0u, bm[half], 1));
          bm[half] = fmaxf(bm[half], __shfl_xor_sync(~0u, bm[half], 2));
          const float mn = fmaxf(m_run[a][half], bm[half]);
          moved |= mn > m_run[a][half];
          sub[half] = mn == -INFINITY ? 0.0f : mn;
          fct[half] = fast_exp2(m_run[a][half] - sub[half]);
          m_run[a][half] = mn;
        }
        if (__any_sync(~0u, moved)) {
#pragma unroll
          for (int half = 0; half < 2; ++half) l_run[a][half] *= fct[half];
#pragma unroll
          for (int j = 0; j < DP / 8; ++j) {
            o[a][j][0] *= fct[0];
            o[a][j][1] *= fct[0];
            o[a][j][2] *= fct[1];
            o[a][j][3] *= fct[1];
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[a][j][e] = fast_exp2(s[a][j][e] - sub[e >> 1]);
          l_run[a][0] += s[a][j][0] + s[a][j][1];
          l_run[a][1] += s[a][j][2] + s[a][j][3];
        }
      }

      // O += P V
#pragma unroll
      for (int k2 = 0; k2 < KB / 16; ++k2) {
        uint32_t pa[MT][4];
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          pa[a][0] = pack2<BF>(s[a][2 * k2][0], s[a][2 * k2][1]);
          pa[a][1] = pack2<BF>(s[a][2 * k2][2], s[a][2 * k2][3]);
          pa[a][2] = pack2<BF>(s[a][2 * k2 + 1][0], s[a][2 * k2 + 1][1]);
          pa[a][3] = pack2<BF>(s[a][2 * k2 + 1][2], s[a][2 * k2 + 1][3]);
        }
        const int row = k2 * 16 + (lane & 15);
#pragma unroll
        for (int j = 0; j < DP / 8; j += 2) {
          if (j < 2 * kd) {
            uint32_t b[4];
            const int c = j + (lane >> 4);
            ldsm4_trans(b, vs + row * ROW + ((c ^ (row & 7)) << 4));
#pragma unroll
            for (int a = 0; a < MT; ++a) {
              mma16816<BF>(o[a][j], pa[a], b[0], b[1]);
              mma16816<BF>(o[a][j + 1], pa[a], b[2], b[3]);
            }
          }
        }
      }
      slot = slot + 1 == NS ? 0 : slot + 1;
      if (x.b >= 0) x.b += W;
    } while (x.b >= 0 && x.b < x.b_end);

    if (bad_values) {  // rare: the infinite and NaN values of the drafted tokens
      const AtView& vv = p.dvalue;
      const unsigned char* dv = vv.data + (long long)x.r * vv.row + (long long)x.h * vv.head;
#pragma unroll
      for (int a = 0; a < 2 * MT; ++a) {
        const int row = (a >> 1) * 16 + (a & 1) * 8 + g;
        const unsigned long long see = row < x.nq ? tree.mask[(x.i0 + row) / p.group] : 0ull;
        for (int nd = 0; nd < p.nodes; ++nd) {
          if (!((see >> nd) & 1ull)) continue;
#pragma unroll
          for (int j = 0; j < DP / 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = j * 8 + 2 * t + e;
              const float v = d < p.dim ? load_elem<DT>(dv + nd * vv.pos + d * 2) : 0.0f;
              if (!isfinite(v)) o[a >> 1][j][2 * (a & 1) + e] += v;
            }
        }
      }
    }
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        l_run[a][half] += __shfl_xor_sync(~0u, l_run[a][half], 1);
        l_run[a][half] += __shfl_xor_sync(~0u, l_run[a][half], 2);
      }
    const long long prow = (((long long)x.r * p.kv_heads + x.h) * p.m + x.i0) * p.splits + x.split;
    if (W == 1) {  // never split
#pragma unroll
      for (int a = 0; a < 2 * MT; ++a) {
        const int row = (a >> 1) * 16 + (a & 1) * 8 + g;
        if (row < x.nq) {
          const float l = l_run[a >> 1][a & 1];
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          unsigned char* out = p.out.data + query_offset(p, p.out, x.r, x.h, x.i0 + row) + t * 4;
#pragma unroll
          for (int j = 0; j < DP / 8; ++j)
            if (j < chunks) {
              const float o0 = l == 0.0f ? 0.0f : o[a >> 1][j][2 * (a & 1)] * inv;
              const float o1 = l == 0.0f ? 0.0f : o[a >> 1][j][2 * (a & 1) + 1] * inv;
              *reinterpret_cast<uint32_t*>(out + j * 16) = pack2<BF>(o0, o1);
            }
        }
      }
    } else {
      // the four warps' results, added in their order
      constexpr int PITCH = DP + 8;
      cp_async_wait<0>();
      __syncthreads();
      float* acc = reinterpret_cast<float*>(mm_raw);
#pragma unroll
      for (int a = 0; a < 2 * MT; ++a) {
        const int row = (a >> 1) * 16 + (a & 1) * 8 + g;
        if (t == 0) {
          wm[warp][row] = m_run[a >> 1][a & 1];
          wl[warp][row] = l_run[a >> 1][a & 1];
        }
        if (row < x.nq) {
#pragma unroll
          for (int j = 0; j < DP / 8; ++j)
            *reinterpret_cast<float2*>(acc + (warp * 16 * MT + row) * PITCH + j * 8 + 2 * t) =
                make_float2(o[a >> 1][j][2 * (a & 1)], o[a >> 1][j][2 * (a & 1) + 1]);
        }
      }
      __syncthreads();
      const int half_dim = p.dim / 2;
      for (int e = threadIdx.x; e < x.nq * half_dim; e += kMmThreads) {
        const int row = e / half_dim, d = (e - row * half_dim) * 2;
        float M = wm[0][row];
#pragma unroll
        for (int w = 1; w < kMmWarps; ++w) M = fmaxf(M, wm[w][row]);
        const float sub = M == -INFINITY ? 0.0f : M;
        float L = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
        for (int w = 0; w < kMmWarps; ++w) {
          const float l = wl[w][row], f = fast_exp2(wm[w][row] - sub);
          L = fmaf(f, l, L);
          const float2 v = *reinterpret_cast<const float2*>(acc + (w * 16 * MT + row) * PITCH + d);
          o0 = add_part(o0, f, v.x, l);
          o1 = add_part(o1, f, v.y, l);
        }
        if (p.splits == 1) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          *reinterpret_cast<uint32_t*>(p.out.data + query_offset(p, p.out, x.r, x.h, x.i0 + row) + d * 2) =
              pack2<BF>(L == 0.0f ? 0.0f : o0 * inv, L == 0.0f ? 0.0f : o1 * inv);
        } else {
          const long long pr = prow + (long long)row * p.splits;
          *reinterpret_cast<float2*>(p.part_o + pr * p.dim + d) = make_float2(o0, o1);
          if (d == 0) p.part_ml[pr] = make_float2(M, L);
        }
      }
    }
  }
  cp_async_wait<0>();
}

template <bool BF, int DP, int MT>
cudaError_t run_mma(const AttendParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  const int most = kMmWarps * mma_smem<DP, MT>(16 * MT, kAtMaxNodes).total;
  const int bytes = kMmWarps * mma_smem<DP, MT>(p.m, p.nodes).total;
  auto kernel = attend_mma_kernel<BF, DP, MT>;
  cudaError_t e = allow_shared(kernel, most, allowed);
  if (e != cudaSuccess) return e;
  long long grid = p.items;
  if (p.warps == 1) {
    int occ = 1;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, kMmThreads, bytes);
    if (e != cudaSuccess) return e;
    const long long need = (p.items + kMmWarps - 1) / kMmWarps, fit = (long long)kAtSms * (occ > 0 ? occ : 1);
    grid = need < fit ? need : fit;
  }
  kernel<<<(unsigned)grid, kMmThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

template <bool BF>
cudaError_t run_mma_dim(const AttendParams& p, cudaStream_t stream) {
  const bool two = attend_mma_queries(p.dim, p.m) == 32;
  if (p.dim <= 64) return two ? run_mma<BF, 64, 2>(p, stream) : run_mma<BF, 64, 1>(p, stream);
  if (p.dim <= 128) return two ? run_mma<BF, 128, 2>(p, stream) : run_mma<BF, 128, 1>(p, stream);
  return run_mma<BF, 256, 1>(p, stream);
}

}  // namespace

int attend_mma_queries(int dim, int m) { return m > 16 && dim <= 128 ? 32 : 16; }

cudaError_t launch_attend_mma(const AttendParams& p, int dtype, cudaStream_t stream) {
  return dtype == DT_BF16 ? run_mma_dim<true>(p, stream) : run_mma_dim<false>(p, stream);
}

}  // namespace lsb
