// New keys and values into the pages of a cache, and positions of it back as dense tensors: copies, or
// with 8-bit pages one quantisation per head vector:
//
//   e4m3: scale = 2^e, e the least with max |x| <= 448 2^e (and e >= -126); code = rn(x / 2^e)
//   i8:   scale = fl(max |x| fl(1 / 127)) (and >= 2^-126); code = the whole number nearest to x / scale
//
// The e4m3 quotient is exact; the i8 one is estimated by a product with 1 / scale, at most one off, and
// put right by the remainder x - code * scale, which f32 holds exactly.
//
// A group of lanes has one head vector of keys and the same of values, 16 elements per lane, so that its
// loads are under way together and the page is looked up once; the largest element is found by exchanges within the group.
// A write's tokens are loaded while their places are looked up, before the count is known: single tokens wait for one
// thing less, but of prompts the tokens past a row's count are read for nothing.
//
// Bound by memory, with reads and writes mixed, and close to it by instructions where codes are made: 16 prompts of 1201 to
// 2048 tokens x 8 heads of 128 bf16 as they are 213 MB, and 28 MB of tokens past the counts, in 40 us, 0.89 of the measured
// copy rate; into e4m3 161 and 28 MB in 33 us, 0.84 (what is needed alone 0.72), 72 % of the issue slots in use; into int8
// 189 MB in 41 us, 0.68 (each code checked by itself 50).
// 16 rows of 1001 to 4000 positions of int8 back to bf16 248 MB in 44.5 us, 0.82 (CTAs of 64 threads; of 128, 46).  1024 single
// tokens x 16 heads of 64 f16 into int8: 4.3 us.
#include <cuda_fp8.h>

#include "ls_paged.cuh"

namespace lsb {
namespace {

constexpr int kMvThreads = 64;  // (128: reads 2 to 3 % slower, for the groups past a row's count)
enum { CT_E4M3 = LS_DTYPE_E4M3, CT_I8 = LS_DTYPE_I8 };

template <int CT>
constexpr int kBytes = CT == DT_F32 ? 4 : CT == DT_F16 || CT == DT_BF16 ? 2 : 1;

template <int DT>
__device__ __forceinline__ float elem_of(const unsigned char* at) { return load_elem<DT>(at); }

__device__ __forceinline__ float scale_of(bool i8, float a) {
  if (i8) return fmaxf(__fmul_rn(a, 1.0f / 127.0f), 0x1p-126f);
  const uint32_t bits = __float_as_uint(a);  // 448 = 1.75 * 2^8
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// x / scale as a whole number, ties to even, by the estimate x * inv.
__device__ __forceinline__ int code_i8(float x, float scale, float inv) {
  float q = rintf(x * inv);
  const float rest = fmaf(-q, scale, x), twice = fabsf(rest) + fabsf(rest);
  if (twice > scale || (twice == scale && ((int)q & 1))) q += copysignf(1.0f, rest);
  return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}
__device__ __forceinline__ uint32_t code2_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

struct Places {
  bool ok;
  long long key, value, kscale, vscale;  // byte offsets of the head vector and its scales
};

// Token i of row r, head h: whether it is to be moved, and where it lies.
__device__ __forceinline__ Places place_of(const PageMoveParams& p, int r, int i, int h, bool lead) {
  Places at{};
  int count = p.count ? __ldg(p.count + r) : p.tokens;
  bool bad = count < 0 || count > p.tokens;
  if (i < count) {
    const long long pos = (long long)(p.start ? __ldg(p.start + r) : 0) + i;
    if (pos < 0 || pos >= p.pages.places) {
      bad = true;
    } else {
      const int s = p.pages.by_page((int)pos), in = (int)pos - s * p.pages.page_size;
      const int page = __ldg(p.pages.table + (long long)r * p.pages.table_row + s);
      if ((unsigned)page < (unsigned)p.pages.num_pages) {
        at.ok = true;
        auto off = [&](const AtView& v) { return (long long)page * v.row + (long long)in * v.pos + (long long)h * v.head; };
        at.key = off(p.pages.key);
        at.value = off(p.pages.value);
        at.kscale = off(p.pages.kscale);
        at.vscale = off(p.pages.vscale);
      } else {
        bad = true;
      }
    }
  }
  if (bad && lead && p.status) atomicOr(p.status, kDevInternal);
  return at;
}

__device__ __forceinline__ long long dense_at(const AtView& v, int r, int i, int h) {
  return (long long)r * v.row + (long long)i * v.pos + (long long)h * v.head;
}

__device__ __forceinline__ uint4 load16(const unsigned char* at) { return __ldg(reinterpret_cast<const uint4*>(at)); }
__device__ __forceinline__ void store16(unsigned char* at, const uint4& x) { *reinterpret_cast<uint4*>(at) = x; }

// A lane's 16 elements of type DT, and back.
template <int DT>
__device__ __forceinline__ void floats_of(const uint4 (&raw)[kBytes<DT>], float (&x)[16]) {
  constexpr int E = Traits<DT>::kVec;
#pragma unroll
  for (int v = 0; v < 16 / E; ++v) {
    float y[E];
    unpack<DT>(raw[v], y);
#pragma unroll
    for (int e = 0; e < E; ++e) x[v * E + e] = y[e];
  }
}
template <int DT>
__device__ __forceinline__ uint32_t pack_two(float a, float b) {
  if constexpr (DT == DT_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <int DT>
__device__ __forceinline__ void store_floats(unsigned char* at, const float (&x)[16]) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      store16(at + 16 * v, make_uint4(__float_as_uint(x[4 * v]), __float_as_uint(x[4 * v + 1]), __float_as_uint(x[4 * v + 2]),
                                      __float_as_uint(x[4 * v + 3])));
  } else {
#pragma unroll
    for (int v = 0; v < 2; ++v)
      store16(at + 16 * v, make_uint4(pack_two<DT>(x[8 * v], x[8 * v + 1]), pack_two<DT>(x[8 * v + 2], x[8 * v + 3]),
                                      pack_two<DT>(x[8 * v + 4], x[8 * v + 5]), pack_two<DT>(x[8 * v + 6], x[8 * v + 7])));
  }
}

// A group of G lanes to a head vector, 16 elements to a lane.
template <int DT, int CT, int G, bool READ>
__global__ void __launch_bounds__(kMvThreads) page_move_kernel(const __grid_constant__ PageMoveParams p) {
  constexpr int B = kBytes<DT>, BC = kBytes<CT>;
  const int lane = threadIdx.x % G;
  const long long n = ((long long)blockIdx.x * kMvThreads + threadIdx.x) / G;
  const bool any = n < p.vectors;  // (whole warps go on: the exchanges are theirs)
  const int t = any ? p.by_head((int)n) : 0, h = any ? (int)n - t * p.heads : 0, r = p.by_token(t), i = t - r * p.tokens;
  // a write's tokens are under way while their places are looked up (those past the count come for nothing)
  constexpr int RAW = READ ? 1 : B;
  uint4 rk[RAW], rv[RAW];
  if constexpr (!READ) {
    if (any && lane * 16 < p.dim) {
      const unsigned char* from_k = p.key.data + dense_at(p.key, r, i, h) + lane * 16 * B;
      const unsigned char* from_v = p.value.data + dense_at(p.value, r, i, h) + lane * 16 * B;
#pragma unroll
      for (int v = 0; v < B; ++v) {
        rk[v] = load16(from_k + 16 * v);
        rv[v] = load16(from_v + 16 * v);
      }
    }
  }
  Places at{};
  if (any) at = place_of(p, r, i, h, lane == 0 && h == 0);
  const bool mine = at.ok && lane * 16 < p.dim;
  unsigned char* dk = p.key.data + dense_at(p.key, r, i, h) + lane * 16 * B;
  unsigned char* dv = p.value.data + dense_at(p.value, r, i, h) + lane * 16 * B;
  unsigned char* pk = p.pages.key.data + at.key + lane * 16 * BC;
  unsigned char* pv = p.pages.value.data + at.value + lane * 16 * BC;
  if constexpr (CT == DT) {
    if (!mine) return;
    if constexpr (READ) {
      uint4 a[B], b[B];
#pragma unroll
      for (int v = 0; v < B; ++v) {
        a[v] = load16(pk + 16 * v);
        b[v] = load16(pv + 16 * v);
      }
#pragma unroll
      for (int v = 0; v < B; ++v) {
        store16(dk + 16 * v, a[v]);
        store16(dv + 16 * v, b[v]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < B; ++v) {
        store16(pk + 16 * v, rk[v]);
        store16(pv + 16 * v, rv[v]);
      }
    }
  } else if constexpr (READ) {
    if (!mine) return;
    const uint4 ck = load16(pk), cv = load16(pv);
    const float sk = __ldg(reinterpret_cast<const float*>(p.pages.kscale.data + at.kscale));
    const float sv = __ldg(reinterpret_cast<const float*>(p.pages.vscale.data + at.vscale));
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint4& d = kv ? cv : ck;
      const float s = kv ? sv : sk;
      const uint32_t w[4] = {d.x, d.y, d.z, d.w};
      float x[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (CT == CT_E4M3) {
          const float2 a = e4m3x2_float(w[j] & 0xffffu), b = e4m3x2_float(w[j] >> 16);
          x[4 * j] = a.x;
          x[4 * j + 1] = a.y;
          x[4 * j + 2] = b.x;
          x[4 * j + 3] = b.y;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * j + e] = (float)(signed char)(w[j] >> 8 * e);
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= s;
      store_floats<DT>(kv ? dv : dk, x);
    }
  } else {
    float xk[16] = {}, xv[16] = {};
    if (any && lane * 16 < p.dim) {
      floats_of<DT>(rk, xk);
      floats_of<DT>(rv, xv);
    }
    float ak = 0.0f, av = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      ak = fmaxf(ak, fabsf(xk[e]));
      av = fmaxf(av, fabsf(xv[e]));
    }
#pragma unroll
    for (int o = 1; o < G; o <<= 1) {
      ak = fmaxf(ak, __shfl_xor_sync(~0u, ak, o));
      av = fmaxf(av, __shfl_xor_sync(~0u, av, o));
    }
    if (!mine) return;
    const float sk = scale_of(CT == CT_I8, ak), sv = scale_of(CT == CT_I8, av);
    if (lane == 0) {
      *reinterpret_cast<float*>(p.pages.kscale.data + at.kscale) = sk;
      *reinterpret_cast<float*>(p.pages.vscale.data + at.vscale) = sv;
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float s = kv ? sv : sk, inv = 1.0f / s;  // exact for a power of two
      uint32_t w[4];
      if constexpr (CT == CT_I8) {
        // the estimates, as the low bytes of a sum with 1.5 * 2^23; one by one where a remainder says that one of them
        // is not the nearest, or a tie
        constexpr float kMagic = 12582912.0f;
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = kv ? xv[4 * j + e] : xk[4 * j + e], f = fmaf(y, inv, kMagic);
            most = fmaxf(most, fabsf(fmaf(-__fsub_rn(f, kMagic), s, y)));
            b[e] = __float_as_uint(f);
          }
          w[j] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        }
        if (most + most < s) {
          store16(kv ? pv : pk, make_uint4(w[0], w[1], w[2], w[3]));
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = kv ? xv[4 * j + e] : xk[4 * j + e];
        if constexpr (CT == CT_E4M3) {
          w[j] = code2_e4m3(y[0] * inv, y[1] * inv) | code2_e4m3(y[2] * inv, y[3] * inv) << 16;
        } else {
          w[j] = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[j] |= ((uint32_t)code_i8(y[e], s, inv) & 0xffu) << 8 * e;
        }
      }
      store16(kv ? pv : pk, make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

// Any layout: a warp to a head vector (of keys, then of values), element by element.
template <int DT, int CT, bool READ>
__global__ void __launch_bounds__(kMvThreads) page_move_any_kernel(const __grid_constant__ PageMoveParams p) {
  constexpr int B = kBytes<DT>, BC = kBytes<CT>;
  const int lane = threadIdx.x & 31;
  const long long n = ((long long)blockIdx.x * kMvThreads + threadIdx.x) / 32;
  if (n >= p.vectors) return;
  const int t = p.by_head((int)n), h = (int)n - t * p.heads, r = p.by_token(t), i = t - r * p.tokens;
  const Places at = place_of(p, r, i, h, lane == 0 && h == 0);
  if (!at.ok) return;
  for (int kv = 0; kv < 2; ++kv) {
    unsigned char* dense = kv ? p.value.data + dense_at(p.value, r, i, h) : p.key.data + dense_at(p.key, r, i, h);
    unsigned char* page = kv ? p.pages.value.data + at.value : p.pages.key.data + at.key;
    float* scale = reinterpret_cast<float*>(kv ? p.pages.vscale.data + at.vscale : p.pages.kscale.data + at.kscale);
    if constexpr (CT == DT) {
      for (int d = lane; d < p.dim; d += 32) {
        unsigned char *from = READ ? page : dense, *to = READ ? dense : page;
        if constexpr (B == 4)
          reinterpret_cast<uint32_t*>(to)[d] = reinterpret_cast<const uint32_t*>(from)[d];
        else
          reinterpret_cast<uint16_t*>(to)[d] = reinterpret_cast<const uint16_t*>(from)[d];
      }
    } else if constexpr (READ) {
      const float s = *scale;
      for (int d = lane; d < p.dim; d += 32) {
        const float c = CT == CT_E4M3 ? e4m3x2_float(page[d]).x : (float)reinterpret_cast<const signed char*>(page)[d];
        pg_store<DT>(dense + d * B, c * s);
      }
    } else {
      float a = 0.0f;
      for (int d = lane; d < p.dim; d += 32) a = fmaxf(a, fabsf(elem_of<DT>(dense + d * B)));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
      const float s = scale_of(CT == CT_I8, a), inv = 1.0f / s;
      if (lane == 0) *scale = s;
      for (int d = lane; d < p.dim; d += 32) {
        const float y = elem_of<DT>(dense + d * B);
        page[d * BC] = CT == CT_E4M3 ? (unsigned char)code2_e4m3(y * inv, 0.0f) : (unsigned char)code_i8(y, s, inv);
      }
    }
  }
}

template <int DT, int CT, bool READ>
cudaError_t run_move(const PageMoveParams& p, bool vec, cudaStream_t stream) {
  const int lanes = !vec ? 32 : p.dim <= 64 ? 4 : p.dim <= 128 ? 8 : 16;
  const unsigned grid = (unsigned)((p.vectors * lanes + kMvThreads - 1) / kMvThreads);
  if (!vec)
    page_move_any_kernel<DT, CT, READ><<<grid, kMvThreads, 0, stream>>>(p);
  else if (lanes == 4)
    page_move_kernel<DT, CT, 4, READ><<<grid, kMvThreads, 0, stream>>>(p);
  else if (lanes == 8)
    page_move_kernel<DT, CT, 8, READ><<<grid, kMvThreads, 0, stream>>>(p);
  else
    page_move_kernel<DT, CT, 16, READ><<<grid, kMvThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int DT, bool READ>
cudaError_t run_move_cache(const PageMoveParams& p, int cache, bool vec, cudaStream_t stream) {
  if (cache == CT_E4M3) return run_move<DT, CT_E4M3, READ>(p, vec, stream);
  if (cache == CT_I8) return run_move<DT, CT_I8, READ>(p, vec, stream);
  return run_move<DT, DT, READ>(p, vec, stream);
}

template <bool READ>
cudaError_t run_move_type(const PageMoveParams& p, int dtype, int cache, bool vec, cudaStream_t stream) {
  if (dtype == DT_F32) return run_move_cache<DT_F32, READ>(p, cache, vec, stream);
  if (dtype == DT_F16) return run_move_cache<DT_F16, READ>(p, cache, vec, stream);
  return run_move_cache<DT_BF16, READ>(p, cache, vec, stream);
}

}  // namespace

cudaError_t launch_page_write(const PageMoveParams& p, int dtype, int cache, bool vec, cudaStream_t stream) {
  return run_move_type<false>(p, dtype, cache, vec, stream);
}
cudaError_t launch_page_read(const PageMoveParams& p, int dtype, int cache, bool vec, cudaStream_t stream) {
  return run_move_type<true>(p, dtype, cache, vec, stream);
}

}  // namespace lsb
