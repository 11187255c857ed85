// C-ABI entry points of the decoder's attention and the draft tree's commit (declared in
// include/ls_beam.h): argument checks on the host, launch plans, and the enqueue of the
// kernels on the caller's stream.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "ls_attend.h"
#include "ls_beam.h"
#include "ls_internal.h"

using namespace lsb;

namespace {

constexpr size_t kAtHeader = 256;  // status word

int es_of(ls_dtype d) { return d == LS_DTYPE_F32 ? 4 : 2; }
bool known(ls_dtype d) { return d == LS_DTYPE_F32 || d == LS_DTYPE_F16 || d == LS_DTYPE_BF16; }
bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// A view's pointer, and strides whose largest byte offset 64 bits hold; `written`: dimensions of more
// than one element need a stride.
bool view_ok(const ls_view* v, int es, bool written, int layers, int rows, int pos, int heads) {
  if (!v || !v->data || misaligned(v->data, (size_t)es)) return false;
  const struct {
    int64_t stride;
    int extent;
  } dims[] = {{v->layer, layers}, {v->row, rows}, {v->pos, pos}, {v->head, heads}};
  for (const auto& d : dims) {
    if (d.stride < 0 || (written && d.extent > 1 && d.stride == 0)) return false;
    if (d.stride > (INT64_MAX >> 4) / es / (d.extent > 1 ? d.extent : 1)) return false;
  }
  return true;
}

AtView view_of(const ls_view* v, int es) {
  return AtView{static_cast<unsigned char*>(v->data), v->row * es, v->pos * es, v->head * es};
}

bool shape_ok(int rows, int k, int q_len, int heads, int kv_heads, int max_len, int dim) {
  return rows >= 0 && k >= 1 && q_len >= 0 && heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0 && max_len >= 0 &&
         dim >= 1 && dim <= kAtMaxDim;
}

// Queries that read the same keys; INT64_MAX where the count does not fit 31 bits.
long long queries_per_key(int k, int q_len, int group) {
  const long long tokens = (long long)k * q_len;
  return tokens > INT_MAX ? INT64_MAX : tokens * group;
}

size_t workspace_size(int rows, int k, int q_len, int heads, int kv_heads, int max_len, int dim) {
  if (!shape_ok(rows, k, q_len, heads, kv_heads, max_len, dim)) return 0;
  const long long m = queries_per_key(k, q_len, heads / kv_heads);
  if (m > INT_MAX) return 0;
  return kAtHeader + (size_t)attend_part_rows((int)m) * (size_t)(dim + 2) * 4;
}

// `need`: workspace_size's answer, 0 where the call has no size at all.
bool workspace_ok(const void* workspace, size_t bytes, size_t need) {
  return workspace && !misaligned(workspace, 256) && need > 0 && bytes >= need;
}

// Parts of each row's keys so that about `ctas` CTAs run, each with `least` keys or more (below that
// the launch that joins them, some 2 us, costs more than the parts save).
int split_of(const AttendParams& p, long long base, long long ctas, int least, int forced) {
  long long s = forced > 0 ? forced : ctas / (base > 0 ? base : 1);
  const long long by_len = ((long long)p.max_len + p.nodes + least - 1) / least;
  const long long by_part = attend_part_rows(p.m) / ((long long)p.rows * p.kv_heads * p.m);
  if (s > by_len && forced <= 0) s = by_len;
  if (s > by_part) s = by_part;
  return s < 1 ? 1 : (int)s;
}

bool vectors16(const AtView& v) {
  return ((reinterpret_cast<uintptr_t>(v.data) | (uint64_t)v.row | (uint64_t)v.pos | (uint64_t)v.head) & 15) == 0;
}

// The tensor-core kernel's tensor maps: key, value, the drafted ones and the queries (copies of the
// key's where there are none).  False where a map cannot describe the tensors.
bool encode_maps(CUtensorMap (&maps)[5], AttendParams& p, int dtype) {
  if (!encode_keys(maps, p, dtype, kAtTcBox)) return false;
  maps[2] = maps[0];
  maps[3] = maps[1];
  maps[4] = maps[0];
  p.q_tma = !p.negate && encode_queries(&maps[4], p, dtype, kAtTcSlot);
  if (!p.nodes) return true;
  for (const AtView& v : {p.dkey, p.dvalue})
    if ((p.rows > 1 && v.row == 0) || (p.kv_heads > 1 && v.head == 0) || (p.nodes > 1 && v.pos == 0)) return false;
  return encode_attend(&maps[2], p.dkey, dtype, p.dim, p.nodes, p.kv_heads, p.rows, kAtTcBox) &&
         encode_attend(&maps[3], p.dvalue, dtype, p.dim, p.nodes, p.kv_heads, p.rows, kAtTcBox);
}

// Whether the tcgen05 kernel takes a 16-bit call, from the times of both kernels over queries per
// key head (1 to 64), row lengths (128 to 6000) and problems (32 to 1500); times in us, warp-level
// kernel / tcgen05, bf16:
//   head 128, 32 queries, 1500 problems: 128 keys 81 / 60, 512 keys 151 / 79
//   head 128, 16 queries, 1500 problems: 256 keys 61 / 64, 512 keys 91 / 77
//   head 128, 8 queries, 256 problems: 1024 keys 28 / 29, 6000 keys 113 / 104
//   head 64, 32 queries, 1500 problems: 256 keys 54 / 67, 512 keys 87 / 76
//   head 64, 40 queries, 3200 problems: 100 keys 95 / 134
//   head 64, 72 queries, 2800 problems: 66 keys 96 / 102; 128 queries: 68 keys 158 / 101
//   head 64, 16 queries: 256 problems, 1024 keys 26 / 24; 1500 problems, 1024 keys 69 / 90
//   head 64, 8 queries, 256 problems: 6000 keys 60 / 65
bool tcgen05_pays(const AttendParams& p, long long problems) {
  const long long keys = (long long)p.max_len + p.nodes;
  if (p.m <= 8) return false;
  if (p.dim > 64) return p.m > 16 || keys > 256;
  if (p.m <= 16) return keys >= 1024 && problems <= 4 * kAtSms;
  return keys * ((p.m + 31) / 32) > 260;
}

// Whether the tiled f32 kernel takes a call and not the streaming one, which reads the keys anew for
// every eight (above head 128 four) queries.  In us, streaming / tiled: 800 problems of head 64, 200 to
// 500 positions, 8 queries 67 / 86, 12 queries 114 / 79; of head 128, 6 queries 118 / 143, 16 queries
// 204 / 140; 1024 of head 256, 300 to 700 positions, 8 queries 417 / 442, 12 queries 592 / 445.
bool tile_pays(const AttendParams& p) { return p.m > 8; }

// CTAs that an SM holds of the kernels that stream keys per warp (registers; above head 128 the rings).
int stream_ctas(const AttendParams& p, bool f32) {
  if (f32) return 4;
  if (p.dim > 128) return 1;
  return p.m <= 8 || (p.dim <= 64 && p.m <= 16) ? 3 : 2;
}

// Whether a warp takes whole rows in these kernels (the other way is four warps to a row or a part of
// it): so many rows that four warps to each would need a second round, each of a few of a warp's
// blocks.  In us, one warp / four: 1500 rows of head 64 and 4 queries, 128 keys 15 / 20, 256 20 / 25,
// 512 32 / 34; of head 128, 128 keys 21 / 28, 256 33 / 36; 256 rows of head 64, 512 keys 18 / 14; f32,
// 4096 rows of head 64, 128 keys 56 / 67, 512 of head 128 and 2000 keys 363 / 57; 16-bit heads of 256,
// 256 rows of 300 keys 30 / 25, 512 rows of 40 keys 18 / 25 and of 300 keys 32 / 42, 800 rows of 300
// keys 57 / 59 and of 500 keys 86 / 75.
bool warp_takes_rows(const AttendParams& p, long long items, bool f32) {
  const int bytes = (p.dim <= 64 ? 64 : p.dim <= 128 ? 128 : 256), most = !f32 && p.dim > 128 ? 90000 : 20000;
  return items >= (f32 ? 6 : 2 * stream_ctas(p, f32)) * kAtSms && ((long long)p.max_len + p.nodes) * bytes <= most;
}

ls_status attend(AttendParams& p, ls_dtype dtype, void* workspace, cudaStream_t stream) {
  const long long base = (long long)p.rows * p.kv_heads;
  if (base > INT_MAX / p.m) return LS_ERR_UNSUPPORTED;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.spin_limit_ns = wait_limit_ns();
  p.part_ml = reinterpret_cast<float2*>(ws + kAtHeader);
  p.part_o = reinterpret_cast<float*>(p.part_ml + attend_part_rows(p.m));
  const AttendDebug dbg = attend_debug();
  const int es = es_of(dtype);
  // whole 16-byte vectors, and steps from key to key that 32 bits hold
  const bool lines = p.dim * es % 16 == 0 && p.key.pos < INT_MAX && p.value.pos < INT_MAX && vectors16(p.q) && vectors16(p.out) && vectors16(p.key) &&
                     vectors16(p.value) && vectors16(p.dkey) && vectors16(p.dvalue);
  const bool tensor = lines && dtype != LS_DTYPE_F32;
  p.kv_row_one = p.rows > 1 && p.key.row == 0;
  p.kv_head_one = p.kv_heads > 1 && p.key.head == 0;
  p.negate = p.scale_log2 < 0.0f;
  CUtensorMap maps[5];
  const bool tc = tensor && p.dim <= kAtTcDim && p.max_len > 0 &&
                  (dbg.kernel ? dbg.kernel == kAtForceTc : tcgen05_pays(p, base)) && encode_maps(maps, p, dtype);
  const bool f32 = lines && dtype == LS_DTYPE_F32 && dbg.kernel != kAtForceSimt;
  const bool tile = f32 && (dbg.kernel ? dbg.kernel == kAtForceTc : tile_pays(p));
  const bool step = f32 && !tile;
  const bool mma = tensor && !tc && dbg.kernel != kAtForceSimt && maps_describe(p);
  p.m_step = tc     ? 2 * kAtTcSlot
             : tile ? attend_tile_queries(p.m)
             : step ? attend_step_queries(p.dim, p.m)
             : mma  ? attend_mma_queries(p.dim, p.m)
                    : attend_simt_queries(dtype, p.m);
  p.m_tiles = (p.m + p.m_step - 1) / p.m_step;
  const long long whole = base * p.m_tiles;
  // The tensor-core kernels take the scale's sign in the queries, and a scale of 0 as 2^-100: masked
  // scores stay -inf, and every weight still is exactly 1.
  if (tc || mma) p.scale_log2 = std::fmax(std::fabs(p.scale_log2), 0x1p-100f);
  if (tc) {
    p.splits = split_of(p, whole, kAtSms, 512, dbg.splits);
  } else if (mma || step) {
    p.warps = dbg.warps ? dbg.warps : warp_takes_rows(p, whole, step) ? 1 : 4;
    // As many CTAs as the GPU holds at once; in f32, where rows of different lengths cost more than
    // joining up to 64 parts, twice as many (37 trees of 6 nodes, 321 to 2357 positions: 170 -> 156 us;
    // but one row of 86753, 76 parts 145 us and 152 parts 172 us), and three times in the tiled kernel
    // (3 trees of 32 nodes, up to 4378 positions: 97 -> 78 us).  16-bit heads above 128 elements, one CTA
    // per SM: three times (42 trees of 8 nodes x 2 key heads of 256, 629 to 12695: 413 -> 172 us).
    long long ctas = (long long)stream_ctas(p, step) * kAtSms;
    if (step && 2 * ctas <= 64 * whole) ctas *= 2;
    if (mma && p.dim > 128) ctas *= 3;
    p.splits = p.warps == 1 ? 1 : split_of(p, whole, ctas, mma ? 512 : 256, dbg.splits);
  } else if (tile) {
    p.splits = split_of(p, whole, 3 * attend_tile_ctas(p.dim, p.m) * kAtSms, 128, dbg.splits);
  } else {
    p.splits = split_of(p, whole, 4 * kAtSms, 128, dbg.splits);
  }
  p.items = base * p.m_tiles * p.splits;
  if (p.items > INT_MAX) return LS_ERR_UNSUPPORTED;
  p.by_split.set(p.splits);
  p.by_tile.set(p.m_tiles);
  p.by_head.set(p.kv_heads);
  p.by_group.set(p.group);
  p.by_q_len.set(p.q_len);
  p.by_m.set(p.m);
  cudaError_t e = tc    ? launch_attend_tc(maps, p, dtype, stream)
                  : tile ? launch_attend_tile(p, stream)
                  : step ? launch_attend_step(p, stream)
                  : mma ? launch_attend_mma(p, dtype, stream)
                        : launch_attend_simt(p, dtype, stream);
  if (e == cudaSuccess && p.splits > 1) e = launch_attend_join(p, dtype, stream);
  return report_cuda(e);
}

}  // namespace

namespace lsb {

bool maps_describe(const AttendParams& p) {
  // a stride of 0 means one element: the same for keys and values, or no map
  if ((p.value.row == 0) != (p.key.row == 0) || (p.value.head == 0) != (p.key.head == 0)) return false;
  for (const AtView& v : {p.key, p.value})
    if (v.row >= 1ll << 40 || v.pos >= 1ll << 40 || v.head >= 1ll << 40) return false;
  return p.max_len <= 1 || (p.key.pos > 0 && p.value.pos > 0);
}

bool encode_keys(CUtensorMap* maps, const AttendParams& p, int dtype, int box) {
  const int rows = p.kv_row_one ? 1 : p.rows, heads = p.kv_head_one ? 1 : p.kv_heads;
  return maps_describe(p) && encode_attend(&maps[0], p.key, dtype, p.dim, p.max_len, heads, rows, box) &&
         encode_attend(&maps[1], p.value, dtype, p.dim, p.max_len, heads, rows, box);
}

}  // namespace lsb

extern "C" {

size_t ls_cross_attention_workspace_size(int batch, int k, int q_len, int heads, int kv_heads, int max_src, int head_dim) {
  return workspace_size(batch, k, q_len, heads, kv_heads, max_src, head_dim);
}

size_t ls_tree_attention_workspace_size(int rows, int nodes, int heads, int kv_heads, int max_len, int head_dim) {
  if (nodes < 1 || nodes > LS_MAX_NODES) return 0;
  return workspace_size(rows, 1, nodes, heads, kv_heads, max_len, head_dim);
}

ls_status ls_cross_attention(const ls_view* q, const ls_view* key, const ls_view* value, ls_dtype dtype,
                             const int32_t* src_len, float scale, int batch, int k, int q_len, int heads, int kv_heads,
                             int max_src, int head_dim, const ls_view* out, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (!known(dtype) || !shape_ok(batch, k, q_len, heads, kv_heads, max_src, head_dim) || !std::isfinite(scale))
    return LS_ERR_INVALID_ARG;
  if (batch == 0 || q_len == 0) return LS_OK;
  const long long m = queries_per_key(k, q_len, heads / kv_heads);
  if ((long long)batch * k > INT_MAX || m > INT_MAX || max_src > kAtMaxKeys) return LS_ERR_UNSUPPORTED;
  const int es = es_of(dtype);
  if (!view_ok(q, es, false, 1, batch * k, q_len, heads) ||
      !view_ok(out, es, true, 1, batch * k, q_len, heads)) return LS_ERR_INVALID_ARG;
  if (max_src > 0 && (!view_ok(key, es, false, 1, batch, max_src, kv_heads) ||
                      !view_ok(value, es, false, 1, batch, max_src, kv_heads)))
    return LS_ERR_INVALID_ARG;
  if (!src_len || misaligned(src_len, 4) ||
      !workspace_ok(workspace, workspace_bytes, workspace_size(batch, k, q_len, heads, kv_heads, max_src, head_dim)))
    return LS_ERR_INVALID_ARG;
  const void* ptrs[] = {q->data, max_src ? key->data : nullptr, max_src ? value->data : nullptr, src_len, out->data,
                        workspace};
  if (!pointers_reachable(ptrs, 6)) return LS_ERR_INVALID_ARG;
  AttendParams p{};
  p.q = view_of(q, es);
  p.out = view_of(out, es);
  if (max_src) {
    p.key = view_of(key, es);
    p.value = view_of(value, es);
  }
  p.len = src_len;
  p.scale_log2 = (float)(scale * 1.4426950408889634);
  p.rows = batch;
  p.beams = k;
  p.q_len = q_len;
  p.kv_heads = kv_heads;
  p.group = heads / kv_heads;
  p.dim = head_dim;
  p.max_len = max_src;
  p.tokens = k * q_len;
  p.m = (int)m;
  return attend(p, dtype, workspace, static_cast<cudaStream_t>(stream));
}

ls_status ls_tree_attention(const ls_view* q, const ls_view* cache_key, const ls_view* cache_value,
                            const int32_t* cache_len, const ls_view* draft_key, const ls_view* draft_value,
                            const int32_t* parent, ls_dtype dtype, float scale, int rows, int nodes, int heads,
                            int kv_heads, int max_len, int head_dim, const ls_view* out, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!known(dtype) || nodes < 1 || nodes > LS_MAX_NODES || !std::isfinite(scale) ||
      !shape_ok(rows, 1, nodes, heads, kv_heads, max_len, head_dim))
    return LS_ERR_INVALID_ARG;
  if (rows == 0) return LS_OK;
  const long long m = queries_per_key(1, nodes, heads / kv_heads);
  if (m > INT_MAX || max_len > kAtMaxKeys) return LS_ERR_UNSUPPORTED;
  const int es = es_of(dtype);
  if (!view_ok(q, es, false, 1, rows, nodes, heads) || !view_ok(out, es, true, 1, rows, nodes, heads) ||
      !view_ok(draft_key, es, false, 1, rows, nodes, kv_heads) || !view_ok(draft_value, es, false, 1, rows, nodes, kv_heads))
    return LS_ERR_INVALID_ARG;
  if (max_len > 0 && (!view_ok(cache_key, es, false, 1, rows, max_len, kv_heads) ||
                      !view_ok(cache_value, es, false, 1, rows, max_len, kv_heads)))
    return LS_ERR_INVALID_ARG;
  if (!cache_len || misaligned(cache_len, 4) || !parent || misaligned(parent, 4) ||
      !workspace_ok(workspace, workspace_bytes, workspace_size(rows, 1, nodes, heads, kv_heads, max_len, head_dim)))
    return LS_ERR_INVALID_ARG;
  const void* ptrs[] = {q->data,   max_len ? cache_key->data : nullptr, max_len ? cache_value->data : nullptr,
                        cache_len, draft_key->data, draft_value->data,  parent, out->data, workspace};
  if (!pointers_reachable(ptrs, 9)) return LS_ERR_INVALID_ARG;
  AttendParams p{};
  p.q = view_of(q, es);
  p.out = view_of(out, es);
  if (max_len) {
    p.key = view_of(cache_key, es);
    p.value = view_of(cache_value, es);
  }
  p.dkey = view_of(draft_key, es);
  p.dvalue = view_of(draft_value, es);
  p.len = cache_len;
  p.parent = parent;
  p.scale_log2 = (float)(scale * 1.4426950408889634);
  p.rows = rows;
  p.beams = 1;
  p.q_len = nodes;
  p.kv_heads = kv_heads;
  p.group = heads / kv_heads;
  p.dim = head_dim;
  p.max_len = max_len;
  p.nodes = nodes;
  p.tokens = nodes;
  p.m = (int)m;
  return attend(p, dtype, workspace, static_cast<cudaStream_t>(stream));
}

ls_status ls_tree_commit(void* cache_key, void* cache_value, const int32_t* cache_len, const ls_view* draft_key,
                         const ls_view* draft_value, ls_dtype dtype, const int32_t* parent, const int32_t* token,
                         const int32_t* target, const uint8_t* finished, int eos_id, int layers, int rows, int nodes,
                         int heads, int max_len, int head_dim, int32_t* out_len, int32_t* out_path, int32_t* out_count,
                         int32_t* out_token, uint8_t* out_finished, void* workspace, void* stream) {
  if (!known(dtype) || layers < 0 || rows < 0 || nodes < 1 || nodes > LS_MAX_NODES || heads < 0 || max_len < 0 ||
      head_dim < 0)
    return LS_ERR_INVALID_ARG;
  if (rows == 0) return LS_OK;
  const int es = es_of(dtype);
  const bool move = layers > 0 && heads > 0 && head_dim > 0 && max_len > 0;
  if (move && (!cache_key || !cache_value || cache_key == cache_value || misaligned(cache_key, (size_t)es) ||
               misaligned(cache_value, (size_t)es) || !view_ok(draft_key, es, false, layers, rows, nodes, heads) ||
               !view_ok(draft_value, es, false, layers, rows, nodes, heads)))
    return LS_ERR_INVALID_ARG;
  const void* words[] = {cache_len, parent, token, target, out_len, out_path, out_count, out_token};
  for (const void* w : words)
    if (!w || misaligned(w, 4)) return LS_ERR_INVALID_ARG;
  // (every layer's block reads these inputs, whichever of them has written the outputs)
  if (out_len == cache_len || (finished && out_finished == finished) || (workspace && misaligned(workspace, 256))) return LS_ERR_INVALID_ARG;
  const void* ptrs[] = {cache_len, parent,    token,     target,       out_len,   out_path, out_count,
                        out_token, finished,  out_finished, workspace, move ? cache_key : nullptr,
                        move ? cache_value : nullptr, move ? draft_key->data : nullptr, move ? draft_value->data : nullptr};
  if (!pointers_reachable(ptrs, 15)) return LS_ERR_INVALID_ARG;
  const long long head_bytes = (long long)head_dim * es;
  // (the copies of a row and layer are counted in 32 bits)
  if (move && (layers > 65535 || (long long)heads * head_dim > (1ll << 30) / (2 * nodes))) return LS_ERR_UNSUPPORTED;
  CommitParams p{};
  if (move) {
    p.cache_key = static_cast<unsigned char*>(cache_key);
    p.cache_value = static_cast<unsigned char*>(cache_value);
    p.dkey = view_of(draft_key, es);
    p.dvalue = view_of(draft_value, es);
    p.dkey_layer = draft_key->layer * es;
    p.dvalue_layer = draft_value->layer * es;
    const uint64_t all = reinterpret_cast<uintptr_t>(cache_key) | reinterpret_cast<uintptr_t>(cache_value) |
                         reinterpret_cast<uintptr_t>(draft_key->data) | reinterpret_cast<uintptr_t>(draft_value->data) |
                         (uint64_t)(p.dkey.row | p.dkey.pos | p.dkey.head | p.dkey_layer | p.dvalue.row | p.dvalue.pos |
                                    p.dvalue.head | p.dvalue_layer | head_bytes);
    p.unit = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 2;
    p.vec_units = (int)(head_bytes / p.unit);
    p.by_units.set(p.vec_units);
    p.by_per.set(heads * p.vec_units);
  }
  p.cache_len = cache_len;
  p.parent = parent;
  p.token = token;
  p.target = target;
  p.finished = finished;
  p.out_len = out_len;
  p.out_path = out_path;
  p.out_count = out_count;
  p.out_token = out_token;
  p.out_finished = out_finished;
  p.status = static_cast<uint32_t*>(workspace);
  p.layers = move ? layers : 1;
  p.rows = rows;
  p.nodes = nodes;
  p.heads = move ? heads : 0;
  p.max_len = max_len;
  p.eos = eos_id;
  return report_cuda(launch_tree_commit(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
