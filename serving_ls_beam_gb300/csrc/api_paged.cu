// C-ABI entry points of the paged cache and of sampling with filters (declared in include/ls_beam.h):
// argument checks on the host, launch plans, and the enqueue of the kernels on the caller's stream.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "ls_beam.h"
#include "ls_filter.h"
#include "ls_internal.h"
#include "ls_paged.h"

using namespace lsb;

namespace {

constexpr size_t kPgHeader = 256;  // status word
constexpr int kPgMaxPlaces = INT32_MAX - 1023;

int bytes_of(ls_dtype d) { return d == LS_DTYPE_F32 ? 4 : d == LS_DTYPE_F16 || d == LS_DTYPE_BF16 ? 2 : 1; }
bool real(ls_dtype d) { return d == LS_DTYPE_F32 || d == LS_DTYPE_F16 || d == LS_DTYPE_BF16; }
bool coded(ls_dtype d) { return d == LS_DTYPE_E4M3 || d == LS_DTYPE_I8; }
bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// A view's pointer, and strides whose largest byte offset 64 bits hold; `written`: dimensions of more
// than one element need a stride.
bool view_fits(const ls_view& v, int es, bool written, int rows, int pos, int heads) {
  if (!v.data || misaligned(v.data, (size_t)es)) return false;
  const struct {
    int64_t stride;
    int extent;
  } dims[] = {{v.row, rows}, {v.pos, pos}, {v.head, heads}};
  for (const auto& d : dims) {
    if (d.stride < 0 || (written && d.extent > 1 && d.stride == 0)) return false;
    if (d.stride > (INT64_MAX >> 4) / es / (d.extent > 1 ? d.extent : 1)) return false;
  }
  return true;
}

AtView bytes_view(const ls_view& v, int es) {
  return AtView{static_cast<unsigned char*>(v.data), v.row * es, v.pos * es, v.head * es};
}

bool lines(const AtView& v) {
  return ((reinterpret_cast<uintptr_t>(v.data) | (uint64_t)v.row | (uint64_t)v.pos | (uint64_t)v.head) & 15) == 0;
}

// The pages' own arguments, for `rows` rows: LS_OK and their byte views, or what is wrong.
ls_status pages_of(const ls_pages* g, ls_dtype dtype, bool written, int rows, PageViews* out) {
  if (!g || !(real(g->dtype) || coded(g->dtype)) || (real(g->dtype) && g->dtype != dtype)) return LS_ERR_INVALID_ARG;
  if (g->num_pages < 0 || g->page_size < 1 || g->max_pages < 0 || g->kv_heads < 1 || g->head_dim < 1 || g->head_dim > kAtMaxDim)
    return LS_ERR_INVALID_ARG;
  if ((long long)g->page_size * g->max_pages > kPgMaxPlaces) return LS_ERR_UNSUPPORTED;
  const int es = bytes_of(g->dtype);
  PageViews v{};
  if (g->num_pages > 0) {
    if (!view_fits(g->key, es, written, g->num_pages, g->page_size, g->kv_heads) ||
        !view_fits(g->value, es, written, g->num_pages, g->page_size, g->kv_heads))
      return LS_ERR_INVALID_ARG;
    if (written && g->key.data == g->value.data) return LS_ERR_INVALID_ARG;
    v.key = bytes_view(g->key, es);
    v.value = bytes_view(g->value, es);
    if (coded(g->dtype)) {
      if (!view_fits(g->key_scale, 4, written, g->num_pages, g->page_size, g->kv_heads) ||
          !view_fits(g->value_scale, 4, written, g->num_pages, g->page_size, g->kv_heads))
        return LS_ERR_INVALID_ARG;
      if (written && g->key_scale.data == g->value_scale.data) return LS_ERR_INVALID_ARG;
      v.kscale = bytes_view(g->key_scale, 4);
      v.vscale = bytes_view(g->value_scale, 4);
    }
  }
  if (g->max_pages > 0) {
    if (!g->table || misaligned(g->table, 4) || g->table_row < 0 || g->table_row > (INT64_MAX >> 4) / 4 / (rows > 0 ? rows : 1))
      return LS_ERR_INVALID_ARG;
  }
  v.table = g->table;
  v.table_row = g->table_row;
  v.num_pages = g->num_pages;
  v.page_size = g->page_size;
  v.places = g->page_size * g->max_pages;
  v.by_page.set(g->page_size);
  *out = v;
  return LS_OK;
}

bool page_lines(const PageViews& v) { return lines(v.key) && lines(v.value); }

ls_status move(const ls_view* key, const ls_view* value, ls_dtype dtype, const int32_t* start, const int32_t* count,
               const ls_pages* pages, int rows, int tokens, bool read, void* workspace, void* stream) {
  if (!real(dtype) || rows < 0 || tokens < 0) return LS_ERR_INVALID_ARG;
  PageMoveParams p{};
  const ls_status s = pages_of(pages, dtype, !read, rows, &p.pages);
  if (s != LS_OK) return s;
  if (rows == 0 || tokens == 0) return LS_OK;
  const int heads = pages->kv_heads, es = bytes_of(dtype);
  if ((long long)rows * tokens > INT_MAX / heads) return LS_ERR_UNSUPPORTED;
  if (!key || !value || !view_fits(*key, es, read, rows, tokens, heads) || !view_fits(*value, es, read, rows, tokens, heads) ||
      (read && key->data == value->data))
    return LS_ERR_INVALID_ARG;
  if ((!read && !start) || misaligned(start, 4) || misaligned(count, 4) || misaligned(workspace, 256)) return LS_ERR_INVALID_ARG;
  const void* ptrs[] = {key->data, value->data, start, count, p.pages.key.data, p.pages.value.data, p.pages.kscale.data,
                        p.pages.vscale.data, pages->max_pages ? p.pages.table : nullptr, workspace};
  if (!pointers_reachable(ptrs, 10)) return LS_ERR_INVALID_ARG;
  p.key = bytes_view(*key, es);
  p.value = bytes_view(*value, es);
  p.start = start;
  p.count = count;
  p.status = static_cast<uint32_t*>(workspace);
  p.rows = rows;
  p.tokens = tokens;
  p.heads = heads;
  p.dim = pages->head_dim;
  p.vectors = (long long)rows * tokens * heads;
  p.by_head.set(heads);
  p.by_token.set(tokens);
  const bool vec = p.dim % 16 == 0 && page_lines(p.pages) && lines(p.key) && lines(p.value);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return report_cuda(read ? launch_page_read(p, dtype, pages->dtype, vec, st) : launch_page_write(p, dtype, pages->dtype, vec, st));
}

// Rows of partial sums: two places for each worker of the largest launch, of up to 16 queries.
long long part_rows(int group, int dim) {
  const int most = dim <= 64 ? kPgMaxWorkers : kPgMaxWorkers / 4 * 3;  // (paged_mma_ctas, paged_simt_ctas)
  return 2ll * (most + 1) * (group < kPgMaxTile ? group : kPgMaxTile);
}

}  // namespace

extern "C" {

ls_status ls_paged_write(const ls_view* key, const ls_view* value, ls_dtype dtype, const int32_t* start, const int32_t* count,
                         const ls_pages* pages, int rows, int tokens, void* workspace, void* stream) {
  return move(key, value, dtype, start, count, pages, rows, tokens, false, workspace, stream);
}

ls_status ls_paged_read(const ls_pages* pages, const int32_t* start, const int32_t* count, const ls_view* key,
                        const ls_view* value, ls_dtype dtype, int rows, int tokens, void* workspace, void* stream) {
  return move(key, value, dtype, start, count, pages, rows, tokens, true, workspace, stream);
}

size_t ls_paged_attention_workspace_size(int rows, int heads, int kv_heads, int head_dim) {
  if (rows < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || head_dim < 1 || head_dim > kAtMaxDim) return 0;
  return kPgHeader + (size_t)kPgMaxWorkers * 4 + (size_t)part_rows(heads / kv_heads, head_dim) * (size_t)(head_dim + 2) * 4;
}

ls_status ls_paged_attention(const ls_view* q, const ls_pages* pages, const int32_t* len, ls_dtype dtype, float scale, int rows,
                             int heads, const ls_view* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!real(dtype) || rows < 0 || heads < 1 || !std::isfinite(scale)) return LS_ERR_INVALID_ARG;
  PagedParams p{};
  const ls_status s = pages_of(pages, dtype, false, rows, &p.pages);
  if (s != LS_OK) return s;
  if (heads % pages->kv_heads != 0) return LS_ERR_INVALID_ARG;
  if (rows == 0) return LS_OK;
  if ((long long)rows * heads > kPgMaxPlaces) return LS_ERR_UNSUPPORTED;  // (rows are counted on by up to 128)
  const int es = bytes_of(dtype);
  if (!q || !out || !view_fits(*q, es, false, rows, 1, heads) || !view_fits(*out, es, true, rows, 1, heads) || !len || misaligned(len, 4))
    return LS_ERR_INVALID_ARG;
  const size_t need = ls_paged_attention_workspace_size(rows, heads, pages->kv_heads, pages->head_dim);
  if (!workspace || misaligned(workspace, 256) || workspace_bytes < need) return LS_ERR_INVALID_ARG;
  const void* ptrs[] = {q->data, out->data, len, p.pages.key.data, p.pages.value.data, p.pages.kscale.data, p.pages.vscale.data,
                        pages->max_pages ? p.pages.table : nullptr, workspace};
  if (!pointers_reachable(ptrs, 9)) return LS_ERR_INVALID_ARG;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.q = bytes_view(*q, es);
  p.out = bytes_view(*out, es);
  p.len = len;
  p.status = reinterpret_cast<uint32_t*>(ws);
  p.arrived = reinterpret_cast<uint32_t*>(ws + kPgHeader);
  p.scale_log2 = (float)(scale * 1.4426950408889634);
  p.rows = rows;
  p.kv_heads = pages->kv_heads;
  p.group = heads / pages->kv_heads;
  p.dim = pages->head_dim;
  p.part_ml = reinterpret_cast<float2*>(p.arrived + kPgMaxWorkers);
  p.part_o = reinterpret_cast<float*>(p.part_ml + part_rows(p.group, p.dim));
  const PagedDebug dbg = paged_debug();
  const int ec = bytes_of(pages->dtype);
  const bool whole = page_lines(p.pages) && p.dim * ec % 16 == 0;  // 16-byte vectors
  const bool mma = whole && dtype != LS_DTYPE_F32 && lines(p.q) && lines(p.out) && dbg.kernel != kPgForceSimt;
  const bool vec = whole && dtype == LS_DTYPE_F32;
  p.tile = mma ? paged_mma_queries(p.dim, p.group) : paged_simt_queries(p.group, vec);
  p.tiles = (p.group + p.tile - 1) / p.tile;
  if (p.tile > p.group) p.tile = p.group;
  p.per_row = p.kv_heads * p.tiles;
  p.by_tiles.set(p.tiles);
  int ctas = kAtSms * (mma ? paged_mma_ctas(p.dim, p.group) : paged_simt_ctas(vec, coded(pages->dtype), p.tile));
  if (dbg.ctas > 0 && dbg.ctas < ctas) ctas = dbg.ctas;
  const bool by_warp = mma && (dbg.warps ? dbg.warps == 1 : paged_mma_warps(p));
  p.workers = by_warp ? ctas * kPgWarps : ctas;
  // Blocks of a part where there is less work than that for each worker: of fewer, joining costs more than it brings; of
  // more, workers stand idle.  With 2, 4, 8, 16 and 32, us: by CTAs, 4 rows x 16 heads of 64 f16, 1024 positions 18.5, 18.6,
  // 11.3, 12.0, 14.4, 2 rows x 8 key heads of 128 e4m3, 4096 positions 21.6, 21.8, 15.2, 16.6, 21.4; by warps, 40 rows x 16
  // heads of 64 f16, 64 positions 10.9, 8.7, 8.5, 8.5, 8.7, 256 positions 19.4, 19.3, 17.7, 21.2, 21.1.
  p.least = dbg.least > 0 && dbg.least < 1 << 20 ? dbg.least : by_warp ? 4 : 8;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return report_cuda(mma ? launch_paged_mma(p, dtype, pages->dtype, by_warp, st) : launch_paged_simt(p, dtype, pages->dtype, vec, st));
}

ls_status ls_sample_filtered(const void* logits, ls_dtype logit_dtype, int64_t row_stride, const float* bias, const float* u,
                             const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p, int rows,
                             int vocab, int32_t* out_token, float* out_logprob, void* workspace, void* stream) {
  if (!real(logit_dtype) || rows < 0 || vocab < 1 || vocab > 1 << 28) return LS_ERR_INVALID_ARG;
  if (rows == 0) return LS_OK;
  const int es = bytes_of(logit_dtype);
  if (!logits || misaligned(logits, (size_t)es) || row_stride < vocab || row_stride > (INT64_MAX >> 4) / es / rows) return LS_ERR_INVALID_ARG;
  const void* words[] = {bias, u, temperature, top_k, top_p, min_p, out_token, out_logprob};
  for (const void* w : words)
    if (misaligned(w, 4)) return LS_ERR_INVALID_ARG;
  if (!u || !out_token || misaligned(workspace, 256)) return LS_ERR_INVALID_ARG;
  if (rows > INT_MAX / kSfMaxCluster) return LS_ERR_UNSUPPORTED;
  const void* ptrs[] = {logits, bias, u, temperature, top_k, top_p, min_p, out_token, out_logprob, workspace};
  if (!pointers_reachable(ptrs, 10)) return LS_ERR_INVALID_ARG;
  FilterParams p{};
  p.logits = static_cast<const unsigned char*>(logits);
  p.row_bytes = row_stride * es;
  p.bias = bias;
  p.u = u;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.out_token = out_token;
  p.out_logprob = out_logprob;
  p.status = static_cast<uint32_t*>(workspace);
  p.rows = rows;
  p.vocab = vocab;
  p.cluster = paged_debug().cluster;  // 0: the plan's
  int bits = 0;
  while ((1 << bits) < vocab) ++bits;
  p.shift = bits <= 18 ? 15 : 33 - bits;
  return report_cuda(launch_sample_filter(p, logit_dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
