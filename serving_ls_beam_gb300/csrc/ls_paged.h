// Internal definitions of the paged cache: its write, its read and the single-token attention over
// it, shared by the host entry points (api_paged.cu) and the kernels.  Nothing here is part of the
// public interface (include/ls_beam.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ls_attend.h"
#include "ls_beam.h"

namespace lsb {

// The pages by byte strides: AtView::row from page to page, pos from place to place.
struct PageViews {
  AtView key, value, kscale, vscale;
  const int32_t* table;
  long long table_row;
  int num_pages, page_size;
  int places;          // max_pages * page_size
  AtDivisor by_page;   // by page_size
};

// LS_BEAM_DEBUG's choices: the attention kernel, a part's warps, the CTAs; the sampler's CTAs of a row (0 = plan)
constexpr int kPgForceSimt = 1;
struct PagedDebug {
  int kernel, warps, ctas, least, cluster;
};
PagedDebug paged_debug();

// One write (dense -> pages) or read (pages -> dense).
struct PageMoveParams {
  PageViews pages;
  AtView key, value;     // [rows, tokens, heads, dim] dense
  const int32_t* start;  // may be null: 0
  const int32_t* count;  // may be null: tokens
  uint32_t* status;      // may be null
  int rows, tokens, heads, dim;
  long long vectors;     // rows * tokens * heads
  AtDivisor by_head, by_token;
};
// vec: every stride and address a multiple of 16 bytes, dim of 16
cudaError_t launch_page_write(const PageMoveParams& p, int dtype, int cache, bool vec, cudaStream_t stream);
cudaError_t launch_page_read(const PageMoveParams& p, int dtype, int cache, bool vec, cudaStream_t stream);

// Blocks of a row's keys are the units of work.  A worker is a CTA of four warps, which take a
// part's blocks in turn, or a warp by itself.
constexpr int kPgWarps = 4;
constexpr int kPgThreads = kPgWarps * 32;
constexpr int kPgMaxWorkers = 4 * kPgWarps * kAtSms;  // the most workers of a launch: four CTAs per SM, by warps
constexpr int kPgMaxTile = 16;          // the most queries of an item

struct PagedParams {
  PageViews pages;
  AtView q, out;        // [rows, -, kv_heads * group, dim]
  const int32_t* len;
  uint32_t* status;
  uint32_t* arrived;    // [workers]: parts of an item that are there; zero between launches
  float* part_o;        // [2 * workers + 2, tile, dim] f32
  float2* part_ml;      // [2 * workers + 2, tile]: maximum (log2 units) and sum
  float scale_log2;     // scale * log2(e)
  int rows, kv_heads, group, dim;
  int tile;             // queries of an item
  int tiles;            // ceil(group / tile)
  int per_row;          // items of a row: kv_heads * tiles
  int workers;
  int least;            // blocks of a part where there is less than that much work for each worker
  AtDivisor by_tiles;
};
// 16-bit queries; every stride and address a multiple of 16 bytes, the vectors of 16
cudaError_t launch_paged_mma(const PagedParams& p, int dtype, int cache, bool by_warp, cudaStream_t stream);
cudaError_t launch_paged_mma_e4m3(const PagedParams& p, int dtype, bool by_warp, cudaStream_t stream);
cudaError_t launch_paged_mma_i8(const PagedParams& p, int dtype, bool by_warp, cudaStream_t stream);
bool paged_mma_warps(const PagedParams& p);
int paged_mma_queries(int dim, int group);
int paged_mma_ctas(int dim, int group);  // CTAs that an SM holds
// any types; vec: f32 queries, every stride and address a multiple of 16 bytes, the vectors of 16
cudaError_t launch_paged_simt(PagedParams p, int dtype, int cache, bool vec, cudaStream_t stream);
int paged_simt_queries(int group, bool vec);
int paged_simt_ctas(bool vec, bool codes, int tile);

}  // namespace lsb
