// What the C entry points of draft_api.cpp hand to their kernels: attention over the paged cache (attend.hip), moving
// and counting its rows and pages (pages.hip), rotary positions (rotary.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "ops.h"

struct AttendArgs {
  CacheArgs cache;  // plane[0].rows: q (bf16) and its strides, plane[1].rows: out and its strides
  const uint8_t* mask;
  int64_t ld_mask;
  int32_t mask_cols, q_heads, out_fp32;
  float scale;
};
uint64_t attend_workspace(const mxfp4_cache_dims* d, int32_t q_heads, int64_t rows, int32_t n_seqs);
int launch_attend(int fmt, const AttendArgs& a, void* workspace, hipStream_t stream);

// A plane of bytes: `row` bytes a token, moved in units of `unit` bytes.
struct BytePlane {
  uint8_t* base;
  int64_t row;
  int32_t unit;
};
struct MoveArgs {
  BytePlane plane[4];
  int64_t num_pages, ld_table, ld_path;
  const int32_t *start, *path, *table;
  int32_t* lengths;
  const int32_t *src, *dst, *rows;  // pages
  int32_t n_seqs, max_pages, page_size, path_cols, n, planes;
};
int launch_compact(const MoveArgs& a, hipStream_t stream);
int launch_copy_pages(const MoveArgs& a, hipStream_t stream);

struct PoolWs {
  uint64_t need, first, from, offset, list, total;
};
struct PoolArgs {
  int64_t num_pages, ld_table;
  int32_t *refs, *table;
  const int32_t *src, *dst, *lengths;  // src, dst: fork
  int32_t *copies, *missing;
  int32_t page_size, n_rows, max_pages, n;
};
int launch_pool(bool fork, const PoolArgs& a, const PoolWs& w, uint8_t* ws, hipStream_t stream);

struct RotaryRows {
  const void* in;
  void* out;  // may be `in`, with its strides
  int64_t in_ldt, in_ldh, out_ldt, out_ldh;
  int32_t heads;
};
struct RotaryArgs {
  const double* turns;
  const int32_t* positions;
  int64_t rows;
  RotaryRows x[2];  // queries, keys (heads 0: none)
  int32_t head_dim, rot_dim, offset;
  float magnitude, sign;
};
int launch_rotary(bool fp32, bool interleaved, const RotaryArgs& a, hipStream_t stream);
