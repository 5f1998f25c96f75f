// What the C entry points of draft_api.cpp hand to their kernels: attention over the paged cache (attend_*.hip), moving
// and counting its rows and pages (pages.hip), rotary positions (rotary.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "ops.h"

struct AttendArgs {
  CacheArgs cache;  // plane[0].rows: q (bf16) and its strides, plane[1].rows: out and its strides
  const uint8_t* mask;
  int64_t ld_mask;
  int32_t mask_cols, group, out_fp32;  // group: query heads of a key head
  // the page that a position below 2^31 lies in: position >> page_shift for page sizes that are powers of two, else the upper
  // half of its product with page_magic, shifted
  uint32_t page_magic;
  int32_t page_shift;
#ifdef __HIPCC__
  __host__ __device__
#endif
  uint32_t page_of(uint32_t position) const {
    return (page_magic ? (uint32_t)(((uint64_t)position * page_magic) >> 32) : position) >> page_shift;
  }
  void set_page_size(int32_t size) {
    int log = 0;
    while ((int64_t(1) << log) < size) log++;
    const bool power = (int64_t(1) << log) == size;
    // 2^(31 + log) / size, rounded up: off by less than 2^log / size of itself, which no position below 2^31 sees
    page_magic = power ? 0u : (uint32_t)(((uint64_t(1) << (31 + log)) + (uint64_t)size - 1) / (uint64_t)size);
    page_shift = power ? log : log - 1;
  }
  int32_t rows_of_tile, part_of_tile;  // tile rows / group, and the remainder
  int32_t unit_log, heads_log;         // positions of a unit and key heads of a worker: powers of two
  int32_t open_items;                  // most items of a head, where they are fewer than its workers, else 0
  float scale;
};
// How a call is cut up: tiles of 16 nt rows, units of 2^unit_log positions, elements of a key and a value in the kernel, workers
// of each 2^heads_log key heads, open_items; the workspace's parts.
struct AttendPlan {
  int32_t nt, unit_log, heads_log, dk, dv, workers, items;
  uint64_t part, ml, open, totals, total;
};
// Waves of a workgroup, workgroups of a compute unit (what their registers and LDS leave room for), waves of a matrix core.
// With keys of 192 elements eight waves share a tile of 64 positions: 12 sequences with up to 264 rows a key head and 5000
// positions, NVFP4, took 84 us with four waves, 32 positions and two workgroups, 75 us so; with keys of 128 the same change
// took 2 x 1024 rows from 192 to 221 us.
constexpr int attend_size(int dk, int nt) { return nt == 16 || (nt == 8 && dk >= 192) ? 8 : 4; }
constexpr int attend_fit(int dk, int nt) { return nt == 1 ? (dk <= 128 ? 3 : 2) : attend_size(dk, nt) == 8 || dk > 192 ? 1 : 2; }
constexpr int attend_waves(int dk, int nt) { return attend_fit(dk, nt) * attend_size(dk, nt) / 4; }
constexpr int kAttendKeys = 64;  // positions of a tile that waves share
// Column tiles of 16 rows of a wave of tiles of 128 rows.
constexpr int attend_columns(int dk) { return dk <= 128 ? 2 : 1; }
int launch_attend_mxfp4(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream);
int launch_attend_nvfp4(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream);
int launch_attend_mxfp8(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream);
// (what those call for results in fp32 with nt > 1)
int launch_attend_mxfp4_fp32(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream);
int launch_attend_nvfp4_fp32(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream);
int launch_attend_mxfp8_fp32(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream);

// A plane of bytes: `row` bytes a token, moved in units of `unit` bytes.
struct BytePlane {
  uint8_t* base;
  int64_t row;
  int32_t unit;
};
struct MoveArgs {
  BytePlane plane[4];
  int64_t ends[4];  // units of a token up to and with each plane
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
