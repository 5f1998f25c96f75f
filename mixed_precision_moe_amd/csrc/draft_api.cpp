// C ABI of attention over the paged cache, the moving and counting of its rows and pages, and rotary positions:
// argument validation before any device work, then the launches.  Declarations and contracts are in
// include/mxfp4moe.h.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "api_checks.h"
#include "drafts.h"

namespace {

constexpr int kMaxDim = 256;        // attention: k_dim, v_dim
constexpr int kMaxHeads = 1 << 16;
constexpr int kCus = 256;
constexpr int kMaxRot = 2048;
constexpr int kMaxTableRows = 1 << 24;
constexpr int kMaxPairs = 1 << 16;  // of a fork

bool table_fits(int64_t ld_table, int32_t n_rows, int32_t max_pages) {
  return n_rows >= 0 && max_pages >= 0 && ld_table >= max_pages && ld_table <= kMaxLd;
}

// The widest access, up to 16 bytes, that every token of a plane starts on.
int unit_of(const void* base, int64_t row) {
  const uint64_t bits = (uint64_t)(uintptr_t)base | (uint64_t)row | 16;
  return (int)(bits & (~bits + 1));
}

int move_planes(MoveArgs& a, const mxfp4_cache_dims* d, void* k_q, void* k_s, void* v_q, void* v_s) {
  const bool two = d->v_dim > 0;
  if (d->num_pages > 0 && (!k_q || !k_s || (two && (!v_q || !v_s)))) return MXFP4_ERR_NULL;
  if (!aligned(k_q, 8) || (two && !aligned(v_q, 8))) return MXFP4_ERR_ALIGN;
  const int64_t per = d->fmt == MXFP4_FMT_MXFP8 ? 1 : 2, g = group_of(d->fmt), h = d->heads;
  void* base[4] = {k_q, k_s, v_q, v_s};
  const int64_t row[4] = {h * (d->k_dim / per), h * (d->k_dim / g), h * (d->v_dim / per), h * (d->v_dim / g)};
  a.planes = two ? 4 : 2;
  int64_t units = 0;
  for (int i = 0; i < 4; i++) {
    if (i < a.planes) {
      a.plane[i] = BytePlane{(uint8_t*)base[i], row[i], unit_of(base[i], row[i])};
      units += row[i] / a.plane[i].unit;
    }
    a.ends[i] = units;
  }
  a.num_pages = d->num_pages;
  a.page_size = d->page_size;
  return MXFP4_OK;
}

int check_pool(int64_t num_pages, int32_t n, int32_t max_pages) {
  if (num_pages < 0 || num_pages >= kMaxRows || n < 0 || n > kMaxTableRows || max_pages < 0 || (int64_t)n * max_pages >= kMaxRows)
    return MXFP4_ERR_SHAPE;
  return MXFP4_OK;
}

PoolWs pool_ws(int64_t num_pages, int32_t n, int32_t max_pages) {
  PoolWs w;
  uint64_t p = 0;
  auto take = [&](uint64_t bytes) { uint64_t o = p; p = up256(p + bytes); return o; };
  const uint64_t most = (uint64_t)n * (uint64_t)max_pages;
  w.need = take(4 * (uint64_t)n);
  w.first = take(4 * (uint64_t)n);
  w.from = take(4 * (uint64_t)n);
  w.offset = take(4 * ((uint64_t)n + 1));
  w.list = take(4 * (most < (uint64_t)num_pages ? most : (uint64_t)num_pages));
  w.total = p;
  return w;
}

int pool_args(PoolArgs& a, int64_t num_pages, int32_t page_size, int32_t* refs, int32_t* page_table, int64_t ld_table,
              int32_t n_rows, int32_t max_pages, const int32_t* lengths, int32_t n, int32_t* copies, int32_t* missing,
              const void* workspace, size_t workspace_bytes) {
  int st = check_pool(num_pages, n, max_pages);
  if (st || (st = check_pool(num_pages, n_rows, max_pages))) return st;
  if (page_size < 1 || !table_fits(ld_table, n_rows, max_pages)) return MXFP4_ERR_SHAPE;
  if (!missing || !workspace) return MXFP4_ERR_NULL;
  if ((num_pages > 0 && !refs) || (n_rows > 0 && max_pages > 0 && !page_table) || (n > 0 && (!lengths || !copies)))
    return MXFP4_ERR_NULL;
  if (!aligned(refs, 4) || !aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(copies, 4) ||
      !aligned(missing, 4) || !aligned(workspace, 256))
    return MXFP4_ERR_ALIGN;
  if (workspace_bytes < pool_ws(num_pages, n, max_pages).total) return MXFP4_ERR_WORKSPACE;
  a = PoolArgs{};
  a.num_pages = num_pages;
  a.ld_table = ld_table;
  a.refs = refs;
  a.table = page_table;
  a.lengths = lengths;
  a.copies = copies;
  a.missing = missing;
  a.page_size = page_size;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.n = n;
  return MXFP4_OK;
}

// The sizes of the attention kernels: dims up to 64, 128, 192 and 128, or 256; tiles of rows by what a sequence has on average:
// up to 16 and 32 the kernel whose waves split the positions, up to 64 (where it exists) and from there on the shared one.
AttendPlan attend_plan(const mxfp4_cache_dims* d, int32_t q_heads, int64_t rows, int32_t n_seqs, int64_t positions) {
  AttendPlan p = {};
  const int k = d->k_dim, v = d->v_dim;
  p.dk = k <= 64 && v <= 64 ? 64 : k <= 128 && v <= 128 ? 128 : k <= 192 && v <= 128 ? 192 : 256;
  p.dv = p.dk == 192 ? 128 : p.dk;
  const int64_t per_seq = (rows + n_seqs - 1) / (n_seqs > 0 ? n_seqs : 1) * (q_heads / d->heads);
  // Up to 32 rows each wave has positions of its own; more share tiles: 35 rows of 8 heads and 130000 positions, MXFP4, took
  // 66 us and 8 to join in tiles of 64 rows, 85 and 8 in tiles of 128, 68 and 20 with waves of three times 16.
  p.nt = per_seq <= 16 ? 1 : per_seq <= 32 ? 2 : 8;
  if (p.nt == 8 && p.dk <= 192) {
    // Tiles of 256 rows read and dequantize for twice the rows, and leave twice as much to join.  4 sequences of 4096
    // positions, MXFP4, us with tiles of 128 and 256 rows, by rows a key head; keys of 128: 256: 34, 42; 512: 44, 45;
    // 8192: 342, 330; of 192: 35, 46; 48, 53; 511, 380; of 64: 29, 36; 36, 35; 285, 245.
    const int64_t wide = (per_seq + 255) / 256 * 256, narrow = (per_seq + 127) / 128 * 128;
    p.nt = per_seq <= 64 && p.dk <= 128 ? 4 : per_seq > 512 && wide * 8 <= narrow * 9 ? 16 : 8;
  }
  if (p.nt <= 2) {
    // Heads side by side: 32 sequences of up to 3900 positions, 8 heads, MXFP8: 49 us and 5 to join, a head a workgroup 59 and 5.  Not
    // where the positions are few: one unit of all four waves then needs no join (78 positions: 7.8 us; 7.2 and 4.2).
    p.heads_log = positions <= 128 ? 0 : d->heads % 4 == 0 ? 2 : d->heads % 2 == 0 ? 1 : 0;
    p.unit_log = 7 - p.heads_log;
  } else {
    p.unit_log = 6;  // kAttendKeys
  }
  const int64_t groups = d->heads >> p.heads_log, fill = (int64_t)kCus * attend_fit(p.dk, p.nt) / groups;
  p.workers = (int32_t)(fill < 1 ? 1 : fill < 8 ? fill : fill & ~int64_t(7));  // as many on each XCD
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) { uint64_t o = at; at = up256(at + bytes); return o; };
  const uint64_t all = (uint64_t)p.workers * (uint64_t)d->heads, part_rows = 2 * all * 16 * (uint64_t)p.nt;
  p.part = take(4 * part_rows * (uint64_t)p.dv);
  p.ml = take(8 * part_rows);
  // tiles, each sequence's last one cut short
  const int64_t items = rows * (q_heads / d->heads) / (16 * p.nt) + n_seqs;
  p.items = items < p.workers ? (int32_t)items : 0;
  p.open = take(16 * (uint64_t)(p.items ? p.items : p.workers) * (uint64_t)groups);
  p.totals = take(16);
  p.total = at;
  return p;
}

// Enough for either plan of a call: it goes by its table too.
uint64_t attend_bytes(const mxfp4_cache_dims* d, int32_t q_heads, int64_t rows, int32_t n_seqs) {
  const uint64_t few = attend_plan(d, q_heads, rows, n_seqs, 0).total, many = attend_plan(d, q_heads, rows, n_seqs, INT64_MAX).total;
  return few > many ? few : many;
}

int check_attend(const mxfp4_cache_dims* d, int32_t q_heads, int64_t rows, int32_t n_seqs) {
  int st = check_cache(d, true);
  if (st) return st;
  if (d->v_dim < 1 || d->k_dim > kMaxDim || d->v_dim > kMaxDim) return MXFP4_ERR_SHAPE;
  if (q_heads < 1 || q_heads > kMaxHeads || q_heads % d->heads) return MXFP4_ERR_SHAPE;
  // rows of a key head, those past the last in a tile too, and positions are counted in 32 bits
  if (rows < 0 || rows >= kMaxRows || n_seqs < 0 || rows * (q_heads / d->heads) >= kMaxRows - 256) return MXFP4_ERR_SHAPE;
  return MXFP4_OK;
}

}  // namespace

// ------------------------------------------------------------------------------------------------
// Attention over the cache.

MX_API size_t mxfp4_cache_attend_workspace_bytes(const mxfp4_cache_dims* d, int32_t q_heads, int64_t rows,
                                                 int32_t n_seqs) {
  if (check_attend(d, q_heads, rows, n_seqs) != MXFP4_OK) return 0;
  return (size_t)attend_bytes(d, q_heads, rows, n_seqs);
}

MX_API int mxfp4_cache_attend(const mxfp4_cache_dims* d, const void* k_q, const void* k_s, const void* v_q,
                              const void* v_s, const void* q_bf16, int64_t q_ldt, int64_t q_ldh, int32_t q_heads,
                              int64_t rows, const int32_t* cu_rows, const int32_t* start, const int32_t* page_table,
                              int64_t ld_table, int32_t n_seqs, int32_t max_pages, const uint8_t* tree_mask,
                              int64_t ld_mask, int32_t mask_cols, float scale, void* out, int64_t out_ldt,
                              int64_t out_ldh, int32_t out_is_fp32, void* workspace, size_t workspace_bytes,
                              void* stream) {
  int st = check_attend(d, q_heads, rows, n_seqs);
  if (st || (st = check_flags(out_is_fp32, 0, 0))) return st;
  if (!table_fits(ld_table, n_seqs, max_pages) || (int64_t)max_pages * d->page_size > kMaxRows - 256) return MXFP4_ERR_SHAPE;
  // what the kernels multiply the scores by: finite too (the comparison also rejects NaN)
  if (!(std::fabs(scale) * 1.44269504f / (d->fmt == MXFP4_FMT_NVFP4 ? d->k_global_scale : 1.0f) <= 3.40282347e38f)) return MXFP4_ERR_SHAPE;
  auto bad_ld = [&](int64_t ldt, int64_t ldh, int32_t dim) {
    return ldt < 0 || ldt % 8 || ldt > kMaxLd || ldh < 0 || ldh % 8 || ldh > kMaxLd || (q_heads > 1 && ldh < dim) ||
           (rows > 1 && ldt < dim);
  };
  if (bad_ld(q_ldt, q_ldh, d->k_dim) || bad_ld(out_ldt, out_ldh, d->v_dim)) return MXFP4_ERR_SHAPE;
  if (tree_mask && (mask_cols < 0 || ld_mask < mask_cols || ld_mask > kMaxLd)) return MXFP4_ERR_SHAPE;
  if (rows == 0 || n_seqs == 0) return MXFP4_OK;
  if (!q_bf16 || !out || !cu_rows || (!page_table && max_pages > 0) || !workspace) return MXFP4_ERR_NULL;
  if (d->num_pages > 0 && (!k_q || !k_s || !v_q || !v_s)) return MXFP4_ERR_NULL;
  if (!aligned(q_bf16, 16) || !aligned(out, 16) || !aligned(k_q, 8) || !aligned(v_q, 8) || !aligned(cu_rows, 4) ||
      !aligned(start, 4) || !aligned(page_table, 4) || !aligned(workspace, 256))
    return MXFP4_ERR_ALIGN;
  const AttendPlan plan = attend_plan(d, q_heads, rows, n_seqs, (int64_t)max_pages * d->page_size);
  if (workspace_bytes < attend_bytes(d, q_heads, rows, n_seqs)) return MXFP4_ERR_WORKSPACE;
  AttendArgs a = {};
  CacheArgs& c = a.cache;
  c.plane[0] = CachePlane{(void*)q_bf16, q_ldt, q_ldh, (uint8_t*)k_q, (uint8_t*)k_s, d->k_dim, d->k_global_scale};
  c.plane[1] = CachePlane{out, out_ldt, out_ldh, (uint8_t*)v_q, (uint8_t*)v_s, d->v_dim, d->v_global_scale};
  c.rows = rows;
  c.num_pages = d->num_pages;
  c.ld_table = ld_table;
  c.cu = cu_rows;
  c.start = start;
  c.table = page_table;
  c.n_seqs = n_seqs;
  c.max_pages = d->num_pages > 0 ? max_pages : 0;  // a table of no page at all has no positions
  c.page_size = d->page_size;
  c.heads = d->heads;
  a.mask = tree_mask;
  a.ld_mask = ld_mask;
  a.mask_cols = mask_cols;
  a.group = q_heads / d->heads;
  a.out_fp32 = out_is_fp32;
  a.set_page_size(d->page_size);
  a.rows_of_tile = 16 * plan.nt / a.group;
  a.part_of_tile = 16 * plan.nt % a.group;
  a.unit_log = plan.unit_log;
  a.heads_log = plan.heads_log;
  a.open_items = plan.items;
  a.scale = scale;
  uint8_t* ws = (uint8_t*)workspace;
  if (d->fmt == MXFP4_FMT_MXFP4) return launch_attend_mxfp4(a, plan, ws, S(stream));
  if (d->fmt == MXFP4_FMT_NVFP4) return launch_attend_nvfp4(a, plan, ws, S(stream));
  return launch_attend_mxfp8(a, plan, ws, S(stream));
}

// ------------------------------------------------------------------------------------------------
// Rows and pages.

MX_API int mxfp4_cache_compact(const mxfp4_cache_dims* d, const int32_t* start, const int32_t* path, int64_t ld_path,
                               int32_t path_cols, const int32_t* page_table, int64_t ld_table, int32_t n_seqs,
                               int32_t max_pages, int32_t* lengths, void* k_q, void* k_s, void* v_q, void* v_s,
                               void* stream) {
  int st = check_cache(d, false);
  if (st) return st;
  if (!table_fits(ld_table, n_seqs, max_pages) || path_cols < 0 || ld_path < path_cols || ld_path > kMaxLd)
    return MXFP4_ERR_SHAPE;
  if (n_seqs == 0) return MXFP4_OK;
  if ((!path && path_cols > 0) || (!page_table && max_pages > 0)) return MXFP4_ERR_NULL;
  MoveArgs a = {};
  if ((st = move_planes(a, d, k_q, k_s, v_q, v_s))) return st;
  if (!aligned(start, 4) || !aligned(path, 4) || !aligned(page_table, 4) || !aligned(lengths, 4)) return MXFP4_ERR_ALIGN;
  a.ld_table = ld_table;
  a.ld_path = ld_path;
  a.start = start;
  a.path = path;
  a.table = page_table;
  a.lengths = lengths;
  a.n_seqs = n_seqs;
  a.max_pages = max_pages;
  a.path_cols = path_cols;
  return launch_compact(a, S(stream));
}

MX_API int mxfp4_cache_copy_pages(const mxfp4_cache_dims* d, const int32_t* src, const int32_t* dst,
                                  const int32_t* rows, int32_t n, void* k_q, void* k_s, void* v_q, void* v_s,
                                  void* stream) {
  int st = check_cache(d, false);
  if (st) return st;
  if (n < 0) return MXFP4_ERR_SHAPE;
  if (n == 0) return MXFP4_OK;
  if (!src || !dst) return MXFP4_ERR_NULL;
  MoveArgs a = {};
  if ((st = move_planes(a, d, k_q, k_s, v_q, v_s))) return st;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(rows, 4)) return MXFP4_ERR_ALIGN;
  a.src = src;
  a.dst = dst;
  a.rows = rows;
  a.n = n;
  return launch_copy_pages(a, S(stream));
}

MX_API size_t mxfp4_pool_workspace_bytes(int64_t num_pages, int32_t n, int32_t max_pages) {
  if (check_pool(num_pages, n, max_pages) != MXFP4_OK) return 0;
  return (size_t)pool_ws(num_pages, n, max_pages).total;
}

MX_API int mxfp4_pool_resize(int64_t num_pages, int32_t page_size, int32_t* refs, int32_t* page_table,
                             int64_t ld_table, int32_t n_rows, int32_t max_pages, const int32_t* lengths,
                             int32_t* copies, int32_t* missing, void* workspace, size_t workspace_bytes, void* stream) {
  PoolArgs a;
  int st = pool_args(a, num_pages, page_size, refs, page_table, ld_table, n_rows, max_pages, lengths, n_rows, copies,
                     missing, workspace, workspace_bytes);
  if (st) return st;
  return launch_pool(false, a, pool_ws(num_pages, n_rows, max_pages), (uint8_t*)workspace, S(stream));
}

MX_API int mxfp4_pool_fork(int64_t num_pages, int32_t page_size, int32_t* refs, int32_t* page_table, int64_t ld_table,
                           int32_t n_rows, int32_t max_pages, const int32_t* src, const int32_t* dst,
                           const int32_t* lengths, int32_t n, int32_t* copies, int32_t* missing, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (n > kMaxPairs) return MXFP4_ERR_SHAPE;
  PoolArgs a;
  int st = pool_args(a, num_pages, page_size, refs, page_table, ld_table, n_rows, max_pages, lengths, n, copies,
                     missing, workspace, workspace_bytes);
  if (st) return st;
  if (n > 0 && (!src || !dst)) return MXFP4_ERR_NULL;
  if (!aligned(src, 4) || !aligned(dst, 4)) return MXFP4_ERR_ALIGN;
  a.src = src;
  a.dst = dst;
  return launch_pool(true, a, pool_ws(num_pages, n, max_pages), (uint8_t*)workspace, S(stream));
}

// ------------------------------------------------------------------------------------------------
// Rotary positions.

MX_API int mxfp4_rotary(const double* turns, const int32_t* positions, int64_t rows, int32_t head_dim, int32_t rot_dim,
                        int32_t offset, int32_t interleaved, float magnitude, int32_t inverse, int32_t is_fp32,
                        const void* q, int64_t q_ldt, int64_t q_ldh, int32_t q_heads, void* q_out, int64_t q_out_ldt,
                        int64_t q_out_ldh, const void* k, int64_t k_ldt, int64_t k_ldh, int32_t k_heads, void* k_out,
                        int64_t k_out_ldt, int64_t k_out_ldh, void* stream) {
  int st = check_flags(interleaved, inverse, is_fp32);
  if (st) return st;
  if (head_dim < 1 || head_dim > (1 << 16) || rot_dim < 2 || rot_dim > kMaxRot || rot_dim % 2 || offset < 0 ||
      offset > head_dim - rot_dim || rows < 0 || rows >= kMaxRows)
    return MXFP4_ERR_SHAPE;
  if (!(magnitude >= -3.40282347e38f && magnitude <= 3.40282347e38f)) return MXFP4_ERR_SHAPE;
  if (!k) k_heads = 0;
  auto bad = [](int64_t ldt, int64_t ldh) { return ldt < 0 || ldt > kMaxLd || ldh < 0 || ldh > kMaxLd; };
  auto overlaps = [&](int64_t ldt, int64_t ldh, int32_t heads) {
    return (heads > 1 && ldh < head_dim) || (rows > 1 && ldt < head_dim);
  };
  if (q_heads < 1 || (int64_t)q_heads * head_dim > kMaxWidth || bad(q_ldt, q_ldh) || bad(q_out_ldt, q_out_ldh) ||
      overlaps(q_out_ldt, q_out_ldh, q_heads))
    return MXFP4_ERR_SHAPE;
  if (k && (k_heads < 1 || (int64_t)k_heads * head_dim > kMaxWidth || bad(k_ldt, k_ldh) || bad(k_out_ldt, k_out_ldh) ||
            overlaps(k_out_ldt, k_out_ldh, k_heads)))
    return MXFP4_ERR_SHAPE;
  if (rows == 0) return MXFP4_OK;
  if (!turns || !positions || !q || !q_out || (k && !k_out)) return MXFP4_ERR_NULL;
  const uintptr_t e = is_fp32 ? 4 : 2;
  if (!aligned(turns, 8) || !aligned(positions, 4) || !aligned(q, e) || !aligned(q_out, e) || !aligned(k, e) ||
      (k && !aligned(k_out, e)))
    return MXFP4_ERR_ALIGN;
  RotaryArgs a = {};
  a.turns = turns;
  a.positions = positions;
  a.rows = rows;
  a.x[0] = RotaryRows{q, q_out, q_ldt, q_ldh, q_out_ldt, q_out_ldh, q_heads};
  if (k) a.x[1] = RotaryRows{k, k_out, k_ldt, k_ldh, k_out_ldt, k_out_ldh, k_heads};
  a.head_dim = head_dim;
  a.rot_dim = rot_dim;
  a.offset = offset;
  a.magnitude = magnitude;
  a.sign = inverse ? -1.0f : 1.0f;
  return launch_rotary(is_fp32, interleaved, a, S(stream));
}
