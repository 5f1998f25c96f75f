// Calls the entry points of csrc/draft_api.cpp on the CPU with valid and invalid arguments; the kernel launchers are stand-ins
// that record what they were given.  Built with AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_drafts_abi.py.
#include <climits>
#include <cmath>
#include <cstdio>

#include "../../mixed_precision_moe_amd/csrc/drafts.h"

static int g_fail = 0, g_launches = 0, g_fmt = -1;
static AttendArgs g_at;
static AttendPlan g_plan;
static MoveArgs g_move;
static PoolArgs g_pool;
static PoolWs g_pool_ws;
static RotaryArgs g_rot;
#define CHECK(c)                                               \
  do {                                                         \
    if (!(c)) {                                                \
      std::printf("FAIL %s:%d: %s\n", __FILE__, __LINE__, #c); \
      g_fail++;                                                \
    }                                                          \
  } while (0)

static int attend(int fmt, const AttendArgs& a, const AttendPlan& p) {
  g_launches++;
  g_fmt = fmt;
  g_at = a;
  g_plan = p;
  return MXFP4_OK;
}
int launch_attend_mxfp4(const AttendArgs& a, const AttendPlan& p, uint8_t*, hipStream_t) { return attend(0, a, p); }
int launch_attend_nvfp4(const AttendArgs& a, const AttendPlan& p, uint8_t*, hipStream_t) { return attend(1, a, p); }
int launch_attend_mxfp8(const AttendArgs& a, const AttendPlan& p, uint8_t*, hipStream_t) { return attend(2, a, p); }
int launch_compact(const MoveArgs& a, hipStream_t) {
  g_launches++;
  g_move = a;
  return MXFP4_OK;
}
int launch_copy_pages(const MoveArgs& a, hipStream_t) {
  g_launches++;
  g_move = a;
  return MXFP4_OK;
}
int launch_pool(bool, const PoolArgs& a, const PoolWs& w, uint8_t*, hipStream_t) {
  g_launches++;
  g_pool = a;
  g_pool_ws = w;
  return MXFP4_OK;
}
int launch_rotary(bool, bool, const RotaryArgs& a, hipStream_t) {
  g_launches++;
  g_rot = a;
  return MXFP4_OK;
}

template <typename T = void>
static T* fake(uintptr_t off = 0) { return (T*)((uintptr_t(1) << 32) + off); }

static const mxfp4_cache_dims kOk = {MXFP4_FMT_MXFP8, 2, 64, 96, 16, 10, 1.0f, 1.0f};

static void test_attend() {
  struct Call {
    mxfp4_cache_dims d = kOk;
    void *kq = fake(), *q = fake(), *out = fake(), *ws = fake();
    int64_t q_ldt = 384, q_ldh = 64, rows = 5, ld_table = 4, ld_mask = 8, o_ldt = 576, o_ldh = 96;
    int32_t q_heads = 6, n = 2, pages = 4, cols = 8, fp32 = 0;
    int32_t *cu = fake<int32_t>(), *start = nullptr, *table = fake<int32_t>();
    uint8_t* mask = nullptr;
    float scale = 0.1f;
    int64_t short_by = 0;
    int run() const {
      const size_t n_ws = mxfp4_cache_attend_workspace_bytes(&d, q_heads, rows, n);
      return mxfp4_cache_attend(&d, kq, fake(), fake(), fake(1), q, q_ldt, q_ldh, q_heads, rows, cu, start, table, ld_table, n, pages,
                                mask, ld_mask, cols, scale, out, o_ldt, o_ldh, fp32, ws, n_ws - short_by, nullptr);
    }
  };
  auto with = [](auto f) {
    Call c;
    f(c);
    return c.run();
  };
  g_launches = 0;
  CHECK(with([](Call& c) { c.d.v_dim = 0; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.d.k_dim = 288; c.q_ldh = 288; c.q_ldt = 2000; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.d.fmt = 7; }) == MXFP4_ERR_LAYOUT);
  CHECK(with([](Call& c) { c.q_heads = 5; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.q_heads = 0; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.q_heads = (1 << 16) + 2; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.rows = -1; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.rows = int64_t(1) << 31; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.n = -1; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.pages = 5; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.q_ldh = 63; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.q_ldh = 56; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.q_ldt = 32; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.o_ldt = 580; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.o_ldh = 64; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.fp32 = 2; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.scale = NAN; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.scale = INFINITY; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.mask = fake<uint8_t>(); c.ld_mask = 7; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.mask = fake<uint8_t>(); c.cols = -1; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.q = nullptr; }) == MXFP4_ERR_NULL);
  CHECK(with([](Call& c) { c.out = nullptr; }) == MXFP4_ERR_NULL);
  CHECK(with([](Call& c) { c.cu = nullptr; }) == MXFP4_ERR_NULL);
  CHECK(with([](Call& c) { c.table = nullptr; }) == MXFP4_ERR_NULL);
  CHECK(with([](Call& c) { c.kq = nullptr; }) == MXFP4_ERR_NULL);
  CHECK(with([](Call& c) { c.ws = nullptr; }) == MXFP4_ERR_NULL);
  CHECK(with([](Call& c) { c.q = fake(8); }) == MXFP4_ERR_ALIGN);
  CHECK(with([](Call& c) { c.out = fake(8); }) == MXFP4_ERR_ALIGN);
  CHECK(with([](Call& c) { c.kq = fake(4); }) == MXFP4_ERR_ALIGN);
  CHECK(with([](Call& c) { c.cu = fake<int32_t>(2); }) == MXFP4_ERR_ALIGN);
  CHECK(with([](Call& c) { c.ws = fake(128); }) == MXFP4_ERR_ALIGN);
  CHECK(with([](Call& c) { c.short_by = 1; }) == MXFP4_ERR_WORKSPACE);
  CHECK(with([](Call& c) { c.rows = 0; }) == MXFP4_OK);
  CHECK(with([](Call& c) { c.n = 0; }) == MXFP4_OK);
  CHECK(g_launches == 0);
  CHECK(with([](Call&) {}) == MXFP4_OK && g_launches == 1 && g_fmt == 2 && g_at.group == 3 && !g_at.mask);
  CHECK(with([](Call& c) { c.kq = nullptr; c.d.num_pages = 0; }) == MXFP4_OK);
  CHECK(with([](Call& c) { c.table = nullptr; c.pages = 0; }) == MXFP4_OK);
  CHECK(with([](Call& c) { c.kq = fake(8); c.d.fmt = MXFP4_FMT_MXFP4; c.mask = fake<uint8_t>(3); c.cols = 0; }) == MXFP4_OK &&
        g_fmt == 0 && g_at.mask && g_at.mask_cols == 0);
  // one row: its strides are not looked at against each other; dims and rows choose the kernel
  CHECK(with([](Call& c) { c.rows = 1; c.q_ldt = 0; c.o_ldt = 0; c.n = 1; }) == MXFP4_OK);
  mxfp4_cache_dims d = kOk;
  for (int dim : {32, 64, 96, 128, 160, 192, 224, 256})
    for (int v : {32, 64, 96, 128, 160, 256})
      for (int64_t rows : {1, 7, 16, 17, 33, 64, 65, 4000})
        for (int heads : {1, 2, 300, 4096}) {
          d.k_dim = dim;
          d.v_dim = v;
          d.heads = heads;
          const int rc = mxfp4_cache_attend(&d, fake(), fake(), fake(), fake(), fake(), 1 << 20, dim, heads, rows, fake<int32_t>(),
                                            nullptr, fake<int32_t>(), 4, 1, 4, nullptr, 0, 0, 1.0f, fake(), 1 << 20, v, 0, fake(),
                                            mxfp4_cache_attend_workspace_bytes(&d, heads, rows, 1), nullptr);
          CHECK(rc == MXFP4_OK);
          CHECK(g_plan.dk >= dim && g_plan.dv >= v && g_plan.nt >= 1 && g_plan.nt <= 16 && g_plan.workers >= 1);
          CHECK(g_plan.total <= mxfp4_cache_attend_workspace_bytes(&d, heads, rows, 1));
          // the parts follow each other inside the workspace
          const uint64_t workers = (uint64_t)g_plan.workers * heads, part_rows = 2 * workers * 16 * g_plan.nt;
          CHECK(g_plan.part + 4 * part_rows * g_plan.dv <= g_plan.ml && g_plan.ml + 8 * part_rows <= g_plan.open &&
                g_plan.open + 16 * ((g_plan.items ? (uint64_t)g_plan.items * heads : workers) >> g_plan.heads_log) <= g_plan.totals &&
                g_plan.totals + 16 <= g_plan.total);
        }
  d = kOk;
  CHECK(mxfp4_cache_attend_workspace_bytes(&d, 3, 5, 2) == 0 && mxfp4_cache_attend_workspace_bytes(nullptr, 4, 5, 2) == 0);
  CHECK(mxfp4_cache_attend_workspace_bytes(&d, 4, 0, 0) > 0);
  // rows of a key head up to the end of the largest tile are counted in 32 bits
  d.heads = 1;
  CHECK(mxfp4_cache_attend_workspace_bytes(&d, 1, (int64_t(1) << 31) - 257, 1) > 0);
  CHECK(mxfp4_cache_attend_workspace_bytes(&d, 1, (int64_t(1) << 31) - 256, 1) == 0);
  CHECK(mxfp4_cache_attend_workspace_bytes(&d, 4, (int64_t(1) << 29) - 64, 1) == 0);
}

// The division by the page size is exact for every position.
static void test_page_of() {
  AttendArgs a = {};
  for (int64_t size : {1ll, 2ll, 3ll, 5ll, 7ll, 16ll, 24ll, 96ll, 100ll, 128ll, 129ll, 1000ll, 65535ll, 65537ll, 1ll << 30, (1ll << 30) + 1, (1ll << 31) - 1}) {
    a.set_page_size((int32_t)size);
    for (int64_t k = 0; k <= (int64_t(1) << 31) / size; k += 1 + k / 50)
      for (int64_t p : {k * size - 1, k * size, k * size + 1, k * size + size / 2})
        if (p >= 0 && p < int64_t(1) << 31) CHECK(a.page_of((uint32_t)p) == (uint32_t)(p / size));
    for (int64_t p = (int64_t(1) << 31) - 1; p > (int64_t(1) << 31) - 3000; p--) CHECK(a.page_of((uint32_t)p) == (uint32_t)(p / size));
  }
}

static void test_moves() {
  int32_t* i = fake<int32_t>();
  void* p = fake();
  auto compact = [&](const mxfp4_cache_dims& d, const int32_t* path, int64_t ldp, int32_t cols, const int32_t* t, int64_t ld, int32_t n,
                     int32_t pages, void* kq, void* vs) {
    return mxfp4_cache_compact(&d, i, path, ldp, cols, t, ld, n, pages, i, kq, p, p, vs, nullptr);
  };
  g_launches = 0;
  CHECK(compact(kOk, i, 3, 4, i, 4, 2, 4, p, p) == MXFP4_ERR_SHAPE);
  CHECK(compact(kOk, i, 4, -1, i, 4, 2, 4, p, p) == MXFP4_ERR_SHAPE);
  CHECK(compact(kOk, i, 4, 4, i, 3, 2, 4, p, p) == MXFP4_ERR_SHAPE);
  CHECK(compact(kOk, i, 4, 4, i, 4, -1, 4, p, p) == MXFP4_ERR_SHAPE);
  CHECK(compact(kOk, nullptr, 4, 4, i, 4, 2, 4, p, p) == MXFP4_ERR_NULL);
  CHECK(compact(kOk, i, 4, 4, nullptr, 4, 2, 4, p, p) == MXFP4_ERR_NULL);
  CHECK(compact(kOk, i, 4, 4, i, 4, 2, 4, nullptr, p) == MXFP4_ERR_NULL);
  CHECK(compact(kOk, i, 4, 4, i, 4, 2, 4, p, nullptr) == MXFP4_ERR_NULL);
  CHECK(compact(kOk, i, 4, 4, i, 4, 2, 4, fake(4), p) == MXFP4_ERR_ALIGN);
  CHECK(compact(kOk, fake<int32_t>(1), 4, 4, i, 4, 2, 4, p, p) == MXFP4_ERR_ALIGN);
  mxfp4_cache_dims bad = kOk;
  bad.page_size = 0;
  CHECK(compact(bad, i, 4, 4, i, 4, 2, 4, p, p) == MXFP4_ERR_SHAPE);
  CHECK(compact(kOk, i, 4, 4, i, 4, 0, 4, p, p) == MXFP4_OK && g_launches == 0);
  CHECK(compact(kOk, i, 4, 4, i, 4, 2, 4, p, p) == MXFP4_OK && g_launches == 1 && g_move.planes == 4);
  // bytes of a token, and the units that its rows are aligned to
  CHECK(g_move.plane[0].row == 128 && g_move.plane[1].row == 4 && g_move.plane[2].row == 192 && g_move.plane[3].row == 6);
  CHECK(g_move.plane[0].unit == 16 && g_move.plane[1].unit == 4 && g_move.plane[2].unit == 16 && g_move.plane[3].unit == 2);
  mxfp4_cache_dims one = {MXFP4_FMT_NVFP4, 1, 16, 0, 4, 10, 0.0f, 0.0f};  // moved as they are: global scales play no part
  CHECK(compact(one, i, 4, 4, i, 4, 2, 4, p, nullptr) == MXFP4_ERR_SHAPE);  // though a cache has them
  one.k_global_scale = 1.0f;
  CHECK(compact(one, i, 4, 4, i, 4, 2, 4, fake(8), nullptr) == MXFP4_OK && g_move.planes == 2);
  CHECK(g_move.plane[0].row == 8 && g_move.plane[0].unit == 8 && g_move.plane[1].row == 1 && g_move.plane[1].unit == 1);
  CHECK(mxfp4_cache_compact(&kOk, nullptr, nullptr, 0, 0, nullptr, 0, 2, 0, nullptr, p, fake(1), p, p, nullptr) == MXFP4_OK &&
        g_move.plane[1].unit == 1);
  g_launches = 0;
  auto copy = [&](const int32_t* s, const int32_t* d, const int32_t* r, int32_t n, void* kq) {
    return mxfp4_cache_copy_pages(&kOk, s, d, r, n, kq, p, p, p, nullptr);
  };
  CHECK(copy(i, i, i, -1, p) == MXFP4_ERR_SHAPE && copy(nullptr, i, i, 2, p) == MXFP4_ERR_NULL);
  CHECK(copy(i, nullptr, i, 2, p) == MXFP4_ERR_NULL && copy(i, i, i, 2, nullptr) == MXFP4_ERR_NULL);
  CHECK(copy(i, i, fake<int32_t>(2), 2, p) == MXFP4_ERR_ALIGN && copy(nullptr, nullptr, nullptr, 0, p) == MXFP4_OK);
  CHECK(g_launches == 0 && copy(i, i, nullptr, 2, p) == MXFP4_OK && g_launches == 1 && !g_move.rows);
}

static void test_pool() {
  int32_t* i = fake<int32_t>();
  g_launches = 0;
  CHECK(mxfp4_pool_workspace_bytes(-1, 4, 4) == 0 && mxfp4_pool_workspace_bytes(4, -1, 4) == 0);
  CHECK(mxfp4_pool_workspace_bytes(int64_t(1) << 31, 4, 4) == 0 && mxfp4_pool_workspace_bytes(4, 1 << 16, 1 << 15) == 0);
  CHECK(mxfp4_pool_workspace_bytes(4, (1 << 24) + 1, 1) == 0);
  auto resize = [&](int64_t pages, int32_t page, int32_t* refs, int32_t* t, int64_t ld, int32_t rows, int32_t cols, const int32_t* len,
                    int32_t* copies, int32_t* missing, void* ws, size_t n) {
    return mxfp4_pool_resize(pages, page, refs, t, ld, rows, cols, len, copies, missing, ws, n, nullptr);
  };
  const size_t n = mxfp4_pool_workspace_bytes(100, 8, 20);
  CHECK(n > 0);
  CHECK(resize(100, 0, i, i, 20, 8, 20, i, i, i, fake(), n) == MXFP4_ERR_SHAPE);
  CHECK(resize(100, 4, i, i, 19, 8, 20, i, i, i, fake(), n) == MXFP4_ERR_SHAPE);
  CHECK(resize(-1, 4, i, i, 20, 8, 20, i, i, i, fake(), n) == MXFP4_ERR_SHAPE);
  CHECK(resize(100, 4, i, i, 20, -8, 20, i, i, i, fake(), n) == MXFP4_ERR_SHAPE);
  CHECK(resize(100, 4, nullptr, i, 20, 8, 20, i, i, i, fake(), n) == MXFP4_ERR_NULL);
  CHECK(resize(100, 4, i, nullptr, 20, 8, 20, i, i, i, fake(), n) == MXFP4_ERR_NULL);
  CHECK(resize(100, 4, i, i, 20, 8, 20, nullptr, i, i, fake(), n) == MXFP4_ERR_NULL);
  CHECK(resize(100, 4, i, i, 20, 8, 20, i, nullptr, i, fake(), n) == MXFP4_ERR_NULL);
  CHECK(resize(100, 4, i, i, 20, 8, 20, i, i, nullptr, fake(), n) == MXFP4_ERR_NULL);
  CHECK(resize(100, 4, i, i, 20, 8, 20, i, i, i, nullptr, n) == MXFP4_ERR_NULL);
  CHECK(resize(100, 4, fake<int32_t>(2), i, 20, 8, 20, i, i, i, fake(), n) == MXFP4_ERR_ALIGN);
  CHECK(resize(100, 4, i, i, 20, 8, 20, i, i, i, fake(16), n) == MXFP4_ERR_ALIGN);
  CHECK(resize(100, 4, i, i, 20, 8, 20, i, i, i, fake(), n - 1) == MXFP4_ERR_WORKSPACE);
  CHECK(g_launches == 0 && resize(100, 4, i, i, 20, 8, 20, i, i, i, fake(), n) == MXFP4_OK && g_launches == 1 && g_pool.n == 8);
  CHECK(g_pool_ws.need + 32 <= g_pool_ws.first && g_pool_ws.first + 32 <= g_pool_ws.from && g_pool_ws.from + 32 <= g_pool_ws.offset);
  CHECK(g_pool_ws.offset + 36 <= g_pool_ws.list && g_pool_ws.list + 400 <= g_pool_ws.total);
  CHECK(resize(0, 4, nullptr, nullptr, 0, 0, 0, nullptr, nullptr, i, fake(), 256) == MXFP4_OK);
  const size_t nf = mxfp4_pool_workspace_bytes(100, 3, 20);
  auto fork = [&](const int32_t* s, const int32_t* d, const int32_t* l, int32_t pairs) {
    return mxfp4_pool_fork(100, 4, i, i, 20, 8, 20, s, d, l, pairs, i, i, fake(), nf, nullptr);
  };
  g_launches = 0;
  CHECK(fork(nullptr, i, i, 3) == MXFP4_ERR_NULL && fork(i, nullptr, i, 3) == MXFP4_ERR_NULL && fork(i, i, nullptr, 3) == MXFP4_ERR_NULL);
  CHECK(fork(i, i, i, -1) == MXFP4_ERR_SHAPE && fork(i, i, i, 65537) == MXFP4_ERR_SHAPE);
  CHECK(fork(i, fake<int32_t>(1), i, 3) == MXFP4_ERR_ALIGN && g_launches == 0);
  CHECK(fork(i, i, i, 3) == MXFP4_OK && g_pool.n == 3 && g_pool.n_rows == 8 && fork(nullptr, nullptr, nullptr, 0) == MXFP4_OK);
}

static void test_rotary() {
  double* turns = fake<double>();
  int32_t* pos = fake<int32_t>();
  struct Call {
    int32_t dim = 64, rot = 32, offset = 16, inter = 0, inverse = 0, fp32 = 0, qh = 4, kh = 2;
    int64_t rows = 3, q_ldt = 256, q_ldh = 64, o_ldt = 256, o_ldh = 64, k_ldt = 128;
    void *q = fake(), *qo = fake(), *k = fake(), *ko = fake();
    float mag = 1.0f;
  };
  auto with = [&](auto f) {
    Call c;
    f(c);
    return mxfp4_rotary(turns, pos, c.rows, c.dim, c.rot, c.offset, c.inter, c.mag, c.inverse, c.fp32, c.q, c.q_ldt, c.q_ldh, c.qh, c.qo,
                        c.o_ldt, c.o_ldh, c.k, c.k_ldt, 64, c.kh, c.ko, 128, 64, nullptr);
  };
  g_launches = 0;
  CHECK(with([](Call& c) { c.rot = 31; }) == MXFP4_ERR_SHAPE && with([](Call& c) { c.rot = 0; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.offset = 33; }) == MXFP4_ERR_SHAPE && with([](Call& c) { c.offset = -1; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.offset = INT_MAX; }) == MXFP4_ERR_SHAPE && with([](Call& c) { c.dim = 0; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.inter = 2; }) == MXFP4_ERR_SHAPE && with([](Call& c) { c.mag = NAN; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.qh = 0; }) == MXFP4_ERR_SHAPE && with([](Call& c) { c.qh = 1 << 15; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.kh = 0; }) == MXFP4_ERR_SHAPE && with([](Call& c) { c.rows = -1; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.q_ldt = -8; }) == MXFP4_ERR_SHAPE && with([](Call& c) { c.o_ldt = 63; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.o_ldh = 32; }) == MXFP4_ERR_SHAPE && with([](Call& c) { c.k_ldt = int64_t(1) << 41; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](Call& c) { c.q = nullptr; }) == MXFP4_ERR_NULL && with([](Call& c) { c.qo = nullptr; }) == MXFP4_ERR_NULL);
  CHECK(with([](Call& c) { c.ko = nullptr; }) == MXFP4_ERR_NULL);
  CHECK(with([](Call& c) { c.q = fake(1); }) == MXFP4_ERR_ALIGN && with([](Call& c) { c.ko = fake(2); c.fp32 = 1; }) == MXFP4_ERR_ALIGN);
  CHECK(with([](Call& c) { c.rows = 0; }) == MXFP4_OK && g_launches == 0);
  CHECK(with([](Call&) {}) == MXFP4_OK && g_rot.x[0].heads == 4 && g_rot.x[1].heads == 2 && g_rot.sign == 1.0f);
  CHECK(with([](Call& c) { c.k = nullptr; c.inverse = 1; }) == MXFP4_OK && g_rot.x[1].heads == 0 && g_rot.sign == -1.0f);
  CHECK(with([](Call& c) { c.q_ldt = c.q_ldh = 0; }) == MXFP4_OK);  // a broadcast input
  CHECK(with([](Call& c) { c.dim = 1 << 16; c.rot = 2048; c.qh = c.kh = 1; c.o_ldt = 1 << 16; c.rows = 1; }) == MXFP4_OK);
}

int main() {
  test_attend();
  test_page_of();
  test_moves();
  test_pool();
  test_rotary();
  if (g_fail) {
    std::printf("%d checks failed\n", g_fail);
    return 1;
  }
  std::printf("draft checks passed\n");
  return 0;
}
