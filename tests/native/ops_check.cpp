// Calls the entry points of csrc/ops_api.cpp on the CPU with valid and invalid arguments (the kernel
// launchers are stand-ins that record what they were given) and walks the paged cache's slot arithmetic over
// good and bad page tables.  Built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_ops_abi.py; the arrays are exactly as long as the calls say, so a read past them is reported.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../../mixed_precision_moe_amd/csrc/cache_slots.h"

static int g_fail = 0, g_launches = 0;
static MatvecArgs g_mv;
static CacheArgs g_cache;
static BalanceWs g_bws;
#define CHECK(c)                                               \
  do {                                                         \
    if (!(c)) {                                                \
      std::printf("FAIL %s:%d: %s\n", __FILE__, __LINE__, #c); \
      g_fail++;                                                \
    }                                                          \
  } while (0)

int32_t balance_blocks(int64_t T, int32_t E) { return T * E < 1000 ? 1 : (int32_t)(T < 512 ? T : 512); }
int launch_balance_forward(const BalanceArgs&, const BalanceWs& w, uint8_t*, hipStream_t) {
  g_launches++;
  g_bws = w;
  return MXFP4_OK;
}
int launch_balance_backward(const float*, int64_t, int32_t, int64_t, const uint8_t*, const float*, const float*, float*,
                            hipStream_t) {
  g_launches++;
  return MXFP4_OK;
}
int launch_matvec(int, const MatvecArgs& a, hipStream_t) {
  g_launches++;
  g_mv = a;
  return MXFP4_OK;
}
int launch_cache_write(int, const CacheArgs& a, hipStream_t) {
  g_launches++;
  g_cache = a;
  return MXFP4_OK;
}
int launch_cache_read(int, const CacheArgs& a, hipStream_t) {
  g_launches++;
  g_cache = a;
  return MXFP4_OK;
}

template <typename T = void>
static T* fake(uintptr_t off = 0) { return (T*)((uintptr_t(1) << 32) + off); }

static void test_balance() {
  float* f = fake<float>();
  int32_t* i = fake<int32_t>();
  const size_t n = moe_balance_workspace_bytes(100, 64);
  CHECK(n > 0);
  CHECK(moe_balance_workspace_bytes(-1, 64) == 0 && moe_balance_workspace_bytes(4, 1025) == 0);
  CHECK(moe_balance_workspace_bytes(INT64_MAX, 64) == 0 && moe_balance_workspace_bytes(0, 1) > 0);
  auto fw = [&](const float* l, int64_t T, int32_t E, int64_t ld, const int32_t* ids, int32_t k, float* loss, void* ws,
                size_t nws) { return moe_balance_forward(l, T, E, ld, ids, k, nullptr, loss, i, f, ws, nws, nullptr); };
  CHECK(fw(f, 100, 64, 63, i, 2, f, fake(), n) == MXFP4_ERR_SHAPE);
  CHECK(fw(f, 100, 64, 64, i, 0, f, fake(), n) == MXFP4_ERR_SHAPE);
  CHECK(fw(f, 100, 64, 64, i, 33, f, fake(), n) == MXFP4_ERR_SHAPE);
  CHECK(fw(f, 100, 4, 64, i, 5, f, fake(), n) == MXFP4_ERR_SHAPE);
  CHECK(fw(f, int64_t(1) << 30, 64, 64, i, 2, f, fake(), n) == MXFP4_ERR_SHAPE);
  CHECK(fw(nullptr, 100, 64, 64, i, 2, f, fake(), n) == MXFP4_ERR_NULL);
  CHECK(fw(f, 100, 64, 64, nullptr, 2, f, fake(), n) == MXFP4_ERR_NULL);
  CHECK(fw(f, 100, 64, 64, i, 2, nullptr, fake(), n) == MXFP4_ERR_NULL);
  CHECK(fw(f, 100, 64, 64, i, 2, f, nullptr, n) == MXFP4_ERR_NULL);
  CHECK(fw(fake<float>(2), 100, 64, 64, i, 2, f, fake(), n) == MXFP4_ERR_ALIGN);
  CHECK(fw(f, 100, 64, 64, i, 2, f, fake(64), n) == MXFP4_ERR_ALIGN);
  CHECK(fw(f, 100, 64, 64, i, 2, f, fake(), n - 1) == MXFP4_ERR_WORKSPACE);
  CHECK(g_launches == 0);
  CHECK(fw(f, 100, 64, 70, i, 2, f, fake(), n) == MXFP4_OK && g_launches == 1);
  // the workspace's parts follow each other inside it
  CHECK(g_bws.parts + 8 * (uint64_t)g_bws.blocks * 64 <= g_bws.part_v);
  CHECK(g_bws.part_v + 4 * (uint64_t)g_bws.blocks <= g_bws.sums && g_bws.sums + 8 * 64 <= g_bws.ticket);
  CHECK(g_bws.ticket + 4 <= g_bws.total && g_bws.total == n && g_bws.sums % 8 == 0);
  // no tokens: loss and counts are still written
  CHECK(fw(nullptr, 0, 64, 64, nullptr, 2, f, fake(), n) == MXFP4_OK && g_launches == 2);
  CHECK(moe_balance_backward(f, 10, 64, 64, nullptr, nullptr, f, f, nullptr) == MXFP4_ERR_NULL);
  CHECK(moe_balance_backward(f, 10, 64, 64, nullptr, f, nullptr, f, nullptr) == MXFP4_ERR_NULL);
  CHECK(moe_balance_backward(f, 10, 64, 60, nullptr, f, f, f, nullptr) == MXFP4_ERR_SHAPE);
  CHECK(moe_balance_backward(f, 10, 64, 64, nullptr, f, f, fake<float>(1), nullptr) == MXFP4_ERR_ALIGN);
  CHECK(g_launches == 2);
  CHECK(moe_balance_backward(nullptr, 0, 64, 64, nullptr, nullptr, nullptr, nullptr, nullptr) == MXFP4_OK);
  CHECK(g_launches == 2);
  CHECK(moe_balance_backward(f, 10, 64, 64, nullptr, f, f, f, nullptr) == MXFP4_OK && g_launches == 3);
}

static void test_matvec() {
  g_launches = 0;
  auto mv = [](int fmt, const void* q, const void* s, float gs, int64_t N, int64_t K, const void* x, int64_t M,
               int64_t ldx, void* y, int64_t ldy, int32_t o = 0) {
    return fp4_matvec(fmt, q, s, gs, N, K, nullptr, 0, x, M, ldx, y, ldy, o, nullptr);
  };
  void* p = fake();
  CHECK(mv(2, p, p, 1, 16, 64, p, 1, 64, p, 16) == MXFP4_ERR_LAYOUT);
  CHECK(mv(7, p, p, 1, 16, 64, p, 1, 64, p, 16) == MXFP4_ERR_LAYOUT);
  CHECK(mv(0, p, p, 1, 16, 48, p, 1, 64, p, 16) == MXFP4_ERR_SHAPE);  // K % 32
  CHECK(mv(1, p, p, 1, 16, 40, p, 1, 64, p, 16) == MXFP4_ERR_SHAPE);  // K % 16
  CHECK(mv(1, p, p, 1, 16, 16, p, 1, 64, p, 16) == MXFP4_ERR_SHAPE);  // K < 32
  CHECK(mv(0, p, p, 1, 0, 64, p, 1, 64, p, 16) == MXFP4_ERR_SHAPE);
  CHECK(mv(0, p, p, 1, 16, 0, p, 1, 64, p, 16) == MXFP4_ERR_SHAPE);
  CHECK(mv(0, p, p, 1, (1 << 20) + 1, 64, p, 1, 64, p, 1 << 21) == MXFP4_ERR_SHAPE);
  CHECK(mv(0, p, p, 1, 16, 64, p, -1, 64, p, 16) == MXFP4_ERR_SHAPE);
  CHECK(mv(0, p, p, 1, 16, 64, p, 1, 56, p, 16) == MXFP4_ERR_SHAPE);
  CHECK(mv(0, p, p, 1, 16, 64, p, 1, 68, p, 16) == MXFP4_ERR_SHAPE);
  CHECK(mv(0, p, p, 1, 16, 64, p, 1, 64, p, 15) == MXFP4_ERR_SHAPE);
  CHECK(mv(0, p, p, 1, 16, 64, p, 1, 64, p, 16, 2) == MXFP4_ERR_SHAPE);
  CHECK(mv(1, p, p, 0.0f, 16, 64, p, 1, 64, p, 16) == MXFP4_ERR_SHAPE);
  CHECK(mv(1, p, p, NAN, 16, 64, p, 1, 64, p, 16) == MXFP4_ERR_SHAPE);
  CHECK(mv(1, p, p, INFINITY, 16, 64, p, 1, 64, p, 16) == MXFP4_ERR_SHAPE);
  CHECK(mv(0, nullptr, p, 1, 16, 64, p, 1, 64, p, 16) == MXFP4_ERR_NULL);
  CHECK(mv(0, p, nullptr, 1, 16, 64, p, 1, 64, p, 16) == MXFP4_ERR_NULL);
  CHECK(mv(0, p, p, 1, 16, 64, nullptr, 1, 64, p, 16) == MXFP4_ERR_NULL);
  CHECK(mv(0, p, p, 1, 16, 64, p, 1, 64, nullptr, 16) == MXFP4_ERR_NULL);
  CHECK(mv(0, fake(8), p, 1, 16, 64, p, 1, 64, p, 16) == MXFP4_ERR_ALIGN);
  CHECK(mv(0, p, p, 1, 16, 64, fake(8), 1, 64, p, 16) == MXFP4_ERR_ALIGN);
  CHECK(mv(0, p, p, 1, 16, 64, p, 1, 64, fake(1), 16) == MXFP4_ERR_ALIGN);
  CHECK(mv(0, p, p, 1, 16, 64, p, 1, 64, fake(2), 16, 1) == MXFP4_ERR_ALIGN);
  CHECK(g_launches == 0);
  CHECK(mv(0, nullptr, nullptr, 1, 16, 64, nullptr, 0, 64, nullptr, 16) == MXFP4_OK && g_launches == 0);
  CHECK(mv(0, p, fake(3), NAN, 17, 64, p, 5, 72, fake(2), 17) == MXFP4_OK && g_launches == 1);
  CHECK(g_mv.gscale == 1.0f && g_mv.E == 1 && g_mv.M == 5 && !g_mv.offsets);

  const float* gs = fake<float>();
  const int32_t* ix = fake<int32_t>();
  auto ex = [&](int fmt, const float* g, int32_t E, int64_t N, int64_t K, int64_t ldx, int32_t k, const int32_t* off,
                const int32_t* pairs, int64_t P, int32_t sw) {
    return fp4_expert_matvec(fmt, p, p, g, E, N, K, nullptr, 0, p, ldx, k, off, pairs, P, sw, p, 0, nullptr);
  };
  CHECK(ex(0, nullptr, 0, 16, 64, 64, 2, ix, ix, 8, 0) == MXFP4_ERR_SHAPE);
  CHECK(ex(0, nullptr, 1025, 16, 64, 64, 2, ix, ix, 8, 0) == MXFP4_ERR_SHAPE);
  CHECK(ex(0, nullptr, 4, 15, 64, 64, 2, ix, ix, 8, 1) == MXFP4_ERR_SHAPE);   // swiglu: even N
  CHECK(ex(0, nullptr, 4, 16, 64, 64, 3, ix, ix, 8, 0) == MXFP4_ERR_SHAPE);   // P % top_k
  CHECK(ex(0, nullptr, 4, 16, 64, 64, 0, ix, ix, 8, 0) == MXFP4_ERR_SHAPE);
  CHECK(ex(0, nullptr, 4, 16, 64, 64, 2, ix, ix, -2, 0) == MXFP4_ERR_SHAPE);
  CHECK(ex(0, nullptr, 4, 16, 64, 64, 2, ix, ix, int64_t(1) << 31, 0) == MXFP4_ERR_SHAPE);
  CHECK(ex(0, nullptr, 4, 16, 64, 64, 2, nullptr, ix, 8, 0) == MXFP4_ERR_NULL);
  CHECK(ex(0, nullptr, 4, 16, 64, 64, 2, ix, nullptr, 8, 0) == MXFP4_ERR_NULL);
  CHECK(ex(1, nullptr, 4, 16, 64, 64, 2, ix, ix, 8, 0) == MXFP4_ERR_NULL);
  CHECK(ex(1, fake<float>(2), 4, 16, 64, 64, 2, ix, ix, 8, 0) == MXFP4_ERR_ALIGN);
  CHECK(ex(0, nullptr, 4, 16, 64, 64, 2, fake<int32_t>(1), ix, 8, 0) == MXFP4_ERR_ALIGN);
  CHECK(g_launches == 1);
  CHECK(ex(0, nullptr, 4, 16, 64, 64, 2, nullptr, nullptr, 0, 0) == MXFP4_OK && g_launches == 1);
  CHECK(ex(1, gs, 4, 16, 48, 48, 2, ix, ix, 8, 1) == MXFP4_OK && g_launches == 2);
  CHECK(g_mv.ldy == 8 && g_mv.gscales == gs && g_mv.M == 8);
}

static void test_cache() {
  g_launches = 0;
  void* p = fake();
  const int32_t* ix = fake<int32_t>();
  auto wr = [&](mxfp4_cache_dims d, int64_t rows, int64_t kt, int64_t kh, int64_t ldt, int32_t B, int32_t mp,
                const void* k, const void* v, const int32_t* cu, void* kq, void* vq) {
    return mxfp4_cache_write(&d, k, kt, kh, v, 512, 128, rows, cu, nullptr, ix, ldt, B, mp, kq, p, vq, p, nullptr);
  };
  const mxfp4_cache_dims ok = {MXFP4_FMT_MXFP4, 4, 64, 128, 16, 100, 1.0f, 1.0f};
  auto with = [&](auto f) { mxfp4_cache_dims d = ok; f(d); return wr(d, 8, 256, 64, 10, 2, 10, p, p, ix, p, p); };
  CHECK(with([](auto& d) { d.fmt = 3; }) == MXFP4_ERR_LAYOUT);
  CHECK(with([](auto& d) { d.heads = 0; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.k_dim = 48; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.k_dim = 0; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.v_dim = 16; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.v_dim = -32; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.page_size = 0; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.num_pages = -1; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.num_pages = INT64_MAX; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.num_pages = int64_t(1) << 31; d.page_size = INT32_MAX; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.heads = INT32_MAX; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.fmt = MXFP4_FMT_NVFP4; d.k_global_scale = 0; }) == MXFP4_ERR_SHAPE);
  CHECK(with([](auto& d) { d.fmt = MXFP4_FMT_NVFP4; d.v_global_scale = NAN; }) == MXFP4_ERR_SHAPE);
  CHECK(wr(ok, -1, 256, 64, 10, 2, 10, p, p, ix, p, p) == MXFP4_ERR_SHAPE);
  CHECK(wr(ok, 8, 248, 32, 10, 2, 10, p, p, ix, p, p) == MXFP4_ERR_SHAPE);  // heads overlap
  CHECK(wr(ok, 8, 252, 64, 10, 2, 10, p, p, ix, p, p) == MXFP4_ERR_SHAPE);  // ldt % 8
  CHECK(wr(ok, 8, 256, 64, 9, 2, 10, p, p, ix, p, p) == MXFP4_ERR_SHAPE);   // ld_table < max_pages
  CHECK(wr(ok, 8, 256, 64, 10, -1, 10, p, p, ix, p, p) == MXFP4_ERR_SHAPE);
  CHECK(wr(ok, 8, 256, 64, 10, 2, 10, nullptr, p, ix, p, p) == MXFP4_ERR_NULL);
  CHECK(wr(ok, 8, 256, 64, 10, 2, 10, p, nullptr, ix, p, p) == MXFP4_ERR_NULL);
  CHECK(wr(ok, 8, 256, 64, 10, 2, 10, p, p, nullptr, p, p) == MXFP4_ERR_NULL);
  CHECK(wr(ok, 8, 256, 64, 10, 2, 10, p, p, ix, nullptr, p) == MXFP4_ERR_NULL);
  CHECK(wr(ok, 8, 256, 64, 10, 2, 10, p, p, ix, p, nullptr) == MXFP4_ERR_NULL);
  CHECK(wr(ok, 8, 256, 64, 10, 2, 10, fake(8), p, ix, p, p) == MXFP4_ERR_ALIGN);
  CHECK(wr(ok, 8, 256, 64, 10, 2, 10, p, p, ix, fake(4), p) == MXFP4_ERR_ALIGN);
  CHECK(mxfp4_cache_write(nullptr, p, 256, 64, p, 512, 128, 8, ix, ix, ix, 10, 2, 10, p, p, p, p, nullptr) ==
        MXFP4_ERR_NULL);
  CHECK(g_launches == 0);
  CHECK(wr(ok, 0, 256, 64, 10, 2, 10, nullptr, nullptr, nullptr, nullptr, nullptr) == MXFP4_OK && g_launches == 0);
  CHECK(wr(ok, 8, 256, 64, 10, 0, 10, nullptr, nullptr, nullptr, nullptr, nullptr) == MXFP4_OK && g_launches == 0);
  CHECK(wr(ok, 8, 256, 64, 10, 2, 10, p, p, ix, p, p) == MXFP4_OK && g_launches == 1);
  CHECK(g_cache.plane[1].dim == 128 && g_cache.heads == 4);
  mxfp4_cache_dims none = ok;
  none.num_pages = 0;
  CHECK(wr(none, 8, 256, 64, 10, 2, 10, p, p, ix, nullptr, nullptr) == MXFP4_OK && g_launches == 2);
  CHECK(mxfp4_cache_write(&ok, p, 256, 64, p, 512, 128, 8, ix, nullptr, nullptr, 0, 2, 0, p, p, p, p, nullptr) == MXFP4_OK);
  CHECK(mxfp4_cache_write(&ok, p, 256, 64, p, 512, 128, 8, ix, nullptr, nullptr, 1, 2, 1, p, p, p, p, nullptr) ==
        MXFP4_ERR_NULL);
  mxfp4_cache_dims one = ok;
  one.v_dim = 0;
  CHECK(wr(one, 8, 256, 64, 10, 2, 10, p, nullptr, ix, p, nullptr) == MXFP4_OK && g_cache.plane[1].dim == 0);
  size_t b[4];
  CHECK(mxfp4_cache_bytes(&ok, b) == MXFP4_OK);
  CHECK(b[0] == 1600u * 4 * 32 && b[1] == 1600u * 4 * 2 && b[2] == 1600u * 4 * 64 && b[3] == 1600u * 4 * 4);
  CHECK(mxfp4_cache_bytes(&one, b) == MXFP4_OK && b[2] == 0 && b[3] == 0);
  CHECK(mxfp4_cache_bytes(&ok, nullptr) == MXFP4_ERR_NULL && mxfp4_cache_bytes(nullptr, b) == MXFP4_ERR_NULL);
}

// Every slot lies in the cache, whatever the table and the sequences hold; good ones follow the definition.
static void test_slots() {
  std::mt19937 r(7);
  for (int trial = 0; trial < 4000; trial++) {
    const int B = 1 + r() % 5, mp = r() % 4, ld = mp + r() % 3, page = 1 + r() % 5;
    const int64_t pages = r() % 6;
    const bool bad = trial % 2;
    std::vector<int32_t> cu(B + 1), start(B), table((size_t)(B - 1) * ld + mp);
    int at = r() % 3;
    for (int i = 0; i <= B; i++) {
      cu[i] = at;
      at += r() % 7;
    }
    for (auto& s : start) s = bad ? (int32_t)(r() % 41) - 20 : (int32_t)(r() % 4);
    for (auto& t : table) t = bad ? (int32_t)r() : (int32_t)(r() % (pages + 1)) - 1;
    if (bad && trial % 3 == 0) cu[r() % (B + 1)] = (int32_t)r();  // not even increasing
    if (bad && trial % 5 == 0) start[r() % B] = r() % 2 ? INT32_MAX : INT32_MIN;
    CacheArgs a = {};
    a.rows = 40;
    a.num_pages = pages;
    a.ld_table = ld;
    a.cu = cu.data();
    a.start = trial % 7 ? start.data() : nullptr;
    a.table = table.data();
    a.n_seqs = B;
    a.max_pages = mp;
    a.page_size = page;
    for (int64_t t = 0; t < a.rows; t++) {
      const int64_t s = slot_of(a, t);
      CHECK(s >= -2 && s < pages * page);
      if (bad) continue;
      int64_t want = -2;
      for (int b = 0; b < B; b++)
        if (t >= cu[b] && t < cu[b + 1]) {
          const int64_t pos = t - cu[b] + (a.start ? start[b] : 0);
          want = -1;
          if (pos / page < mp) {
            const int32_t g = table[(size_t)b * ld + pos / page];
            if (g >= 0 && g < pages) want = g * page + pos % page;
          }
        }
      CHECK(s == want);
    }
  }
}

int main() {
  test_balance();
  test_matvec();
  test_cache();
  test_slots();
  if (g_fail) {
    std::printf("%d checks failed\n", g_fail);
    return 1;
  }
  std::printf("ops checks passed\n");
  return 0;
}
