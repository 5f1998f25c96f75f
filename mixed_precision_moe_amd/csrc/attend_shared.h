// Attention for many rows a key head: a worker's waves share tiles of K and V, dequantized into LDS.
//
// A worker takes 16 NT WR rows, W waves: WR of them with 16 NT rows each, in W / WR groups that have each their part of a
// tile's positions.  Per tile every thread dequantizes its pieces of 16 bytes of codes, so that is paid once for all rows, and
// codes leave the caches once for all of them.  Two tiles of K and V are in LDS: while one is worked on, the codes of the next
// are on their way to registers, and they are dequantized into the other behind it, with one barrier a tile.  Pages are
// looked up four tiles ahead, and made addresses three tiles ahead.
//
// Bound, where rows are many, by the matrix cores beside the exponentials and conversions: two waves a matrix core overlap them
// in part.  By LDS too (what a wave reads it uses for 16 NT rows: 32 took 66 us where 16, with twice the waves, took 92),
// so NT is 2 where the registers of two waves hold it, and 1 for more than 128 elements (256: 726 us against 1427 with two
// column tiles and one wave).  4 sequences of 1024 rows of 8 query heads on each of 4 key heads, 4096 positions before them,
// with the join: MXFP8 905 TFLOP/s (128 elements), 845 (256), MXFP4 935, 801 and 1020 (192 and 128), NVFP4 877, 768 and 945.
// Few rows and long contexts by what a worker does once: 12 sequences of up to 264 rows a key head (208 on average) and up to
// 5000 positions (3754) took 65 us, 23 of them for finding and loading what comes first.
#pragma once

#include "attend_common.h"

namespace {

constexpr int KEYS = kAttendKeys;  // a lane each where they are looked up
static_assert(KEYS == 64, "the lanes of a wave");

template <int FMT, int DK, int DV, int NT, int W, int WR>
struct Shared {
  static constexpr int kThreads = 64 * W;
  static constexpr int kWK = W / WR;           // groups of waves that share the positions
  static constexpr int kRows = 16 * NT * WR;
  static constexpr int kKT = KEYS / kWK / 16;   // tiles of 16 positions of a wave
  static constexpr int kElems = 16 * kPerByte<FMT>;
  static constexpr int kScales = kElems / kBlock<FMT> ? kElems / kBlock<FMT> : 1;
  static constexpr int kStrideK = DK + 16, kStrideV = DV + 16;  // rows 32 bytes on: eight of them meet no bank twice
  static constexpr int kTileBytes = 2 * KEYS * (kStrideK + kStrideV);
};

// A thread's pieces of a plane's tile.
template <int FMT, int D, int kThreads>
struct Pieces {
  static constexpr int kElems = 16 * kPerByte<FMT>, kPerKey = D / kElems, kAll = KEYS * kPerKey;
  static constexpr int kN = (kAll + kThreads - 1) / kThreads;
  static constexpr int kScales = kElems / kBlock<FMT> ? kElems / kBlock<FMT> : 1;
  u32x4_t codes[kN];
  uint32_t scales[kN];  // a byte a block

  // vectors: the cache's vector of each position, -1: none
  MX_DEV void load(const CachePlane& p, const int64_t* vectors) {
    const int64_t bytes = p.dim / kPerByte<FMT>;
    const int blocks = p.dim / kBlock<FMT>;
#pragma unroll
    for (int i = 0; i < kN; i++) {
      const int id = i * kThreads + threadIdx.x, key = id / kPerKey, piece = id % kPerKey, e = piece * kElems;
      codes[i] = u32x4_t{0, 0, 0, 0};
      scales[i] = 0;
      const int64_t at = kAll % kThreads && id >= kAll ? -1 : vectors[key];
      if (at < 0 || e >= p.dim) continue;
      const uint8_t* src = p.q + at * bytes + 16 * piece;
      const uint8_t* s = p.s + at * blocks + e / kBlock<FMT>;
      if (kScales == 1) {
        codes[i] = *reinterpret_cast<const u32x4_a8*>(src);
        scales[i] = s[0];
      } else if (e + kElems <= p.dim) {
        codes[i] = *reinterpret_cast<const u32x4_a8*>(src);
        scales[i] = *reinterpret_cast<const u16_a1*>(s);
      } else {  // the last block of an odd number
        const u32x2_t x = *reinterpret_cast<const u32x2_a8*>(src);
        codes[i][0] = x[0];
        codes[i][1] = x[1];
        scales[i] = s[0];
      }
    }
  }

  // Dequantized, to rows of LDS.
  MX_DEV void store(uint16_t* dst, int stride) const {
#pragma unroll
    for (int i = 0; i < kN; i++) {
      const int id = i * kThreads + threadIdx.x, key = id / kPerKey, piece = id % kPerKey;
      if (kAll % kThreads && id >= kAll) continue;
      uint16_t* to = dst + key * stride + piece * kElems;
#pragma unroll
      for (int j = 0; j < kElems / 8; j++)
        *reinterpret_cast<bf16x8_t*>(to + 8 * j) = FMT == MXFP4_FMT_MXFP8 ? values8<FMT>(codes[i][2 * j], codes[i][2 * j + 1], scales[i])
                                                                          : values8<FMT>(codes[i][j], 0, scales[i] >> 8 * (8 * j / kBlock<FMT>) & 0xFFu);
    }
  }

  // Positions whose values are not finite become zeros and leave their bit in `bad`.
  MX_DEV void drop_not_finite(uint32_t* bad) {
#pragma unroll
    for (int i = 0; i < kN; i++) {
      const int id = i * kThreads + threadIdx.x, key = id / kPerKey;
      bool x = false;
#pragma unroll
      for (int j = 0; j < kScales; j++) x = x || not_finite<FMT>(scales[i] >> 8 * j & 0xFFu);
      if (FMT == MXFP4_FMT_MXFP8)
        x = x || has_nan_code(codes[i][0]) || has_nan_code(codes[i][1]) || has_nan_code(codes[i][2]) || has_nan_code(codes[i][3]);
      if (!x) continue;
      codes[i] = u32x4_t{0, 0, 0, 0};
      scales[i] = 0;
      atomicOr(&bad[key >> 5], 1u << (key & 31));
    }
  }
};

template <int FMT, int DK, int DV, int NT, int W, int WR, int WAVES, bool FINE>
__global__ __launch_bounds__(64 * W, WAVES) void attend_shared_kernel(AttendArgs given, float* __restrict__ part,
                                                                        float2* __restrict__ part_ml,
                                                                        Open* __restrict__ open, Totals* __restrict__ totals, int workers) {
  using Sh = Shared<FMT, DK, DV, NT, W, WR>;
  constexpr int MT = Sh::kRows, R = 16 * NT, KT = Sh::kKT;
  static_assert(KT % 2 == 0, "32 positions a matrix instruction");
  constexpr int kBytes = 2 * Sh::kTileBytes;
  // the sums take the place of the tiles, as many waves' rows at a time as fit
  constexpr int kFit = kBytes / (R * (DV + 4) * 4), kGroups = kFit >= WR ? WR : kFit >= 4 ? 4 : kFit >= 2 ? 2 : 1;
  static_assert(kFit > 0, "a wave's rows at least");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kBytes];
  __shared__ int64_t vectors[4][KEYS];
  __shared__ uint64_t valid[4];
  __shared__ uint32_t bad[4][2];
  __shared__ float ms[Sh::kWK][MT], ls[Sh::kWK][MT];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, kg = lane >> 4;
  const int wr = wave % WR, wk = wave / WR;
  Work<MT> w;
  if (!w.begin(given, workers, open, totals, lane)) return;
  const float sc = score_scale<FMT>(given);

  for (;;) {
    w.settle();
    const Seq& s = w.s;
    const int32_t k0 = w.k0, k1 = w.k1(), end = w.ti.end;
    const AttendArgs a = arguments();
    // the positions before this one are seen by all of the wave's rows: with a mask the context, else the first row's drafts too
    const int32_t seen = (int32_t)min((int64_t)s.start + (a.mask ? 0 : (uint32_t)(w.ti.tile * MT + R * wr) / (uint32_t)a.group + 1), (int64_t)INT32_MAX);
    Rows<NT, DV / 16, FINE> rows;
    rows.clear();

    // the page of this lane's position of tile k, and that position's vector
    const int32_t* const table = a.cache.table + (int64_t)w.b * a.cache.ld_table;
    const auto look_up = [&](int32_t k) -> int32_t {
      return end > 0 ? table[a.page_of(min((uint32_t)k * KEYS + lane, (uint32_t)end - 1))] : -1;
    };
    const auto find = [&](int32_t k, int32_t page) -> int64_t {
      const CacheArgs& c = a.cache;
      const uint32_t pos = (uint32_t)k * KEYS + lane;
      if (pos >= (uint32_t)end || page < 0 || page >= c.num_pages) return -1;
      const uint32_t at = pos - a.page_of(pos) * (uint32_t)c.page_size;
      return ((int64_t)page * c.page_size + at) * c.heads + w.group;
    };
    const auto note = [&](int32_t k, int64_t vector) {
      vectors[k & 3][lane] = vector;
      const uint64_t there = __ballot(vector >= 0);
      if (lane == 0) valid[k & 3] = there;
    };
    Pieces<FMT, DK, Sh::kThreads> kp;
    Pieces<FMT, DV, Sh::kThreads> vp;
    const auto tile_k = [&](int32_t k) { return (uint16_t*)(lds + (k & 1) * Sh::kTileBytes); };
    const auto tile_v = [&](int32_t k) { return (uint16_t*)(lds + (k & 1) * Sh::kTileBytes) + KEYS * Sh::kStrideK; };
    const auto load = [&](int32_t k) {
      kp.load(a.cache.plane[0], vectors[k & 3]);
      vp.load(a.cache.plane[1], vectors[k & 3]);
    };
    const auto store = [&](int32_t k) {
      // hidden drafts' values must not meet zero weights unless they are numbers
      if ((int64_t)k * KEYS + KEYS > s.start) vp.drop_not_finite(bad[k & 3]);
      kp.store(tile_k(k), Sh::kStrideK);
      vp.store(tile_v(k), Sh::kStrideV);
    };

    if (threadIdx.x < 8) (&bad[0][0])[threadIdx.x] = 0;
    const int32_t first_page = look_up(k0 + min(wave, 2));
    int32_t page = look_up(k0 + 3);
    const auto element = [&](int i) { return 32 * i + 8 * kg; };
    Query<NT, DK / 32> query;
    query.load(a, s, w.ti.tile * MT + R * wr, w.group, element);
    if (wave < 3) note(k0 + wave, find(k0 + wave, first_page));
    __syncthreads();
    load(k0);
    query.finish(a, element);
    const auto& q = query.q;
    const auto& draft = query.draft;
    store(k0);
    if (k0 + 1 < k1) load(k0 + 1);
    __syncthreads();
    for (int32_t k = k0; k < k1; k++) {
      const int32_t base = k * KEYS + 16 * KT * wk;
      const int32_t ahead = look_up(k + 4);
      f32x4_t sv[NT][KT];
      const uint16_t* keys = tile_k(k) + (16 * KT * wk + col) * Sh::kStrideK + 8 * kg;
#pragma unroll
      for (int t = 0; t < KT; t++)
#pragma unroll
        for (int n = 0; n < NT; n++) sv[n][t] = f32x4_t{0, 0, 0, 0};
      __builtin_amdgcn_s_setprio(1);  // the matrix cores' turn, while other waves do the rest
      bf16x8_t x[2][KT];
#pragma unroll
      for (int t = 0; t < KT; t++) x[0][t] = *reinterpret_cast<const bf16x8_t*>(keys + 16 * t * Sh::kStrideK);
#pragma unroll
      for (int i = 0; i < DK / 32; i++) {
        if (i + 1 < DK / 32) {
#pragma unroll
          for (int t = 0; t < KT; t++) x[(i + 1) & 1][t] = *reinterpret_cast<const bf16x8_t*>(keys + 16 * t * Sh::kStrideK + 32 * (i + 1));
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < KT; t++)
#pragma unroll
          for (int n = 0; n < NT; n++) sv[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i & 1][t], q[n][i], sv[n][t], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      constexpr uint64_t kFull = KT == 4 ? ~0ull : ~0u;
      const uint64_t there = valid[k & 3] >> (16 * KT * wk) & kFull;
      const uint64_t b = ((uint64_t)bad[k & 3][1] << 32 | bad[k & 3][0]) >> (16 * KT * wk) & kFull;
      if (__builtin_expect(there != kFull || b != 0 || base + 16 * KT > seen, 0)) hide<NT, KT>(arguments(), s, draft, base, there, b, kg, sv);
      Weights<NT, KT, FINE> p;
      rows.template weights<KT>(sv, sc, p);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int h = 0; h < KT / 2; h++)
        rows.template add_values<4, KT>(tile_v(k) + (16 * KT * wk + 32 * h) * Sh::kStrideV, Sh::kStrideV, p, h, lane);
      __builtin_amdgcn_s_setprio(0);
      // the other tiles' turn
      if (k + 1 < k1) store(k + 1);
      if (wave == 0) note(k + 3, find(k + 3, page));
      page = ahead;
      asm volatile("" : "+v"(page));  // here, and not behind the loads that follow
      if (k + 2 < k1) load(k + 2);
      if (threadIdx.x < 2) bad[(k + 2) & 3][threadIdx.x] = 0;
      __syncthreads();
    }

#pragma unroll
    for (int n = 0; n < NT; n++)
      if (kg == 0) {
        ms[wk][R * wr + 16 * n + col] = rows.m[n];
        ls[wk][R * wr + 16 * n + col] = rows.l[n][0];
      }
    for (int first = 0; first < WR; first += kGroups) {
      for (int x = 0; x < Sh::kWK; x++) {
        __syncthreads();
        if (x != wk || wr < first || wr >= first + kGroups) continue;
#pragma unroll
        for (int n = 0; n < NT; n++) {
          const int r = R * wr + 16 * n;
          float top = ms[0][r + col];
#pragma unroll
          for (int y = 1; y < Sh::kWK; y++) top = fmaxf(top, ms[y][r + col]);
          rows.join(n, (float*)lds + (r - R * first) * (DV + 4), DV + 4, top, x == 0, lane);
        }
      }
      __syncthreads();
      write_item<FMT, DV, MT>(arguments(), w, w.group, workers, R * first, R * kGroups, (const float*)lds, ms[0], ls[0], Sh::kWK, threadIdx.x,
                              Sh::kThreads, part, part_ml);
    }
    w.leave_open(arguments(), open, workers);
    __syncthreads();
    if (!w.next(arguments())) break;
  }
}

}  // namespace
