// Attention for few rows a key head: the four waves of a worker take four heads, or two or one with positions of their own,
// and meet once an item.  Heads side by side read whole stretches of tokens: 8 heads of 128 bytes were read at 5.4 TB/s by
// waves with a head each, at 4.6 TB/s by waves with 32 positions each of one head.
//
// Codes of K go from memory to registers as they are needed there (a lane: a quarter of a key's elements); V's are
// dequantized into the wave's own piece of LDS.  The next tile's codes are on their way while a tile is worked on: K's
// during its softmax and second product, V's during the next tile's first product.
//
// Bound by memory once a worker is under way, and by the trips to memory before that (lengths, pages, codes: about 12 us with
// the launch and the sums' way out).  32 sequences of up to 3900 positions (3032 on average), 8 key heads, 4 rows each, MXFP8:
// 49.0 us, 4.2 TB/s of codes and scales with all of that, and 5.1 us for the join; one sequence of 78 positions: 8.0 us.  The
// 4-bit formats read half the bytes behind the same trips and conversions: 33 us (MXFP4) and 40 us (NVFP4), with the join.
#pragma once

#include "attend_common.h"

namespace {

constexpr int kTile = 32;  // positions of a wave at a time

template <int FMT, int DK, int DV, int NT>
struct Shape {
  static constexpr int kRows = 16 * NT;
  static constexpr int kSteps = DK / 32;                       // matrix instructions a 16 x 16 tile of S
  static constexpr int kQuarter = DK / 4;                      // elements of a key in a lane
  static constexpr int kCodes = kQuarter / kPerByte<FMT> / 4;  // registers of their codes
  // scales of a lane's quarter: it may begin inside a block
  static constexpr int kScales = kQuarter <= kBlock<FMT> ? 1 : (kQuarter + kBlock<FMT> - 1) / kBlock<FMT>;
  static constexpr int kElems = 16 * kPerByte<FMT>;            // elements of a 16-byte piece of V
  static constexpr int kPerKey = DV / kElems;
  static constexpr int kPieces = kTile * kPerKey / 64;
  static constexpr int kPieceScales = kElems / kBlock<FMT> ? kElems / kBlock<FMT> : 1;
  static constexpr int kVT = DV / 16;
  static constexpr int kStride = DV + 16;  // of V's rows in LDS: 32 bytes on, so that eight rows meet no bank twice
};

// PAGED: pages of whole tiles, and dimensions that are DK and DV.  A tile's page is then looked up once, and a lane's part
// of the addresses does not change from tile to tile.  The same sequences, with the join, us with pages of 64 and of 16 tokens:
// MXFP8 45, 59 (128 elements), 52, 81 (192 and 128), 95, 159 (256); MXFP4 33, 54; 41, 68; 59, 104; NVFP4 41, 64; 58, 85; 69,
// 120.  Other sizes take the second form with any page, and the work of the size that they are padded to: 96 elements 55 (MXFP8),
// 50, 57 us; 160 elements 135, 94, 108 us (floors 30, 15, 16 and 50, 26, 27).
template <int FMT, int DK, int DV, int NT, int WAVES, bool PAGED, bool FINE>
__global__ __launch_bounds__(kThreads, WAVES) void attend_split_kernel(AttendArgs given, float* __restrict__ part,
                                                                 float2* __restrict__ part_ml, Open* __restrict__ open,
                                                                 Totals* __restrict__ totals, int workers) {
  using Sh = Shape<FMT, DK, DV, NT>;
  using Found = std::conditional_t<PAGED, int32_t, int64_t>;
  constexpr int MT = Sh::kRows;
  constexpr int kBytes = kWaves * kTile * Sh::kStride * 2;
  static_assert(16 * (DV + 4) * 4 <= kBytes / kWaves, "sixteen rows' sums take the place of a wave's V");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kBytes];
  __shared__ float ms[kWaves][MT], ls[kWaves][MT];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, kg = lane >> 4;
  Work<MT> w;
  if (!w.begin(given, workers, open, totals, lane)) return;
  const CacheArgs& c = given.cache;
  const float sc = score_scale<FMT>(given);
  const int heads = c.heads, k_dim = PAGED ? DK : c.plane[0].dim, v_dim = PAGED ? DV : c.plane[1].dim;
  const int64_t k_bytes = k_dim / kPerByte<FMT>, v_bytes = v_dim / kPerByte<FMT>;
  const int k_blocks = k_dim / kBlock<FMT>, v_blocks = v_dim / kBlock<FMT>;
  // this lane's part of a key's and of a value's codes and scales; PAGED: among the tile's
  const uint32_t in_tile = PAGED ? col * heads : 0, v_in_tile = PAGED ? lane / Sh::kPerKey * heads : 0;
  const uint32_t k_at = in_tile * (DK / kPerByte<FMT>) + kg * (Sh::kCodes * 4);
  const uint32_t ks_at = in_tile * (DK / kBlock<FMT>) + kg * Sh::kQuarter / kBlock<FMT>;
  const uint32_t v_at = v_in_tile * (DV / kPerByte<FMT>) + 16 * (lane % Sh::kPerKey);
  const uint32_t vs_at = v_in_tile * (DV / kBlock<FMT>) + lane % Sh::kPerKey * Sh::kElems / kBlock<FMT>;
  uint16_t* const vt = (uint16_t*)lds + wave * kTile * Sh::kStride;

  // 2^heads_log heads of a worker, for each of them `side` waves; a unit is a tile of each wave
  const int side_log = 2 - given.heads_log, side = 1 << side_log, first_wave = wave & ~(side - 1);

  for (;;) {
    w.settle();
    const Seq& s = w.s;
    const int32_t k0 = w.k0, k1 = w.k1(), end = w.ti.end, g = (w.group << given.heads_log) + (wave >> side_log);
    const auto base_of = [&](int32_t k) { return ((k << side_log) + (wave & (side - 1))) * kTile; };
    const int32_t* const pages = c.table + (int64_t)w.b * c.ld_table;

    // Where a tile's codes are.  PAGED: its page, in every lane; else in the lanes 0 to 31 the cache's vector of each of its
    // positions, -1: none.  No load waits for another, or hangs on a branch, which would make the waits for it wait for
    // those behind it as well: places past the end, without a page or past a vector are replaced by some that are there, and
    // what comes from them is dropped.
    const auto find = [&](int32_t k) {
      const int32_t pos = base_of(k) + (PAGED ? 0 : lane & 31), there = min(pos, end - 1);
      const uint32_t p = given.page_of((uint32_t)there);
      const int32_t page = pages[p];
      Found f = page;
      if (!PAGED)
        f = pos < end && page >= 0 && page < c.num_pages
                ? ((int64_t)page * c.page_size + ((uint32_t)there - p * (uint32_t)c.page_size)) * heads + g
                : -1;
      return f;
    };
    // PAGED: the tile's first vector.  Its positions past the end lie in the page too.
    const auto first_vector = [&](int32_t k, Found f) -> int64_t {
      const int32_t page = uniform((int)f), there = page < 0 || page >= c.num_pages ? 0 : page;
      const uint32_t pos = base_of(k);
      return ((int64_t)there * c.page_size + (pos - given.page_of(pos) * (uint32_t)c.page_size)) * heads + g;
    };
    uint32_t kc[2][Sh::kCodes], ks[2][Sh::kScales];
    // a lane's quarter of a key
    const auto load_key = [&](int t, const uint8_t* src, const uint8_t* scales) {
      if constexpr (PAGED) {
        if constexpr (Sh::kCodes % 4 == 0) {
#pragma unroll
          for (int i = 0; i < Sh::kCodes; i += 4) {
            const u32x4_t x = *reinterpret_cast<const u32x4_a8*>(src + 4 * i);
            kc[t][i] = x[0];
            kc[t][i + 1] = x[1];
            kc[t][i + 2] = x[2];
            kc[t][i + 3] = x[3];
          }
        } else {
#pragma unroll
          for (int i = 0; i < Sh::kCodes; i += 2) {
            const u32x2_t x = *reinterpret_cast<const u32x2_a8*>(src + 4 * i);
            kc[t][i] = x[0];
            kc[t][i + 1] = x[1];
          }
        }
#pragma unroll
        for (int i = 0; i < Sh::kScales; i++) ks[t][i] = scales[i];
      } else {
        constexpr int per = FMT == MXFP4_FMT_MXFP8 ? 2 : 1;  // registers of eight codes
#pragma unroll
        for (int i = 0; i < Sh::kSteps; i++) {
          const bool in = kg * Sh::kQuarter + 8 * i < k_dim;
          const uint8_t* from = src + (in ? (int)k_at + 4 * per * i : 0);
          if constexpr (per == 2) {
            const u32x2_t x = *reinterpret_cast<const u32x2_a8*>(from);
            kc[t][2 * i] = in ? x[0] : 0;
            kc[t][2 * i + 1] = in ? x[1] : 0;
          } else {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(from);
            kc[t][i] = in ? x : 0;
          }
        }
#pragma unroll
        for (int i = 0; i < Sh::kScales; i++) ks[t][i] = scales[min((int)ks_at + i, k_blocks - 1)];
      }
    };
    const auto load_k = [&](int32_t k, Found f) {
      const int64_t first = PAGED ? first_vector(k, f) : 0;
#pragma unroll
      for (int t = 0; t < 2; t++) {
        if (PAGED) {  // the tile's part of the addresses is the same for all lanes, the lane's for all tiles
          const int64_t at = first + 16 * t * heads;
          load_key(t, c.plane[0].q + at * k_bytes + k_at, c.plane[0].s + at * k_blocks + ks_at);
        } else {
          const int64_t at = shfl64(f, 16 * t + col), there = at < 0 ? 0 : at;
          load_key(t, c.plane[0].q + there * k_bytes, c.plane[0].s + there * k_blocks);
        }
      }
    };
    u32x4_t vc[Sh::kPieces];
    uint32_t vs[Sh::kPieces][Sh::kPieceScales];
    const auto load_v = [&](int32_t k, Found f) {
      const int64_t first = PAGED ? first_vector(k, f) : 0;
#pragma unroll
      for (int i = 0; i < Sh::kPieces; i++) {
        constexpr int keys = 64 / Sh::kPerKey;  // of 64 pieces
        if (PAGED) {
          const int64_t at = first + keys * i * heads;
          vc[i] = *reinterpret_cast<const u32x4_a8*>(c.plane[1].q + at * v_bytes + v_at);
          const uint8_t* scales = c.plane[1].s + at * v_blocks + vs_at;
#pragma unroll
          for (int j = 0; j < Sh::kPieceScales; j++) vs[i][j] = scales[j];
        } else {
          const int64_t at = shfl64(f, keys * i + lane / Sh::kPerKey), there = at < 0 ? 0 : at;
          // in halves: the last piece of a vector may be one
          const int e = lane % Sh::kPerKey * Sh::kElems;
          const bool in = e < v_dim, all = e + Sh::kElems <= v_dim;
          const uint8_t* src = c.plane[1].q + there * v_bytes;
          const u32x2_t x = *reinterpret_cast<const u32x2_a8*>(src + (in ? v_at : 0)), y = *reinterpret_cast<const u32x2_a8*>(src + (all ? v_at + 8 : 0));
          vc[i] = u32x4_t{in ? x[0] : 0, in ? x[1] : 0, all ? y[0] : 0, all ? y[1] : 0};
          const uint8_t* scales = c.plane[1].s + there * v_blocks;
#pragma unroll
          for (int j = 0; j < Sh::kPieceScales; j++) vs[i][j] = scales[min((int)vs_at + j, v_blocks - 1)];
        }
      }
    };

    Found found = -1, next = -1;
    if (end > 0) {
      found = find(k0);
      next = find(k0 + 1);
    }
    const auto element = [&](int i) { return kg * Sh::kQuarter + 8 * i; };
    Query<NT, Sh::kSteps> query;
    query.load(arguments(), s, w.ti.tile * MT, g, element);
    if (end > 0) {
      load_k(k0, found);
      load_v(k0, found);
    }
    query.finish(arguments(), element);
    const auto& q = query.q;
    const auto& draft = query.draft;
    Rows<NT, Sh::kVT, FINE> rows;
    rows.clear();

    const auto step = [&](int32_t k, auto more) {
      constexpr bool kMore = decltype(more)::value;  // another tile follows
      const int32_t base = base_of(k);
      // which of the tile's positions have a vector, and whether all rows see them all
      uint32_t there;
      if (PAGED) {
        const int32_t page = uniform((int)found), left = end - base;
        there = page < 0 || page >= c.num_pages || left <= 0 ? 0u : left >= kTile ? ~0u : (1u << left) - 1;
      } else {
        there = (uint32_t)__ballot(found >= 0);
      }
      const bool whole = there == ~0u && base + kTile <= s.start;
      Found after = -1;
      if (kMore) after = find(k + 2);

      f32x4_t sv[NT][2];
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int n = 0; n < NT; n++) sv[n][t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < Sh::kSteps; i++)
#pragma unroll
        for (int t = 0; t < 2; t++) {
          constexpr int per = FMT == MXFP4_FMT_MXFP8 ? 2 : 1;
          uint32_t scale = ks[t][0];
          if constexpr (Sh::kScales > 1) {
            // the block of this chunk, counted from the quarter's first; the quarter may begin inside one
            constexpr int B = kBlock<FMT>;
            const int even = 8 * i / B, odd = (Sh::kQuarter % B + 8 * i) / B;  // kg even, kg odd
            scale = Sh::kQuarter % B && (kg & 1) ? ks[t][odd < Sh::kScales ? odd : Sh::kScales - 1] : ks[t][even];
          }
          const bf16x8_t x = values8<FMT>(kc[t][per * i], kc[t][per * i + per - 1], scale);
#pragma unroll
          for (int n = 0; n < NT; n++) sv[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, q[n][i], sv[n][t], 0, 0, 0);
        }
      if (kMore) load_k(k + 1, next);

      if (!whole) {
        // Positions whose values are not finite must not meet the zero weights of rows that do not see them: they count as
        // zeros, and make the score of rows that do see them NaN.  Those without a page count as zeros.
        uint32_t bad = 0;
        if (base + kTile > s.start) {
#pragma unroll
          for (int i = 0; i < Sh::kPieces; i++) {
            bool x = false;
#pragma unroll
            for (int j = 0; j < Sh::kPieceScales; j++) x = x || not_finite<FMT>(vs[i][j]);
            if (FMT == MXFP4_FMT_MXFP8)
              x = x || has_nan_code(vc[i][0]) || has_nan_code(vc[i][1]) || has_nan_code(vc[i][2]) || has_nan_code(vc[i][3]);
            for (uint64_t who = __ballot(x); who; who &= who - 1)
              bad |= 1u << ((i * 64 + __ffsll((unsigned long long)who) - 1) / Sh::kPerKey);
          }
        }
        if (const uint32_t zero = bad | ~there) {
#pragma unroll
          for (int i = 0; i < Sh::kPieces; i++)
            if (zero >> ((i * 64 + lane) / Sh::kPerKey) & 1) {
              vc[i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
              for (int j = 0; j < Sh::kPieceScales; j++) vs[i][j] = 0;
            }
        }
        hide<NT, 2>(arguments(), s, draft, base, there, bad, kg, sv);
      }

      Weights<NT, 2, FINE> p;
      rows.template weights<2>(sv, sc, p);

      // V into LDS, a row a position
#pragma unroll
      for (int i = 0; i < Sh::kPieces; i++) {
        const int id = i * 64 + lane;
        uint16_t* dst = vt + id / Sh::kPerKey * Sh::kStride + id % Sh::kPerKey * Sh::kElems;
#pragma unroll
        for (int j = 0; j < Sh::kElems / 8; j++) {
          const bf16x8_t x = FMT == MXFP4_FMT_MXFP8 ? values8<FMT>(vc[i][2 * j], vc[i][2 * j + 1], vs[i][0])
                                                    : values8<FMT>(vc[i][j], 0, vs[i][8 * j / kBlock<FMT>]);
          *reinterpret_cast<bf16x8_t*>(dst + 8 * j) = x;
        }
      }
      if (kMore) load_v(k + 1, next);
      __builtin_amdgcn_wave_barrier();
      rows.template add_values<1, 2>(vt, Sh::kStride, p, 0, lane);
      __builtin_amdgcn_wave_barrier();
      found = next;
      next = after;
    };
    if (end > 0) {
      for (int32_t k = k0; k + 1 < k1; k++) step(k, std::true_type{});
      step(k1 - 1, std::false_type{});
    }

    // the sums of a head's waves, joined
#pragma unroll
    for (int n = 0; n < NT; n++)
      if (kg == 0) {
        ms[wave][16 * n + col] = rows.m[n];
        ls[wave][16 * n + col] = rows.l[n][0];
      }
    float* const sums = (float*)(lds + first_wave * (kBytes / kWaves));
#pragma unroll
    for (int n = 0; n < NT; n++) {
      for (int x = 0; x < side; x++) {
        __syncthreads();
        if (first_wave + x != wave) continue;
        float top = ms[first_wave][16 * n + col];
        for (int y = 1; y < side; y++) top = fmaxf(top, ms[first_wave + y][16 * n + col]);
        rows.join(n, sums, DV + 4, top, x == 0, lane);
      }
      __syncthreads();
      write_item<FMT, DV, MT>(arguments(), w, g, workers, 16 * n, 16, sums, ms[first_wave], ls[first_wave], side,
                              (wave - first_wave) * 64 + lane, side * 64, part, part_ml);
    }
    w.leave_open(arguments(), open, workers);
    __syncthreads();
    if (!w.next(arguments())) break;
  }
}

}  // namespace
