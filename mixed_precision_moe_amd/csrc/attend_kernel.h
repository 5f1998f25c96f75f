// Attention over the block-quantized paged cache: rows see the positions before their sequence's drafts, and of the
// drafts those that a mask or their order leaves.
//
//   out[t, h] = sum_j p_j V[j, g] / sum_j p_j,  p_j = exp2(s_j - m),  s_j = scale log2(e) q[t, h] . K[j, g],  m >= s_j
//
// Work.  The rows of a sequence that share a key head (drafts times query heads of the group) are cut into tiles of 16 NT.
// A tile and the positions it sees are an item; items are cut into units of 128 positions, and a head's units are dealt
// out evenly to its workers (workgroups), each a contiguous range: a worker's first and last item may be parts, which
// go to the workspace as sums with their maximum and are joined by a second launch, in worker order.  Every worker finds
// its range from the lengths on the device, so nothing about them has to be known on the host.
//
// A worker's four waves take 32 positions of a unit each and meet once an item.  A wave forms S^T = K Q^T and O^T = V^T P^T:
// a row of q is a column of both, so its maximum, sum and rescaling stay in one lane (and three others, which hold
// other positions), and S^T leaves the matrix instruction as P^T enters the next one.  Codes of K go from memory to registers
// as they are needed there (a lane: a quarter of a key's elements); V's are dequantized into the wave's own piece of LDS and
// read back transposed.  Values are exact in bf16 (at most six significant bits), so both products are what the cache holds.
// The next tile's codes are on their way while a tile is worked on: K's during its softmax and second product, V's during the
// next tile's first product.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "cache_slots.h"
#include "drafts.h"

#define MX_DEV __device__ __forceinline__

namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef u32x4_t u32x4_a8 __attribute__((aligned(8)));  // vectors of codes start on 8 bytes
typedef u32x2_t u32x2_a8 __attribute__((aligned(8)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kTile = 32;               // positions of a wave at a time
constexpr int kUnit = kTile * kWaves;   // and of a worker

template <int FMT>
constexpr int kBlock = FMT == MXFP4_FMT_NVFP4 ? 16 : 32;
template <int FMT>
constexpr int kPerByte = FMT == MXFP4_FMT_MXFP8 ? 1 : 2;

// What a worker leaves for the join, next to its sums: the item that it begins and another worker ends.
struct Open {
  int32_t tile, seq, last;  // last: the worker that ends it; -1: none
};

// ---------------------------------------------------------------------------------------------
// Eight values as bf16: c their codes (4-bit formats: c[0]), s the block's scale byte.
template <int FMT>
MX_DEV bf16x8_t values8(uint32_t c0, uint32_t c1, uint32_t s) {
  u32x4_t o;
  if (FMT == MXFP4_FMT_MXFP8) {
    const float f = __uint_as_float(s << 23);
    o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, f, false));
    o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, f, true));
    o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, f, false));
    o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, f, true));
  } else if (FMT == MXFP4_FMT_MXFP4) {
    const float f = __uint_as_float(s << 23);
    o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c0, f, 0));
    o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c0, f, 1));
    o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c0, f, 2));
    o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c0, f, 3));
  } else {
    // the product has at most six significant bits, so the upper halves of its binary32 form are all of it
    const float f = __builtin_amdgcn_cvt_f32_fp8((int)s, 0);
    auto two = [&](auto v) {
      return __builtin_amdgcn_perm(__float_as_uint(v[1] * f), __float_as_uint(v[0] * f), 0x07060302u);
    };
    o[0] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c0, 1.0f, 0));
    o[1] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c0, 1.0f, 1));
    o[2] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c0, 1.0f, 2));
    o[3] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c0, 1.0f, 3));
  }
  return __builtin_bit_cast(bf16x8_t, o);
}

// Whether a block with this scale (and for MXFP8 these codes) may hold values that are not finite in bf16.
template <int FMT>
MX_DEV bool not_finite(uint32_t s) {
  return FMT == MXFP4_FMT_NVFP4 ? (s & 0x7Fu) == 0x7Fu : FMT == MXFP4_FMT_MXFP8 ? s > 246u : s > 252u;
}
MX_DEV bool has_nan_code(uint32_t c) {  // a byte whose lower seven bits are all set
  const uint32_t x = ~c & 0x7F7F7F7Fu;
  return ((x - 0x01010101u) & ~x & 0x80808080u) != 0;
}

// ---------------------------------------------------------------------------------------------
// Sequences, items and units.

struct Seq {
  int32_t first;   // its first row
  int32_t drafts;  // of its own
  int32_t rows;    // of them that q holds
  int32_t start;
};

MX_DEV Seq sequence(const AttendArgs& a, int b) {
  const CacheArgs& c = a.cache;
  const int32_t at = c.cu[b], end = c.cu[b + 1], there = min((int64_t)end, c.rows);
  const bool some = at >= 0 && there > at;
  return Seq{at, some ? end - at : 0, some ? there - at : 0, c.start ? c.start[b] : 0};
}

// Of a sequence, tile by tile: the positions that some row of the tile sees are below `end`, 128 of them are a unit; a tile
// has one at least, since its rows are written where nothing is seen too.
struct Tiles {
  int32_t tile, tiles, end, units;
  int32_t row, part;  // without a mask: the draft of the row behind the tile, and that row's place in its group

  MX_DEV void set(const AttendArgs& a, const Seq& s) {
    const int64_t n = a.mask ? s.drafts : min(s.rows, row + (part > 0));
    const int64_t e = min(s.start + n, (int64_t)a.cache.max_pages * a.cache.page_size);
    end = e < 0 ? 0 : (int32_t)e;
    units = end <= kUnit ? 1 : (end + kUnit - 1) / kUnit;
  }
  MX_DEV void begin(const AttendArgs& a, const Seq& s, int mt) {
    tile = 0;
    tiles = (s.rows * a.group + mt - 1) / mt;
    row = a.rows_of_tile;
    part = a.part_of_tile;
    set(a, s);
  }
  MX_DEV void next(const AttendArgs& a, const Seq& s) {
    tile++;
    row += a.rows_of_tile;
    part += a.part_of_tile;
    if (part >= a.group) {
      part -= a.group;
      row++;
    }
    set(a, s);
  }
};

MX_DEV int64_t seq_units(const AttendArgs& a, const Seq& s, int mt) {
  Tiles t;
  t.begin(a, s, mt);
  if (a.mask) return (int64_t)t.tiles * t.units;
  int64_t n = 0;
  while (t.tile < t.tiles) {
    n += t.units;
    t.next(a, s);
  }
  return n;
}

MX_DEV int64_t shfl64(int64_t v, int lane) {
  const int lo = __shfl((int)v, lane), hi = __shfl((int)(v >> 32), lane);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}
MX_DEV int64_t lane64(int64_t v, int lane) {  // the same for the whole wave, and known to be
  const int lo = __builtin_amdgcn_readlane((int)v, lane), hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}
MX_DEV int64_t shfl64_up(int64_t v, int by) {
  const int lo = __shfl_up((int)v, by), hi = __shfl_up((int)(v >> 32), by);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// Units of the 64 sequences from b0 on, summed up to and including each lane's.
MX_DEV int64_t scan_units(const AttendArgs& a, int b0, int lane, int mt) {
  int64_t n = 0;
  if (b0 + lane < a.cache.n_seqs) n = seq_units(a, sequence(a, b0 + lane), mt);
#pragma unroll
  for (int h = 1; h < 64; h <<= 1) {
    const int64_t o = shfl64_up(n, h);
    if (lane >= h) n += o;
  }
  return n;
}

// Eight elements of a row of the result from its sums x, y and the sum of its weights.
template <int FMT>
MX_DEV void write_row(const AttendArgs& a, const Seq& s, int32_t r, int g, int e, f32x4_t x, f32x4_t y, float sum) {
  const CachePlane& pv = a.cache.plane[1];
  const int32_t d = (uint32_t)r / (uint32_t)a.group;
  const int64_t at = (int64_t)(s.first + d) * pv.ldt + (g * a.group + (r - d * a.group)) * pv.ldh + e;
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    x[i] *= f;
    y[i] *= f;
    if (FMT == MXFP4_FMT_NVFP4) {
      x[i] /= pv.gs;
      y[i] /= pv.gs;
    }
  }
  if (a.out_fp32) {
    f32x4_t* dst = reinterpret_cast<f32x4_t*>((float*)pv.rows + at);
    dst[0] = x;
    dst[1] = y;
  } else {
    bf16x8_t v;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[i] = (__bf16)x[i];
      v[4 + i] = (__bf16)y[i];
    }
    *reinterpret_cast<bf16x8_t*>((uint16_t*)pv.rows + at) = v;
  }
}

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
  static constexpr int kSums = DV + 4;     // of the joined sums' rows
};

// PAGED: pages of whole tiles, and dimensions that are DK and DV.  A tile's page is then looked up once, and a lane's part
// of the addresses does not change from tile to tile.
template <int FMT, int DK, int DV, int NT, int WAVES, bool PAGED>
__global__ __launch_bounds__(kThreads, WAVES) void attend_kernel(AttendArgs a, float* __restrict__ part,
                                                                 float2* __restrict__ part_ml, Open* __restrict__ open,
                                                                 int workers) {
  using Sh = Shape<FMT, DK, DV, NT>;
  using Found = std::conditional_t<PAGED, int32_t, int64_t>;
  constexpr int MT = Sh::kRows;
  constexpr int kBytes = kWaves * kTile * Sh::kStride * 2;
  static_assert(MT * Sh::kSums * 4 <= kBytes, "the sums take the place of V");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kBytes];
  __shared__ float ms[kWaves][MT], ls[kWaves][MT];
  const CacheArgs& c = a.cache;
  const CachePlane &pk = c.plane[0], &pv = c.plane[1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, kg = lane >> 4;
  // Workgroups go to the eight XCDs in turn: a worker's heads, which read pieces of the same tokens, share one.
  int g, worker;
  if (workers % 8 == 0) {
    const int i = blockIdx.x / 8;
    g = i % c.heads;
    worker = i / c.heads * 8 + blockIdx.x % 8;
  } else {
    g = blockIdx.x % c.heads;
    worker = blockIdx.x / c.heads;
  }
  const int64_t at_worker = (int64_t)g * workers + worker;  // as the join counts them

  // this worker's units
  int64_t all = 0;
  for (int b = 0; b < c.n_seqs; b += 64) all += lane64(scan_units(a, b, lane, MT), 63);
  const int64_t used = min((int64_t)workers, all);
  if (threadIdx.x == 0) open[at_worker] = Open{0, 0, -1};
  if (worker >= used) return;
  const int64_t u0 = all / used * worker + all % used * worker / used;
  const int64_t u1 = all / used * (worker + 1) + all % used * (worker + 1) / used;
  // the item of the first of them
  int b = 0;
  int64_t item = 0;  // its first unit
  for (int b0 = 0; b0 < c.n_seqs; b0 += 64) {
    const int64_t sums = item + scan_units(a, b0, lane, MT);
    const uint64_t past = __ballot(sums > u0);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      b = b0 + l;
      if (l > 0) item = lane64(sums, l - 1);
      break;
    }
    item = lane64(sums, 63);
  }
  Seq s = sequence(a, b);
  Tiles ti;
  ti.begin(a, s, MT);
  while (item + ti.units <= u0) {
    item += ti.units;
    ti.next(a, s);
  }

  // not 0, so that its product with a hidden position's -inf is one
  const float sc = fmaxf((a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * 1.44269504f / (FMT == MXFP4_FMT_NVFP4 ? pk.gs : 1.0f), 1e-38f);
  const float per_sc = 1.0f / sc;
  // the scale's sign goes to q; with a scale of 0 all of it is 0
  const uint32_t q_and = a.scale == 0.0f ? 0u : ~0u, q_xor = a.scale < 0.0f ? 0x80008000u : 0u;
  const int k_dim = PAGED ? DK : pk.dim, v_dim = PAGED ? DV : pv.dim;
  const int64_t k_bytes = k_dim / kPerByte<FMT>, v_bytes = v_dim / kPerByte<FMT>;
  const int k_blocks = k_dim / kBlock<FMT>, v_blocks = v_dim / kBlock<FMT>;
  // PAGED: this lane's part of the addresses of codes and scales
  const uint32_t k_at = (uint32_t)(col * c.heads) * (DK / kPerByte<FMT>) + kg * (Sh::kCodes * 4);
  const uint32_t ks_at = (uint32_t)(col * c.heads) * (DK / kBlock<FMT>) + kg * Sh::kQuarter / kBlock<FMT>;
  const uint32_t v_at = (uint32_t)(lane / Sh::kPerKey * c.heads) * (DV / kPerByte<FMT>) + 16 * (lane % Sh::kPerKey);
  const uint32_t vs_at = (uint32_t)(lane / Sh::kPerKey * c.heads) * (DV / kBlock<FMT>) + lane % Sh::kPerKey * Sh::kElems / kBlock<FMT>;
  uint16_t* const vt = (uint16_t*)lds + wave * kTile * Sh::kStride;

  int64_t u = u0;
  while (u < u1) {
    const int32_t k0 = (int32_t)(u - item), k1 = (int32_t)min((int64_t)ti.units, u1 - item), end = ti.end;
    // the rows of this lane's columns
    bf16x8_t q[NT][Sh::kSteps];
    int32_t draft[NT];  // -1: no such row
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const int32_t r = ti.tile * MT + 16 * n + col;
      const int32_t d = (uint32_t)r / (uint32_t)a.group;
      draft[n] = d < s.rows ? d : -1;
      const uint16_t* src = (const uint16_t*)pk.rows + (int64_t)(s.first + d) * pk.ldt + (g * a.group + (r - d * a.group)) * pk.ldh;
#pragma unroll
      for (int i = 0; i < Sh::kSteps; i++) {
        const int e = kg * Sh::kQuarter + 8 * i;
        u32x4_t x = {0, 0, 0, 0};
        if (draft[n] >= 0 && e < k_dim) x = *reinterpret_cast<const u32x4_t*>(src + e);
#pragma unroll
        for (int j = 0; j < 4; j++) x[j] = (x[j] & q_and) ^ q_xor;
        q[n][i] = __builtin_bit_cast(bf16x8_t, x);
      }
    }
    // sums, of the weights too; the exponents' subtrahend m, and the score from which on it is raised
    f32x4_t o[NT][Sh::kVT], l[NT];
    float m[NT], limit[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) {
      m[n] = limit[n] = -INFINITY;
      l[n] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < Sh::kVT; v++) o[n][v] = f32x4_t{0, 0, 0, 0};
    }

    // Where a tile's codes are.  PAGED: its page, in every lane; else the cache's vector of each of its positions, -1: none,
    // in the lanes 0 to 31.
    const int32_t* const pages = c.table + (int64_t)b * c.ld_table;
    const auto find = [&](int32_t k) {
      const int32_t pos = k * kUnit + wave * kTile + (PAGED ? 0 : lane & 31);
      Found f = -1;
      if (pos < end) {
        const uint32_t p = a.page_shift >= 0 ? (uint32_t)pos >> a.page_shift : (uint32_t)pos / (uint32_t)c.page_size;
        const int32_t page = pages[p];
        if (PAGED)
          f = page;
        else if (page >= 0 && page < c.num_pages)
          f = ((int64_t)page * c.page_size + ((uint32_t)pos - p * (uint32_t)c.page_size)) * c.heads + g;
      }
      return f;
    };
    // PAGED: the tile's first vector, -1: none.  Its positions past the end lie in the page too.
    const auto first_vector = [&](int32_t k, Found f) -> int64_t {
      const int32_t page = __builtin_amdgcn_readfirstlane((int)f);
      if (page < 0 || page >= c.num_pages) return -1;
      const uint32_t pos = (uint32_t)k * kUnit + (uint32_t)wave * kTile;
      const uint32_t in_page = a.page_shift >= 0 ? pos & (uint32_t)(c.page_size - 1) : pos % (uint32_t)c.page_size;
      return ((int64_t)page * c.page_size + in_page) * c.heads + g;
    };
    uint32_t kc[2][Sh::kCodes], ks[2][Sh::kScales];
    // a lane's quarter of a key
    const auto load_key = [&](int t, const uint8_t* src, const uint8_t* scales) {
      if (PAGED || pk.dim == DK) {
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
      } else {
        constexpr int per = FMT == MXFP4_FMT_MXFP8 ? 2 : 1;  // registers of eight codes
#pragma unroll
        for (int i = 0; i < Sh::kSteps; i++) {
          const int e = kg * Sh::kQuarter + 8 * i;
#pragma unroll
          for (int j = 0; j < per; j++) {
            kc[t][per * i + j] = 0;
            if (e < pk.dim) kc[t][per * i + j] = *reinterpret_cast<const uint32_t*>(src + 4 * (per * i + j));
          }
        }
      }
      const int b0 = kg * Sh::kQuarter / kBlock<FMT>;
#pragma unroll
      for (int i = 0; i < Sh::kScales; i++) {
        ks[t][i] = 0;
        if (PAGED || b0 + i < k_blocks) ks[t][i] = scales[i];
      }
    };
    const auto load_k = [&](int32_t k, Found f) {
      const int64_t first = PAGED ? first_vector(k, f) : 0;
#pragma unroll
      for (int t = 0; t < 2; t++) {
        if (PAGED) {  // the tile's part of the addresses is the same for all lanes, the lane's for all tiles
          const int64_t at = first + 16 * t * c.heads;
          if (first >= 0) load_key(t, pk.q + at * k_bytes + k_at, pk.s + at * k_blocks + ks_at);
        } else {
          const int64_t at = shfl64(f, 16 * t + col);
          if (at >= 0) load_key(t, pk.q + at * k_bytes + kg * (Sh::kCodes * 4), pk.s + at * k_blocks + kg * Sh::kQuarter / kBlock<FMT>);
        }
      }
    };
    u32x4_t vc[Sh::kPieces];
    uint32_t vs[Sh::kPieces][Sh::kPieceScales];
    const auto load_piece = [&](int i, const uint8_t* src, const uint8_t* scales) {
      const int e = lane % Sh::kPerKey * Sh::kElems;
      if (PAGED || e + Sh::kElems <= pv.dim) {
        vc[i] = *reinterpret_cast<const u32x4_a8*>(src);
      } else if (e < pv.dim) {
        const u32x2_t x = *reinterpret_cast<const u32x2_a8*>(src);
        vc[i] = u32x4_t{x[0], x[1], 0, 0};
      }
      const int b0 = e / kBlock<FMT>;
#pragma unroll
      for (int j = 0; j < Sh::kPieceScales; j++)
        if (PAGED || b0 + j < v_blocks) vs[i][j] = scales[j];
    };
    const auto load_v = [&](int32_t k, Found f) {
      const int64_t first = PAGED ? first_vector(k, f) : 0;
#pragma unroll
      for (int i = 0; i < Sh::kPieces; i++) {
        constexpr int keys = 64 / Sh::kPerKey;  // of 64 pieces
        if (PAGED) {
          const int64_t at = first + keys * i * c.heads;
          if (first >= 0) load_piece(i, pv.q + at * v_bytes + v_at, pv.s + at * v_blocks + vs_at);
        } else {
          vc[i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < Sh::kPieceScales; j++) vs[i][j] = 0;
          const int64_t at = shfl64(f, keys * i + lane / Sh::kPerKey);
          const int piece = lane % Sh::kPerKey;
          if (at >= 0) load_piece(i, pv.q + at * v_bytes + 16 * piece, pv.s + at * v_blocks + piece * Sh::kElems / kBlock<FMT>);
        }
      }
    };

    Found found = find(k0);
    load_k(k0, found);
    load_v(k0, found);
    for (int32_t k = k0; k < k1; k++) {
      const int32_t base = k * kUnit + wave * kTile;
      // which of the tile's positions have a vector, and whether all rows see them all
      uint32_t there;
      if (PAGED) {
        const int32_t page = __builtin_amdgcn_readfirstlane((int)found);
        const int32_t left = end - base;
        there = page < 0 || page >= c.num_pages || left <= 0 ? 0u : left >= kTile ? ~0u : (1u << left) - 1;
      } else {
        there = (uint32_t)__ballot(found >= 0);
      }
      const bool whole = there == ~0u && base + kTile <= s.start;
      const Found next = k + 1 < k1 ? find(k + 1) : -1;

      f32x4_t sv[NT][2];
#pragma unroll
      for (int t = 0; t < 2; t++) {
#pragma unroll
        for (int n = 0; n < NT; n++) sv[n][t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < Sh::kSteps; i++) {
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
      }
      if (k + 1 < k1) load_k(k + 1, next);

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
#pragma unroll
        for (int n = 0; n < NT; n++) {
          const uint8_t* mask = a.mask + (int64_t)(s.first + draft[n]) * a.ld_mask;
          const int64_t most = a.mask ? min(s.drafts, a.mask_cols) : (int64_t)draft[n] + 1;  // drafts past it are not seen
#pragma unroll
          for (int t = 0; t < 2; t++) {
            asm volatile("");  // a few loads of the mask at a time: all at once cost the registers of the loop around
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const int key = 16 * t + 4 * kg + i;
              const int64_t j = (int64_t)base + key - s.start;
              bool sees = draft[n] >= 0 && (there >> key & 1) && j < most;
              if (sees && j >= 0 && a.mask) sees = mask[j];
              if (!sees)
                sv[n][t][i] = -INFINITY;
              else if (bad >> key & 1)
                sv[n][t][i] = NAN;
            }
          }
        }
      }

      // m is raised, and all sums with it, where a score is over it by more than 8: weights stay below 2^8, and most tiles
      // need no maximum over the row's four lanes and no rescaling
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; n++) {
        float top = sv[n][0][0];
#pragma unroll
        for (int i = 1; i < 8; i++) top = fmaxf(top, sv[n][i >> 2][i & 3]);
        over = over || top > limit[n];
      }
      if (__any(over)) {
#pragma unroll
        for (int n = 0; n < NT; n++) {
          float top = sv[n][0][0];
#pragma unroll
          for (int i = 1; i < 8; i++) top = fmaxf(top, sv[n][i >> 2][i & 3]);
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          const float now = fmaxf(m[n], top * sc);
          const float keep = now > -INFINITY ? __builtin_amdgcn_exp2f(m[n] - now) : 1.0f;
#pragma unroll
          for (int i = 0; i < 4; i++) l[n][i] *= keep;
#pragma unroll
          for (int v = 0; v < Sh::kVT; v++)
#pragma unroll
            for (int i = 0; i < 4; i++) o[n][v][i] *= keep;
          m[n] = now;
          limit[n] = (now + 8.0f) * per_sc;
        }
      }
      // the weights' sum is taken of them as they are rounded, by the matrix instruction
      const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
      bf16x8_t p[NT];
#pragma unroll
      for (int n = 0; n < NT; n++) {
        const float by = m[n] > -INFINITY ? -m[n] : 0.0f;  // nothing seen yet
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = __builtin_amdgcn_exp2f(fmaf(sv[n][i >> 2][i & 3], sc, by));
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const bf16x2_t two = __builtin_convertvector(f32x2_t{w[i], w[i + 1]}, bf16x2_t);
          p[n][i] = two[0];
          p[n][i + 1] = two[1];
        }
        l[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, p[n], l[n], 0, 0, 0);
      }

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
      if (k + 1 < k1) load_v(k + 1, next);
      __builtin_amdgcn_wave_barrier();
      // two blocks of four positions by sixteen elements a group of sixteen lanes, transposed
      typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
      const uint16_t* src = vt + (4 * kg + (col >> 2)) * Sh::kStride + 4 * (col & 3);
#pragma unroll
      for (int v = 0; v < Sh::kVT; v++) {
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + 16 * v));
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + 16 * Sh::kStride + 16 * v));
        const bf16x8_t x = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
        for (int n = 0; n < NT; n++) o[n][v] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, p[n], o[n][v], 0, 0, 0);
      }
      __builtin_amdgcn_wave_barrier();
      found = next;
    }

    // the waves' sums, joined
#pragma unroll
    for (int n = 0; n < NT; n++) {
      if (kg == 0) {
        ms[wave][16 * n + col] = m[n];
        ls[wave][16 * n + col] = l[n][0];
      }
    }
    float* sums = (float*)lds;
    for (int w = 0; w < kWaves; w++) {
      __syncthreads();
      if (w != wave) continue;
#pragma unroll
      for (int n = 0; n < NT; n++) {
        float top = ms[0][16 * n + col];
#pragma unroll
        for (int x = 1; x < kWaves; x++) top = fmaxf(top, ms[x][16 * n + col]);
        const float f = top > -INFINITY ? __builtin_amdgcn_exp2f(m[n] - top) : 0.0f;
        float* dst = sums + (16 * n + col) * Sh::kSums + 4 * kg;
#pragma unroll
        for (int v = 0; v < Sh::kVT; v++) {
          f32x4_t x = o[n][v];
#pragma unroll
          for (int i = 0; i < 4; i++) x[i] *= f;
          if (w > 0) {
            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(dst + 16 * v);
#pragma unroll
            for (int i = 0; i < 4; i++) x[i] += y[i];
          }
          *reinterpret_cast<f32x4_t*>(dst + 16 * v) = x;
        }
      }
    }
    __syncthreads();
    // rows of the tile that exist, eight elements a thread
    const int there = min(MT, s.rows * a.group - ti.tile * MT);
    const bool whole_item = k0 == 0 && k1 == ti.units;
    const int64_t slot = 2 * at_worker + (k0 == 0 ? 1 : 0);
    for (int id = threadIdx.x; id < there * (DV / 8); id += kThreads) {
      const int r = id / (DV / 8), e = id % (DV / 8) * 8;
      float top = ms[0][r], sum = 0.0f;
      for (int x = 1; x < kWaves; x++) top = fmaxf(top, ms[x][r]);
      for (int x = 0; x < kWaves; x++) sum += top > -INFINITY ? ls[x][r] * __builtin_amdgcn_exp2f(ms[x][r] - top) : 0.0f;
      const f32x4_t *src = reinterpret_cast<const f32x4_t*>(sums + r * Sh::kSums + e);
      f32x4_t x = src[0], y = src[1];
      if (!whole_item) {
        f32x4_t* dst = reinterpret_cast<f32x4_t*>(part + (slot * MT + r) * DV + e);
        dst[0] = x;
        dst[1] = y;
        if (e == 0) part_ml[slot * MT + r] = float2{top, sum};
      } else if (e < v_dim) {
        write_row<FMT>(a, s, ti.tile * MT + r, g, e, x, y, sum);
      }
    }
    if (threadIdx.x == 0 && k0 == 0 && k1 < ti.units) {
      // the worker of the item's last unit
      const int64_t last = item + ti.units - 1;
      const int64_t w = ((last + 1) * used - 1) / all;
      open[at_worker] = Open{ti.tile, b, (int32_t)w};
    }
    __syncthreads();

    u += k1 - k0;
    item += ti.units;
    if (u >= u1) break;
    ti.next(a, s);
    if (ti.tile >= ti.tiles) {
      do s = sequence(a, ++b);
      while (s.rows == 0);
      ti.begin(a, s, MT);
    }
  }
}

// Joins the parts of the item that a worker begins and another ends; blockIdx.y: sixteen of its rows.
template <int FMT, int DV, int NT>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(AttendArgs a, const float* __restrict__ part,
                                                               const float2* __restrict__ part_ml,
                                                               const Open* __restrict__ open, int workers) {
  constexpr int MT = 16 * NT;
  const Open it = open[blockIdx.x];
  if (it.last < 0) return;
  const int g = blockIdx.x / workers, worker = blockIdx.x % workers;
  const Seq s = sequence(a, it.seq);
  const int there = min(MT, s.rows * a.group - it.tile * MT);
  for (int id = threadIdx.x; id < 16 * (DV / 8); id += kThreads) {
    const int r = 16 * blockIdx.y + id / (DV / 8), e = id % (DV / 8) * 8;
    if (r >= there || e >= a.cache.plane[1].dim) continue;
    // the first part is the second of its worker's two, the others are the first of theirs
    auto slot = [&](int w) { return 2 * ((int64_t)g * workers + w) + (w == worker ? 1 : 0); };
    float top = -INFINITY;
    for (int w = worker; w <= it.last; w++) top = fmaxf(top, part_ml[slot(w) * MT + r].x);
    f32x4_t x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
    float sum = 0.0f;
    if (top > -INFINITY) {
#pragma unroll 4
      for (int w = worker; w <= it.last; w++) {
        const float2 ml = part_ml[slot(w) * MT + r];
        const f32x4_t* src = reinterpret_cast<const f32x4_t*>(part + (slot(w) * MT + r) * DV + e);
        const float f = __builtin_amdgcn_exp2f(ml.x - top);
        const f32x4_t p = src[0], q = src[1];
        sum += f * ml.y;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          x[i] += f * p[i];
          y[i] += f * q[i];
        }
      }
    }
    write_row<FMT>(a, s, it.tile * MT + r, g, e, x, y, sum);
  }
}

// ---------------------------------------------------------------------------------------------

template <int FMT, int DK, int DV, int NT, int WAVES>
int launch_shape(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  float* part = (float*)(ws + p.part);
  float2* ml = (float2*)(ws + p.ml);
  Open* open = (Open*)(ws + p.open);
  const unsigned n = (unsigned)p.workers * (unsigned)a.cache.heads;
  const CacheArgs& c = a.cache;
  if (c.page_size % kTile == 0 && c.plane[0].dim == DK && c.plane[1].dim == DV)
    hipLaunchKernelGGL((attend_kernel<FMT, DK, DV, NT, WAVES, true>), dim3(n), dim3(kThreads), 0, stream, a, part, ml, open,
                       p.workers);
  else
    hipLaunchKernelGGL((attend_kernel<FMT, DK, DV, NT, WAVES, false>), dim3(n), dim3(kThreads), 0, stream, a, part, ml, open,
                       p.workers);
  // one unit holds the longest context that the table can: nothing to join
  if (hipGetLastError() != hipSuccess) return MXFP4_ERR_DEVICE;
  if ((int64_t)a.cache.max_pages * a.cache.page_size <= kUnit) return MXFP4_OK;
  hipLaunchKernelGGL((attend_join_kernel<FMT, DV, NT>), dim3(n, NT), dim3(kThreads), 0, stream, a, part, ml, open, p.workers);
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

template <int FMT, int DK, int DV>
int launch_dims(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  if (p.nt == 1) return launch_shape<FMT, DK, DV, 1, attend_waves(DK, 1)>(a, p, ws, stream);
  if (p.nt == 2) return launch_shape<FMT, DK, DV, 2, attend_waves(DK, 2)>(a, p, ws, stream);
  if constexpr (DK <= 192) {
    if (p.nt == 3) return launch_shape<FMT, DK, DV, 3, attend_waves(DK, 3)>(a, p, ws, stream);
    return launch_shape<FMT, DK, DV, 4, attend_waves(DK, 4)>(a, p, ws, stream);
  }
  return MXFP4_ERR_SHAPE;
}

template <int FMT>
int launch_format(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  if (p.dk == 64) return launch_dims<FMT, 64, 64>(a, p, ws, stream);
  if (p.dk == 128) return launch_dims<FMT, 128, 128>(a, p, ws, stream);
  if (p.dk == 192) return launch_dims<FMT, 192, 128>(a, p, ws, stream);
  return launch_dims<FMT, 256, 256>(a, p, ws, stream);
}

}  // namespace
