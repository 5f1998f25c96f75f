// Attention over the block-quantized paged cache: rows see the positions before their sequence's drafts, and of the
// drafts those that a mask or their order leaves.
//
//   out[t, h] = sum_j p_j V[j, g] / sum_j p_j,  p_j = exp2(s_j - m),  s_j = scale log2(e) q[t, h] . K[j, g],  m >= s_j - 8
//
// Work.  The rows of a sequence that share a key head (drafts times query heads of the group) are cut into tiles.  A tile
// and the positions it sees are an item; items are cut into units of positions, and a head's units are dealt out evenly to
// its workers (workgroups), each a contiguous range: a worker's first and last item may be parts, which go to the
// workspace as sums with their maximum and are joined by a second launch, in worker order.  Every worker finds its range
// from the lengths on the device, so nothing about them has to be known on the host.
//
// Both kernels form S^T = K Q^T and O^T = V^T P^T: a row of q is a column of both, so its maximum, sum and rescaling stay in
// one lane (and three others, which hold other positions), and S^T leaves the matrix instruction as P^T enters the next one.
// Values are exact in bf16 (at most six significant bits), so both products are of what the cache holds; V is read back from
// LDS transposed.  The weights are rounded to bf16, as the second product needs them, and their sum is of the rounded ones:
// 2^-8 of each weight, as much as rounding the result to bf16 then costs.  FINE: what that rounding leaves is a second bf16
// term, for another product with the values that are in registers then, and 2^-16 are lost.  It is taken for results in fp32, and
// for up to 16 rows a key head, where memory hides it (32 sequences of up to 3900 positions, 4 rows, MXFP8: 53.5 us without
// and 53.3 with it; over formats, sizes and page sizes 0 to 4 % more).  With more rows it costs more than the third of a bit that
// a bf16 result would gain: 24 rows MXFP8, pages of 16: 78.5 and 80.9 us, MXFP4: 46 and 50; 2 x 1024 rows MXFP8: 164 and 206;
// 12 trees of up to 33 drafts, NVFP4: 67 and 75; 130000 positions, MXFP4: 67 and 76.
// Few rows a key head (up to 32): attend_split.h; more: attend_shared.h.
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
typedef uint16_t u16_a1 __attribute__((aligned(1)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;

template <int FMT>
constexpr int kBlock = FMT == MXFP4_FMT_NVFP4 ? 16 : 32;
template <int FMT>
constexpr int kPerByte = FMT == MXFP4_FMT_MXFP8 ? 1 : 2;

// What a worker leaves for the join, next to its sums: an item that it begins and others go on with.  The entries are the
// items', where there are fewer of those than workers, else the workers', of whose items only the last can go on.
struct Open {
  int32_t tile, seq, worker, rest;  // rest: units of the item behind the worker's range, 0: none
};
struct Totals {
  int64_t units, items;  // of a head; the heads' are alike
};

// The kernels' first argument, read again where it is needed: what the kernels use of it is more than the scalar registers
// hold over their loops, and reading it back from where those are spilled costs vector instructions.
MX_DEV AttendArgs arguments() {
#ifdef __HIP_DEVICE_COMPILE__
  auto* p = (const __attribute__((address_space(4))) AttendArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *p;
#else
  return AttendArgs{};
#endif
}

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

// Of a sequence, tile by tile of MT rows: the positions that some row of the tile sees are below `end`, 2^unit_log of them are
// a unit; a tile has one at least, since its rows are written where nothing is seen too.
template <int MT>
struct Tiles {
  int32_t tile, tiles, end, units;
  int32_t row, part;  // without a mask: the draft of the row behind the tile, and that row's place in its group

  MX_DEV void set(const AttendArgs& a, const Seq& s) {
    const int64_t n = a.mask ? s.drafts : min(s.rows, row + (part > 0));
    const int64_t e = min(s.start + n, (int64_t)a.cache.max_pages * a.cache.page_size);
    end = e < 0 ? 0 : (int32_t)e;
    units = end == 0 ? 1 : ((end - 1) >> a.unit_log) + 1;
  }
  MX_DEV void begin(const AttendArgs& a, const Seq& s) {
    tile = 0;
    tiles = (s.rows * a.group + MT - 1) / MT;
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

template <int MT>
MX_DEV int64_t seq_units(const AttendArgs& a, const Seq& s) {
  Tiles<MT> t;
  t.begin(a, s);
  if (a.mask) return (int64_t)t.tiles * t.units;
  int64_t n = 0;
  while (t.tile < t.tiles) {
    n += t.units;
    t.next(a, s);
  }
  return n;
}

MX_DEV int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }  // known to be the same for the wave
MX_DEV int64_t shfl64(int64_t v, int lane) {
  const int lo = __shfl((int)v, lane), hi = __shfl((int)(v >> 32), lane);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}
MX_DEV int64_t lane64(int64_t v, int lane) {  // the same for the whole wave, and known to be
  const int lo = __builtin_amdgcn_readlane((int)v, lane), hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// n, and that of the lane that DPP control CTRL names, in the rows of 16 lanes of ROWS.
template <int CTRL, int ROWS>
MX_DEV int64_t add_lane(int64_t n) {
  const int lo = __builtin_amdgcn_update_dpp(0, (int)n, CTRL, ROWS, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(n >> 32), CTRL, ROWS, 0xF, false);
  return n + (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}
// Sums over the lanes up to and including each.
MX_DEV int64_t scan_lanes(int64_t n) {
  n = add_lane<0x111, 0xF>(n);  // from 1, 2, 4 and 8 lanes below in a row
  n = add_lane<0x112, 0xF>(n);
  n = add_lane<0x114, 0xF>(n);
  n = add_lane<0x118, 0xF>(n);
  n = add_lane<0x142, 0xA>(n);         // from the last lane of the row below
  return add_lane<0x143, 0xC>(n);      // from lane 31
}

// Of 64 sequences from b0 on: each lane's, and its units and tiles with those of the lanes before.
template <int MT>
struct Scan {
  Seq s;
  int64_t units, tiles;

  MX_DEV Scan(const AttendArgs& a, int b0, int lane) : s{0, 0, 0, 0} {
    if (b0 + lane < a.cache.n_seqs) s = sequence(a, b0 + lane);
    tiles = scan_lanes((s.rows * a.group + MT - 1) / MT);
    units = scan_lanes(s.rows > 0 ? seq_units<MT>(a, s) : 0);
  }
};

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

// The units [first, end) of a head's `all` that a worker has.
MX_DEV void worker_range(int64_t all, int workers, int worker, int64_t& first, int64_t& end) {
  const int64_t used = min((int64_t)workers, all);
  first = end = 0;
  if (worker >= used) return;
  first = all / used * worker + all % used * worker / used;
  end = all / used * (worker + 1) + all % used * (worker + 1) / used;
}

// Where a worker is in its range of units; every wave has the same.
template <int MT>
struct Work {
  int32_t group, worker, b, k0;  // group: of heads; k0: the first of the item's units that are the worker's
  int64_t left;                   // units from there on
  int32_t index;                  // the item's, among all
  Seq s;
  Tiles<MT> ti;

  // False: nothing to do.
  MX_DEV bool begin(const AttendArgs& a, int workers, Open* open, Totals* totals, int lane) {
    const CacheArgs& c = a.cache;
    const int groups = c.heads >> a.heads_log;
    // Workgroups go to the eight XCDs in turn: a worker's heads, which read pieces of the same tokens, share one.
    if (workers % 8 == 0) {
      const int i = blockIdx.x / 8;
      group = i % groups;
      worker = i / groups * 8 + blockIdx.x % 8;
    } else {
      group = blockIdx.x % groups;
      worker = blockIdx.x / groups;
    }
    Scan<MT> first(a, 0, lane);
    int64_t all = lane64(first.units, 63), items = lane64(first.tiles, 63), u, u1;
    for (int b0 = 64; b0 < c.n_seqs; b0 += 64) {
      const Scan<MT> more(a, b0, lane);
      all += lane64(more.units, 63);
      items += lane64(more.tiles, 63);
    }
    if (threadIdx.x == 0) {
      if (!a.open_items) open[(int64_t)group * workers + worker] = Open{0, 0, 0, 0};
      if (worker == 0 && group == 0) *totals = Totals{all, items};
    }
    worker_range(all, workers, worker, u, u1);
    if (u == u1) return false;
    b = 0;
    index = 0;
    int64_t item = 0;
    uint64_t past;
    while (!(past = __ballot(item + first.units > u))) {
      if (b + 64 >= c.n_seqs) return false;  // not with cu_rows and start that stay
      item += lane64(first.units, 63);
      index += (int32_t)lane64(first.tiles, 63);
      b += 64;
      first = Scan<MT>(a, b, lane);
    }
    const int l = __ffsll((unsigned long long)past) - 1;
    b += l;
    if (l > 0) {
      item += lane64(first.units, l - 1);
      index += (int32_t)lane64(first.tiles, l - 1);
    }
    const auto of = [&](int32_t v) { return __builtin_amdgcn_readlane(v, l); };
    s = Seq{of(first.s.first), of(first.s.drafts), of(first.s.rows), of(first.s.start)};
    ti.begin(a, s);
    while (item + ti.units <= u) {
      item += ti.units;
      index++;
      ti.next(a, s);
    }
    k0 = (int32_t)(u - item);
    left = u1 - u;
    return true;
  }
  // The end of the item's units that are the worker's.
  MX_DEV int32_t k1() const { return (int32_t)min((int64_t)ti.units, k0 + left); }
  // The same, in scalar registers again after a loop's end that the compiler takes to differ between lanes.
  MX_DEV void settle() {
    group = uniform(group);
    worker = uniform(worker);
    b = uniform(b);
    index = uniform(index);
    k0 = uniform(k0);
    left = lane64(left, 0);
    s = Seq{uniform(s.first), uniform(s.drafts), uniform(s.rows), uniform(s.start)};
    ti.tile = uniform(ti.tile);
    ti.tiles = uniform(ti.tiles);
    ti.end = uniform(ti.end);
    ti.units = uniform(ti.units);
    ti.row = uniform(ti.row);
    ti.part = uniform(ti.part);
  }
  // On to the next item.  False: the range ends.
  MX_DEV bool next(const AttendArgs& a) {
    left -= k1() - k0;
    if (left <= 0) return false;
    k0 = 0;
    index++;
    ti.next(a, s);
    if (ti.tile >= ti.tiles) {
      do s = sequence(a, ++b);
      while (s.rows == 0);
      ti.begin(a, s);
    }
    return true;
  }
  // What the join needs to know of an item that begins here.
  MX_DEV void leave_open(const AttendArgs& a, Open* open, int workers) const {
    if (threadIdx.x != 0 || k0 != 0) return;
    const Open o = {ti.tile, b, worker, ti.units - k1()};
    if (a.open_items) {
      if (index < a.open_items) open[(int64_t)group * a.open_items + index] = o;  // there are no more with cu_rows in order
    } else if (o.rest > 0)
      open[(int64_t)group * workers + worker] = o;
  }
};

// ---------------------------------------------------------------------------------------------
// Softmax.

// What the scores are multiplied by before exp2.  Not 0, so that its product with a hidden position's -inf is one: the smallest
// number that binary32 has, with which no score reaches 2^-20.  Finite: the host has seen to that.
template <int FMT>
MX_DEV float score_scale(const AttendArgs& a) {
  const float s = a.scale == 0.0f ? 1.0f : fabsf(a.scale);
  return fmaxf(s * 1.44269504f / (FMT == MXFP4_FMT_NVFP4 ? a.cache.plane[0].gs : 1.0f), 0x1p-149f);
}

// A wave's 16 NT rows of q, a lane's elements first(i) to first(i) + 7 of them.  `load` asks for places that are there
// throughout, so that no wait for what was asked for before waits for q too; `finish` waits.
template <int NT, int STEPS>
struct Query {
  bf16x8_t q[NT][STEPS];
  int32_t draft[NT];  // of this lane's columns; -1: no such row

  template <typename F>
  MX_DEV void load(const AttendArgs& a, const Seq& s, int32_t row0, int g, F first) {
    const CachePlane& query = a.cache.plane[0];
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const int32_t r = row0 + 16 * n + (threadIdx.x & 15), d = (uint32_t)r / (uint32_t)a.group;
      draft[n] = d < s.rows ? d : -1;
      const uint16_t* src = (const uint16_t*)query.rows + (int64_t)(s.first + min(d, s.rows - 1)) * query.ldt +
                            (g * a.group + (r - d * a.group)) * query.ldh;
#pragma unroll
      for (int i = 0; i < STEPS; i++) q[n][i] = *reinterpret_cast<const bf16x8_t*>(src + (first(i) < query.dim ? first(i) : 0));
    }
  }
  // The scale's sign goes to q, and with a scale of 0 it is 0.
  template <typename F>
  MX_DEV void finish(const AttendArgs& a, F first) {
    const uint32_t sign = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int i = 0; i < STEPS; i++) {
        const uint32_t keep = draft[n] >= 0 && first(i) < a.cache.plane[0].dim && a.scale != 0.0f ? ~0u : 0u;
        u32x4_t x = __builtin_bit_cast(u32x4_t, q[n][i]);
#pragma unroll
        for (int j = 0; j < 4; j++) x[j] = (x[j] & keep) ^ (sign & keep);
        q[n][i] = __builtin_bit_cast(bf16x8_t, x);
      }
  }
};

// Weights of 16 KT positions, in one or (FINE) two terms.
template <int NT, int KT, bool FINE>
struct Weights {
  bf16x8_t p[NT][KT / 2], rest[FINE ? NT : 1][FINE ? KT / 2 : 1];
};

// The sums of a wave's 16 NT rows, of their weights too; the exponents' subtrahend m, and the score from which on it is
// raised.
template <int NT, int VT, bool FINE>
struct Rows {
  f32x4_t o[NT][VT], l[NT];
  float m[NT], limit[NT];

  MX_DEV void clear() {
#pragma unroll
    for (int n = 0; n < NT; n++) {
      m[n] = limit[n] = -INFINITY;
      l[n] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < VT; v++) o[n][v] = f32x4_t{0, 0, 0, 0};
    }
  }

  // Scores of 16 KT positions to weights in bf16.  m is raised, and all sums with it, where a score is over it by more than
  // 8: weights stay below 2^8, and most tiles need no maximum over the row's four lanes and no rescaling.
  template <int KT>
  MX_DEV void weights(const f32x4_t (&s)[NT][KT], float sc, Weights<NT, KT, FINE>& to) {
    bool over = false;
    float top[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) {
      top[n] = s[n][0][0];
#pragma unroll
      for (int i = 1; i < 4 * KT; i++) top[n] = fmaxf(top[n], s[n][i >> 2][i & 3]);
      over = over || top[n] > limit[n];
    }
    if (__any(over)) {
#pragma unroll
      for (int n = 0; n < NT; n++) {
        top[n] = fmaxf(top[n], __shfl_xor(top[n], 16));
        top[n] = fmaxf(top[n], __shfl_xor(top[n], 32));
        const float now = fmaxf(m[n], top[n] * sc);
        const float keep = now > -INFINITY ? __builtin_amdgcn_exp2f(m[n] - now) : 1.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) l[n][i] *= keep;
#pragma unroll
        for (int v = 0; v < VT; v++)
#pragma unroll
          for (int i = 0; i < 4; i++) o[n][v][i] *= keep;
        m[n] = now;
        limit[n] = (now + 8.0f) / sc;
      }
    }
    // the weights' sum is taken of them as they are rounded, by the matrix instruction
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const float by = m[n] > -INFINITY ? -m[n] : 0.0f;  // nothing seen yet
#pragma unroll
      for (int h = 0; h < KT / 2; h++) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = __builtin_amdgcn_exp2f(fmaf(s[n][2 * h + (i >> 2)][i & 3], sc, by));
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const bf16x2_t two = __builtin_convertvector(f32x2_t{w[i], w[i + 1]}, bf16x2_t);
          to.p[n][h][i] = two[0];
          to.p[n][h][i + 1] = two[1];
          if constexpr (FINE) {
            const bf16x2_t rest = __builtin_convertvector(f32x2_t{w[i] - (float)two[0], w[i + 1] - (float)two[1]}, bf16x2_t);
            to.rest[n][h][i] = rest[0];
            to.rest[n][h][i + 1] = rest[1];
          }
        }
        l[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, to.p[n][h], l[n], 0, 0, 0);
        if constexpr (FINE) l[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, to.rest[n][h], l[n], 0, 0, 0);
      }
    }
  }

  // O^T += V^T P^T for 32 positions: their values are rows of LDS, `stride` elements apart.
  template <int AHEAD, int KT>
  MX_DEV void add_values(const uint16_t* v0, int stride, const Weights<NT, KT, FINE>& w, int h, int lane) {
    // two blocks of four positions by sixteen elements a group of sixteen lanes, transposed
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
    const int col = lane & 15, kg = lane >> 4;
    const uint16_t* src = v0 + (4 * kg + (col >> 2)) * stride + 4 * (col & 3);
    // AHEAD columns of tiles are read ahead of the products of the AHEAD before
    static_assert(VT % AHEAD == 0, "whole steps");
    s16x4_t x[2][AHEAD][2];
    const auto read = [&](int v0) {
#pragma unroll
      for (int v = 0; v < AHEAD; v++)
#pragma unroll
        for (int y = 0; y < 2; y++)
          x[v0 / AHEAD & 1][v][y] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(src + 16 * y * stride + 16 * (v0 + v)));
    };
    read(0);
#pragma unroll
    for (int v0 = 0; v0 < VT; v0 += AHEAD) {
      if (v0 + AHEAD < VT) read(v0 + AHEAD);
      if (AHEAD > 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int v = 0; v < AHEAD; v++) {
        const auto& t = x[v0 / AHEAD & 1][v];
        const bf16x8_t both = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(t[0], t[1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
        for (int n = 0; n < NT; n++) {
          o[n][v0 + v] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(both, w.p[n][h], o[n][v0 + v], 0, 0, 0);
          if constexpr (FINE) o[n][v0 + v] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(both, w.rest[n][h], o[n][v0 + v], 0, 0, 0);
        }
      }
      if (AHEAD > 1) __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Adds the sums of the rows of column tile n, brought to the maximum `top`, to those in LDS (first: puts them there).
  MX_DEV void join(int n, float* sums, int stride, float top, bool first, int lane) const {
    const float f = top > -INFINITY ? __builtin_amdgcn_exp2f(m[n] - top) : 0.0f;
    float* dst = sums + (lane & 15) * stride + 4 * (lane >> 4);
#pragma unroll
    for (int v = 0; v < VT; v++) {
      f32x4_t x = o[n][v];
#pragma unroll
      for (int i = 0; i < 4; i++) x[i] *= f;
      if (!first) {
        const f32x4_t y = *reinterpret_cast<const f32x4_t*>(dst + 16 * v);
#pragma unroll
        for (int i = 0; i < 4; i++) x[i] += y[i];
      }
      *reinterpret_cast<f32x4_t*>(dst + 16 * v) = x;
    }
  }
};

// Takes from the scores of a tile's 16 KT positions from `base` on what the rows do not see: there, bad: bits of positions
// that have a page, and whose values are not finite.
template <int NT, int KT>
MX_DEV void hide(const AttendArgs& a, const Seq& s, const int32_t (&draft)[NT], int32_t base, uint64_t there, uint64_t bad, int kg,
                 f32x4_t (&sv)[NT][KT]) {
  const int64_t first = (int64_t)base - s.start + 4 * kg;  // as a draft: the first position of this lane
#pragma unroll
  for (int n = 0; n < NT; n++) {
    // drafts from `most` on are not seen
    const int64_t most = draft[n] < 0 ? INT64_MIN : a.mask ? min(s.drafts, a.mask_cols) : (int64_t)draft[n] + 1;
    const uint8_t* mask = a.mask + (int64_t)(s.first + max(draft[n], 0)) * a.ld_mask;
    uint32_t seen = 0, nan = 0;  // bit 4 t + i; a loop, which costs no registers of the one around
#pragma unroll 1
    for (int t = 0; t < KT; t++) {
      uint32_t four = (uint32_t)(there >> (16 * t + 4 * kg)) & 15u;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int64_t j = first + 16 * t + i;
        if (j >= most || (j >= 0 && a.mask && !mask[j])) four &= ~(1u << i);
      }
      seen |= four << (4 * t);
      nan |= ((uint32_t)(bad >> (16 * t + 4 * kg)) & four) << (4 * t);
    }
    // with masks of bits, which stay in vector registers
#pragma unroll
    for (int t = 0; t < KT; t++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)seen, 4 * t + i, 1), none = __builtin_amdgcn_sbfe((int)nan, 4 * t + i, 1);
        const uint32_t x = __float_as_uint(sv[n][t][i]) | (none & 0x7FFFFFFFu);
        sv[n][t][i] = __uint_as_float((x & keep) | (~keep & 0xFF800000u));
      }
  }
}

// The result of `n` of an item's rows from `r0` on for key head g, or their part for the join, by `threads` threads: their
// sums in LDS, and the maxima and sums of weights of the `parts` waves that had them, MT of each a wave.
template <int FMT, int DV, int MT>
MX_DEV void write_item(const AttendArgs& a, const Work<MT>& w, int g, int workers, int r0, int n, const float* sums, const float* ms,
                       const float* ls, int parts, int thread, int threads, float* part, float2* part_ml) {
  const int there = min(n, w.s.rows * a.group - w.ti.tile * MT - r0);
  const bool whole = w.k0 == 0 && w.k1() == w.ti.units;
  const int64_t slot = 2 * ((int64_t)g * workers + w.worker) + (w.k0 == 0 ? 1 : 0);
  for (int id = thread; id < there * (DV / 8); id += threads) {
    const int r = r0 + id / (DV / 8), e = id % (DV / 8) * 8;
    float top = ms[r], sum = 0.0f;
    for (int x = 1; x < parts; x++) top = fmaxf(top, ms[x * MT + r]);
    // a row without a maximum has sums of 0, or of NaN where all its scores are
    for (int x = 0; x < parts; x++) sum += ls[x * MT + r] * (top > -INFINITY ? __builtin_amdgcn_exp2f(ms[x * MT + r] - top) : 1.0f);
    const f32x4_t* src = reinterpret_cast<const f32x4_t*>(sums + (r - r0) * (DV + 4) + e);
    const f32x4_t x = src[0], y = src[1];
    if (!whole) {
      f32x4_t* dst = reinterpret_cast<f32x4_t*>(part + (slot * MT + r) * DV + e);
      dst[0] = x;
      dst[1] = y;
      if (e == 0) part_ml[slot * MT + r] = float2{top, sum};
    } else if (e < a.cache.plane[1].dim) {
      write_row<FMT>(a, w.s, w.ti.tile * MT + r, g, e, x, y, sum);
    }
  }
}

}  // namespace
