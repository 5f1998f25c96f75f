// Paged cache in a block format: rows quantized as they are written through a page table, and read back.
#include <hip/hip_runtime.h>

#include "cache_slots.h"
#include "ops.h"

#define MX_DEV __device__ __forceinline__

namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int64_t kMaxGrid = 65536;
constexpr int64_t kFull = 32768;  // waves, beyond what is resident at a time, that keep the chip evenly loaded

template <int CTRL>
MX_DEV uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// A unit is eight consecutive elements of a row's plane; a block is four units (NVFP4: two), which sit in
// neighbouring lanes.
template <int FMT>
constexpr int kUnitsPerBlock = FMT == MXFP4_FMT_NVFP4 ? 2 : 4;
template <int FMT>
constexpr int kUnitBytes = FMT == MXFP4_FMT_MXFP8 ? 8 : 4;

struct Unit {
  uint32_t q[2];  // 4-bit formats: q[0]
  uint32_t s;
};

// The unit's codes and its block's scale: the rules of the quantizers (quantize.hip) and of the MXFP8
// activations.  All lanes of a block take part.
template <int FMT>
MX_DEV Unit encode(u32x4_t v, float gs) {
  Unit u = {};
  const uint32_t w[4] = {v[0], v[1], v[2], v[3]};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  m = max(m, dpp<0xB1>(m));                                   // lane ^ 1
  if (FMT != MXFP4_FMT_NVFP4) m = max(m, dpp<0x4E>(m));  // lane ^ 2
  if (FMT == MXFP4_FMT_NVFP4) {
    const float sf = gs * (__uint_as_float(m << 16) * 0x1.555556p-3f);  // the binary32 nearest to 1/6
    s16x2_t sb = s16x2_t{0, 0};
    sb = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(sb, fminf(sf, 448.0f), 0.0f, 1.0f, false);
    u.s = __builtin_bit_cast(uint32_t, sb) & 0xFFu;
    const float held = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(u.s, 1.0f, false)[0];
    const float rs = held > 0.0f ? gs / held : 0.0f;
    uint32_t p = 0;
    auto lo = [&](int i) { return __uint_as_float(w[i] << 16) * rs; };
    auto hi = [&](int i) { return __uint_as_float(w[i] & 0xFFFF0000u) * rs; };
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, lo(0), hi(0), 1.0f, 0);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, lo(1), hi(1), 1.0f, 1);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, lo(2), hi(2), 1.0f, 2);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, lo(3), hi(3), 1.0f, 3);
    u.q[0] = p;
    return u;
  }
  // E8M0: the biased exponent of the maximum, one more from a significand of 1.75 on, less the elements'
  // largest exponent (E2M1: 2, E4M3: 8)
  constexpr uint32_t top = FMT == MXFP4_FMT_MXFP8 ? 8u : 2u;
  const uint32_t bits = m << 16, b = ((bits + (1u << 21)) >> 23) & 0xFFu;
  u.s = bits == 0u || b < top ? 0u : min(b - top, 254u);
  const float sc = __uint_as_float(u.s << 23);
  if (FMT == MXFP4_FMT_MXFP4) {
    uint32_t p = 0;
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(p, __builtin_bit_cast(bf16x2_t, w[0]), sc, 0);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(p, __builtin_bit_cast(bf16x2_t, w[1]), sc, 1);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(p, __builtin_bit_cast(bf16x2_t, w[2]), sc, 2);
    p = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(p, __builtin_bit_cast(bf16x2_t, w[3]), sc, 3);
    u.q[0] = p;
  } else {
#pragma unroll
    for (int d = 0; d < 2; d++) {
      s16x2_t p = s16x2_t{0, 0};
      p = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(p, __builtin_bit_cast(bf16x2_t, w[2 * d]), sc, false);
      p = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(p, __builtin_bit_cast(bf16x2_t, w[2 * d + 1]), sc, true);
      u.q[d] = __builtin_bit_cast(uint32_t, p);
    }
  }
  return u;
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));
MX_DEV uint32_t bf16_pair(f32x2_t v) {  // nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

template <int FMT>
MX_DEV u32x4_t decode(const uint32_t* q, uint32_t s, float gs) {
  u32x4_t o;
  if (FMT == MXFP4_FMT_MXFP4) {
    const float sc = __uint_as_float(s << 23);
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[0], sc, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[0], sc, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[0], sc, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[0], sc, 3));
  } else if (FMT == MXFP4_FMT_MXFP8) {
    const float sc = __uint_as_float(s << 23);
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[0], sc, false));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[0], sc, true));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[1], sc, false));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[1], sc, true));
  } else {
    // one division a block: scale / global scale, rounded to binary32, times the code.  Under a small global scale the
    // quotient may be past binary32's range where its product with a code of 0 or 1/2 is not: 2^-30 keeps it inside
    // (448 * 2^-30 over the smallest number is below 2^128), and the code takes it back.
    const bool small = gs < 1.0f;
    const float up = small ? 0x1p30f : 1.0f;
    const float f = __builtin_amdgcn_cvt_f32_fp8((int)s, 0) * (small ? 0x1p-30f : 1.0f) / gs;
    auto two = [&](auto v) { return bf16_pair(f32x2_t{v[0] * f, v[1] * f}); };
    o[0] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], up, 0));
    o[1] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], up, 1));
    o[2] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], up, 2));
    o[3] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], up, 3));
  }
  return o;
}

// A wave takes `chunk` rows at a time: its lanes look their slots up side by side (one chain of searches a chunk
// instead of one a row), then run over the chunk's units of both planes, kBatch of them on their way in each lane.
// The rows of a plane are whole blocks, so a block's units stay in neighbouring lanes.
//
// Both directions are bound by memory: a value costs 2 bytes on one side and 1.03 (MXFP8), 0.56 or 0.53 on the other.
// Measured: 93600 rows of 2 x 1024 values read back from MXFP8, 581 MB, 126 us (4.6 TB/s, 0.9 of a large copy's
// rate); with a wave a row and 8-byte accesses in a loop 165 us, 8 rows a wave 146 us, 1 row 134 us, batches of 2 or 8
// 170 and 143 us; streaming (nontemporal) accesses take 3 to 6 % off.  18126 rows of 8 x 320 to and from NVFP4, 119 MB
// each way: written in 32 us (3.7 TB/s; scales go out a byte at a time, and rows come in by ordinary loads), read back in
// 23.6 us (5.0 TB/s).
constexpr int kBatch = 4;

template <int FMT, bool WRITE, bool SPREAD>  // SPREAD: heads apart in some plane's rows
__global__ __launch_bounds__(kThreads) void cache_kernel(CacheArgs a, int chunk) {
  const int lane = threadIdx.x & 63;
  const uint32_t u0 = (uint32_t)a.heads * (a.plane[0].dim / 8), u1 = (uint32_t)a.heads * (a.plane[1].dim / 8);
  const uint32_t row_units = u0 + u1;
  const int64_t waves = (int64_t)gridDim.x * (kThreads / 64);
  for (int64_t c = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); c * chunk < a.rows; c += waves) {
    const int64_t t0 = c * chunk;
    const int rows = (int)min((int64_t)chunk, a.rows - t0);
    int64_t slot = -2;
    if (lane < rows) slot = slot_of(a, t0 + lane);
    const uint32_t units = rows * row_units;
    for (uint32_t first = 0; first < units; first += 64 * kBatch) {
      u32x4_t x[kBatch];
      uint32_t q[kBatch][2], sc[kBatch];
      int64_t at[kBatch], unit[kBatch];  // at: element of the rows; unit: of the plane, -1: zeros, -2: none
      bool second[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; i++) {
        const uint32_t id = min(first + 64 * i + lane, units - 1);
        const uint32_t row = chunk == 1 ? 0 : id / row_units;
        uint32_t u = id - row * row_units;
        second[i] = u >= u0;
        u -= second[i] ? u0 : 0;
        const CachePlane &p0 = a.plane[0], &p1 = a.plane[1];
        const int64_t s = __shfl(slot, (int)row);
        const int64_t ldt = second[i] ? p1.ldt : p0.ldt;
        at[i] = (t0 + row) * ldt;
        if (SPREAD) {
          const uint32_t per_head = (uint32_t)(second[i] ? p1.dim : p0.dim) / 8, head = u / per_head;
          at[i] += head * (second[i] ? p1.ldh : p0.ldh) + (u - head * per_head) * 8;
        } else {
          at[i] += u * 8;
        }
        unit[i] = s < 0 ? s : s * (second[i] ? u1 : u0) + u;
        if (first + 64 * i + lane >= units) unit[i] = -2;
        if (WRITE) {
          // every lane reads (clamped: its block's maximum is taken over four lanes), those with a slot write
          x[i] = u32x4_t{0, 0, 0, 0};
          if (unit[i] >= 0)
            x[i] = *reinterpret_cast<const u32x4_t*>((const uint16_t*)(second[i] ? p1.rows : p0.rows) + at[i]);
        } else {
          const int64_t from = unit[i] < 0 ? 0 : unit[i];
          q[i][0] = q[i][1] = sc[i] = 0;
          if (unit[i] >= 0) {
            const uint8_t* src = (second[i] ? p1.q : p0.q) + from * kUnitBytes<FMT>;
            if (FMT == MXFP4_FMT_MXFP8) {
              const u32x2_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(src));
              q[i][0] = w[0];
              q[i][1] = w[1];
            } else {
              q[i][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(src));
            }
            sc[i] = (second[i] ? p1.s : p0.s)[from / kUnitsPerBlock<FMT>];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; i++) {
        const CachePlane &p0 = a.plane[0], &p1 = a.plane[1];
        const float gs = second[i] ? p1.gs : p0.gs;
        if (WRITE) {
          const Unit e = encode<FMT>(x[i], gs);
          if (unit[i] >= 0) {
            uint8_t* dst = (second[i] ? p1.q : p0.q) + unit[i] * kUnitBytes<FMT>;
            if (FMT == MXFP4_FMT_MXFP8)
              *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{e.q[0], e.q[1]};
            else
              *reinterpret_cast<uint32_t*>(dst) = e.q[0];
            if (unit[i] % kUnitsPerBlock<FMT> == 0)
              (second[i] ? p1.s : p0.s)[unit[i] / kUnitsPerBlock<FMT>] = (uint8_t)e.s;
          }
        } else if (unit[i] >= -1) {
          const u32x4_t v = decode<FMT>(q[i], sc[i], gs);
          u32x4_t* dst = reinterpret_cast<u32x4_t*>((uint16_t*)(second[i] ? p1.rows : p0.rows) + at[i]);
          const u32x4_t zero = {0, 0, 0, 0}, out = unit[i] < 0 ? zero : v;
          __builtin_nontemporal_store(out, dst);
        }
      }
    }
  }
}

template <int FMT, bool WRITE>
void launch_fmt(const CacheArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.heads * (a.plane[0].dim + a.plane[1].dim) / 8;
  // rows of a chunk: as many as leave kFull waves, as fill a wave's batch at least, at most one a lane
  int64_t chunk = a.rows / kFull;
  const int64_t fill = (64 * kBatch + units - 1) / units;
  chunk = chunk < fill && a.rows / fill >= 256 ? fill : chunk;
  chunk = chunk < 1 ? 1 : chunk > 64 ? 64 : chunk;
  while (chunk > 1 && chunk * units > (1 << 24)) chunk /= 2;
  const int64_t n = (a.rows + chunk * (kThreads / 64) - 1) / (chunk * (kThreads / 64));
  const dim3 grid((unsigned)(n < kMaxGrid ? n : kMaxGrid));
  const bool spread = (a.heads > 1) && (a.plane[0].ldh != a.plane[0].dim || (a.plane[1].dim && a.plane[1].ldh != a.plane[1].dim));
  if (spread)
    hipLaunchKernelGGL((cache_kernel<FMT, WRITE, true>), grid, dim3(kThreads), 0, stream, a, (int)chunk);
  else
    hipLaunchKernelGGL((cache_kernel<FMT, WRITE, false>), grid, dim3(kThreads), 0, stream, a, (int)chunk);
}

template <bool WRITE>
int launch(int fmt, const CacheArgs& a, hipStream_t stream) {
  if (fmt == MXFP4_FMT_MXFP4)
    launch_fmt<MXFP4_FMT_MXFP4, WRITE>(a, stream);
  else if (fmt == MXFP4_FMT_NVFP4)
    launch_fmt<MXFP4_FMT_NVFP4, WRITE>(a, stream);
  else
    launch_fmt<MXFP4_FMT_MXFP8, WRITE>(a, stream);
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

}  // namespace

int launch_cache_write(int fmt, const CacheArgs& a, hipStream_t stream) { return launch<true>(fmt, a, stream); }
int launch_cache_read(int fmt, const CacheArgs& a, hipStream_t stream) { return launch<false>(fmt, a, stream); }
