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

MX_DEV uint32_t bf16_bits(float f) {  // round to nearest even, infinities pass
  const uint32_t u = __float_as_uint(f);
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
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
    // code * scale is exact in binary32; one rounding by the division, one to bf16
    const float f = __builtin_amdgcn_cvt_f32_fp8((int)s, 0);
    auto two = [&](auto v) { return bf16_bits(v[0] * f / gs) | (bf16_bits(v[1] * f / gs) << 16); };
    o[0] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 0));
    o[1] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 1));
    o[2] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 2));
    o[3] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 3));
  }
  return o;
}

// 2^LOG threads a row, each taking every 2^LOG-th unit of both planes.
template <int FMT, bool WRITE>
__global__ __launch_bounds__(kThreads) void cache_kernel(CacheArgs a, int log_tpr) {
  const int tpr = 1 << log_tpr;
  const int in_row = threadIdx.x & (tpr - 1);
  const int per_block = kThreads >> log_tpr;
  for (int64_t t = (int64_t)blockIdx.x * per_block + (threadIdx.x >> log_tpr); t < a.rows;
       t += (int64_t)gridDim.x * per_block) {
    const int64_t slot = slot_of(a, t);
    if (slot == -2 || (WRITE && slot < 0)) continue;
#pragma unroll
    for (int which = 0; which < 2; which++) {
      const CachePlane& p = a.plane[which];
      const int per_head = p.dim >> 3, units = per_head * a.heads;
      const int64_t ubase = slot * units;
      uint16_t* row = (uint16_t*)p.rows + t * p.ldt;
      for (int u = in_row; u < units; u += tpr) {
        const int head = u / per_head;
        u32x4_t* x = reinterpret_cast<u32x4_t*>(row + head * p.ldh + (u - head * per_head) * 8);
        uint8_t* q = p.q + (ubase + u) * kUnitBytes<FMT>;
        uint8_t* s = p.s + (ubase + u) / kUnitsPerBlock<FMT>;
        if (WRITE) {
          const Unit e = encode<FMT>(*x, p.gs);
          if (FMT == MXFP4_FMT_MXFP8)
            *reinterpret_cast<u32x2_t*>(q) = u32x2_t{e.q[0], e.q[1]};
          else
            *reinterpret_cast<uint32_t*>(q) = e.q[0];
          if (u % kUnitsPerBlock<FMT> == 0) *s = (uint8_t)e.s;
        } else if (slot < 0) {
          *x = u32x4_t{0, 0, 0, 0};
        } else {
          uint32_t w[2] = {*reinterpret_cast<const uint32_t*>(q), 0};
          if (FMT == MXFP4_FMT_MXFP8) w[1] = *reinterpret_cast<const uint32_t*>(q + 4);
          *x = decode<FMT>(w, *s, p.gs);
        }
      }
    }
  }
}

template <bool WRITE>
int launch(int fmt, const CacheArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.heads * (a.plane[0].dim > a.plane[1].dim ? a.plane[0].dim : a.plane[1].dim) / 8;
  int log_tpr = 2;  // a block's lanes together
  while (log_tpr < 6 && (int64_t(1) << log_tpr) < units) log_tpr++;
  const int64_t n = (a.rows + (kThreads >> log_tpr) - 1) / (kThreads >> log_tpr);
  const dim3 grid((unsigned)(n < kMaxGrid ? n : kMaxGrid));
  if (fmt == MXFP4_FMT_MXFP4)
    hipLaunchKernelGGL((cache_kernel<MXFP4_FMT_MXFP4, WRITE>), grid, dim3(kThreads), 0, stream, a, log_tpr);
  else if (fmt == MXFP4_FMT_NVFP4)
    hipLaunchKernelGGL((cache_kernel<MXFP4_FMT_NVFP4, WRITE>), grid, dim3(kThreads), 0, stream, a, log_tpr);
  else
    hipLaunchKernelGGL((cache_kernel<MXFP4_FMT_MXFP8, WRITE>), grid, dim3(kThreads), 0, stream, a, log_tpr);
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

}  // namespace

int launch_cache_write(int fmt, const CacheArgs& a, hipStream_t stream) { return launch<true>(fmt, a, stream); }
int launch_cache_read(int fmt, const CacheArgs& a, hipStream_t stream) { return launch<false>(fmt, a, stream); }
