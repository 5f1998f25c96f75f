// Matrix-vector products with 4-bit weights in the standard layout: y = x W^T (/ global scale) + b for a few
// rows of x, and the same product of every routed pair with its expert's matrix (with SwiGLU on request).
//
// What bounds them is the weights' way from memory (0.53 or 0.56 bytes each, read once per 16 rows of x), and for small
// matrices the chain of a launch, one load, one join.  So the weights are dequantized to bf16 in registers (exact: two
// significant bits times a power of two, or times four bits) and multiplied on the matrix cores whatever the number of
// rows, the waves of a workgroup share K and meet once, and nothing is set up or waited for before the first load of
// weights but, in the expert form, the expert's number.  NVFP4's dequantization takes four instructions a pair of weights
// (MXFP4: one) and then bounds small numbers of rows: there the scale goes behind the matrix instruction (tile_sums_nv).
// Measured (kernel alone, averages; weights from memory, in brackets from the last-level cache):
//   1 x 7168 x 7168           MXFP4  8.5 us (7.8; 3.2 TB/s from memory), NVFP4 10.6 us (9.6; 2.7 TB/s)
//   1 x 28672 x 7168          MXFP4 24.8 us (24.1; 4.4 TB/s), NVFP4 23.8 us (23.5; 4.9 TB/s)
//   16 x 7168 x 2048          MXFP4  6.4 us (5.2)
//   16 x 7168 x 7168          MXFP4 12.5 us (10.8), NVFP4 15.1 us (12.8): every workgroup reads all of x
//   64 tokens, top-8 of 128   2048 x 768: MXFP4 28 us, NVFP4 32 us; 1536 x 2048 with SwiGLU 47 and 56 us (4.5, 4.0 TB/s)
//   16 tokens, the latter     MXFP4 30 us, NVFP4 38 us
//   1 token, the latter       MXFP4 8.3 us (1.6 TB/s), NVFP4 9.5 us: eight waves are launched for four blocks of K
// Tried and slower: scales a byte at a time beside the codes (a third of the time); x 16 bytes a row from memory (half of
// the time at 16 rows); scales and x of the whole workgroup in LDS behind a barrier (7168 x 7168: 11 to 14 us); a ring or a
// second set of registers for the next block (spills, or fewer waves: 12 to 18 us).
#include <hip/hip_runtime.h>

#include "ops.h"

#define MX_DEV __device__ __forceinline__

namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
// rows of NVFP4 weights start on 8-byte boundaries
typedef u32x4_t u32x4_a8 __attribute__((aligned(8)));

constexpr int kStep = 128;     // K elements of one step: 32 for each quarter of the wave
constexpr int64_t kFull = 2048;      // waves that fill the chip (1 x 7168 x 7168 NVFP4: 9.5 us, with 1024 and 4096 11.0, 11.4)
constexpr int64_t kFullWide = 6144;  // waves of four tiles (1536 x 2048 with SwiGLU, NVFP4: 56 us, with 2048 60 us)
constexpr int64_t kWide = 4096;      // tiles that are enough for a wave to take four of them
template <int CTRL>
MX_DEV float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Eight weights (one dword of codes) as bf16, times their scale: exact.
template <int FMT>
MX_DEV bf16x8_t dequant8(uint32_t codes, float scale) {
  u32x4_t out;
  if (FMT == MXFP4_FMT_MXFP4) {
    out[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    out[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    out[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    out[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  } else {
    // the product has at most six significant bits, so the upper halves of its binary32 form are all of it
    auto two = [&](auto v) {
      return __builtin_amdgcn_perm(__float_as_uint(v[1] * scale), __float_as_uint(v[0] * scale), 0x07060302u);
    };
    out[0] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0));
    out[1] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1));
    out[2] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2));
    out[3] = two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3));
  }
  return __builtin_bit_cast(bf16x8_t, out);
}

// The codes of 32 elements, from byte `at` of a row on.  NVFP4 rows start on 8-byte boundaries.
template <int FMT>
MX_DEV u32x4_t load_codes(const uint8_t* q, uint32_t at) {
  if (FMT == MXFP4_FMT_MXFP4) return *reinterpret_cast<const u32x4_t*>(q + at);
  return *reinterpret_cast<const u32x4_a8*>(q + at);
}

// Past a row's end its last 32 elements are loaded again (nothing out of bounds: x is zero there).  NVFP4 rows may end
// inside the 32 (K % 32 == 16): then what was loaded starts 16 elements early, and moves here.
template <int FMT>
MX_DEV void settle(u32x4_t& q, int k, int K) {
  if (FMT == MXFP4_FMT_MXFP4 || K % 32 == 0) return;
  const bool early = k == K - 16;
  q[0] = early ? q[2] : q[0];
  q[1] = early ? q[3] : q[1];
}

MX_DEV float bias_at(const void* b, int fp32, int64_t i) {
  return fp32 ? ((const float*)b)[i] : __uint_as_float((uint32_t)((const uint16_t*)b)[i] << 16);
}

MX_DEV uint16_t to_bf16(float f) {  // round to nearest even; infinities pass, NaN stays NaN
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

template <int FMT>
constexpr int kBlock = FMT == MXFP4_FMT_NVFP4 ? 16 : 32;

// The weights of R tiles of 16 rows: where each tile's codes and scales start (the same for all lanes), how many bytes
// of scales the tensor has from there on, and the lane's row of the tile (rows past the last repeat it).
template <int R>
struct Tiles {
  const uint8_t *q[R], *s[R];
  int32_t s_left[R];
  uint32_t row[R];
};

// DW dwords from byte `at` on of `left` bytes, of which the first `n` are the row's own (at < left where n > 0); what
// lies past either reads as zeros: another row's scale may be one whose product with a code and a zero is NaN.
// near_end: some lane has n < 4 DW.
template <int DW>
MX_DEV void load_bytes(const uint8_t* t, uint32_t at, int left, bool near_end, int n, uint32_t* v) {
  typedef unsigned vec_t __attribute__((ext_vector_type(DW)));
  typedef vec_t vec_a1 __attribute__((aligned(1)));
  if (near_end && left < 4 * DW) {  // less than a load altogether
#pragma unroll 1
    for (int i = 0; i < DW; i++) {
      uint32_t d = 0;
#pragma unroll 1
      for (int b = 0; b < 4; b++) d |= 4 * i + b < n && (int)at + 4 * i + b < left ? (uint32_t)t[at + 4 * i + b] << (8 * b) : 0;
#pragma unroll
      for (int j = 0; j < DW; j++) v[j] = i == j ? d : v[j];
    }
    return;
  }
  const uint32_t from = near_end ? min(at, (uint32_t)(left - 4 * DW)) : at;
  const vec_t w = *reinterpret_cast<const vec_a1*>(t + from);
#pragma unroll
  for (int i = 0; i < DW; i++) v[i] = w[i];
  if (near_end) {
    const uint32_t d = at - from;  // the bytes from d < 4 DW on move to the front
#pragma unroll
    for (int h = DW / 2; h > 0; h >>= 1)
#pragma unroll
      for (int i = 0; i < DW; i++) v[i] = d / (4 * h) % 2 ? (i + h < DW ? v[i + h] : 0) : v[i];
#pragma unroll
    for (int i = 0; i < DW; i++) {
      const int own = n - 4 * i;
      v[i] = __builtin_amdgcn_alignbyte(i + 1 < DW ? v[i + 1] : 0, v[i], d & 3);
      v[i] &= own >= 4 ? ~0u : own <= 0 ? 0u : (1u << (8 * own)) - 1;
    }
  }
}

// Sums over the 16 rows of R tiles against XR rows of x, over this wave's blocks of K, to `part` [R][16 columns][16].
//
// A step is 128 elements of K: each quarter of the wave holds 32 of them, 16 bytes of codes a lane (a 64-byte piece of
// 16 rows), which make four operands of the matrix instruction.  A block is SB steps that one load each of a row's
// scales and one or a few loads of x serve; all loads of a block go out together, and the other waves of the SIMD work
// meanwhile.  x goes through a piece of LDS of the wave's own (xs), which turns whole rows as they are loaded into the
// instruction's other operand.
// That operand has 16 columns.  FEW (XR <= 4): four columns belong to a row of x and hold different eighths of the
// quarter's 32 elements, so that one 16-byte read serves all four operands of W.  Operand j's product is wanted in
// the columns that hold the eighth j alone: each j has sums of its own, and a row's four columns are added up at
// the end.  What the other columns sum up is dropped, also where it is not finite.
template <int FMT, int R, int XR, int SB, bool FEW, typename RowX>
MX_DEV void tile_sums(const Tiles<R>& w, int K, int wave, int waves, RowX row_of, uint16_t* xs, float* part) {
  constexpr int kB = SB * kStep, DW = SB * (FMT == MXFP4_FMT_NVFP4 ? 2 : 1);
  constexpr int PR = kB / 8, RPL = 64 / PR;              // 16-byte pieces of a row's block; rows of one load
  constexpr int XL = XR > RPL ? XR / RPL : 1;            // loads of x
  constexpr int kPitch = kB + 8;                         // 16 bytes more than the row: no two columns in a bank
  const int lane = threadIdx.x & 63, rc = lane & 15, quarter = lane >> 4;
  const int k_lane = quarter * 32, k_x = lane % PR * 8;
  const uint16_t* x[XL];
#pragma unroll
  for (int l = 0; l < XL; l++) x[l] = row_of(l * RPL + lane / PR);
  uint16_t* xput = xs + lane / PR * kPitch + k_x;
  const uint16_t* xget = xs + (FEW ? (rc >> 2) % XR * kPitch + (rc & 3) * 8 : rc % XR * kPitch) + k_lane;
  struct Block {
    u32x4_t q[R][SB], x[XL];
    uint32_t s[R][DW];
  };
  uint32_t q_at[R], s_at[R];
#pragma unroll
  for (int r = 0; r < R; r++) {
    q_at[r] = w.row[r] * (uint32_t)(K / 2);
    s_at[r] = w.row[r] * (uint32_t)(K / kBlock<FMT>);
  }
  auto load = [&](Block& b, int k0) {
    const bool near_end = k0 + kB > K;
    if (!near_end) {
#pragma unroll
      for (int l = 0; l < XL; l++) b.x[l] = *reinterpret_cast<const u32x4_t*>(x[l] + k0 + k_x);
    } else {
#pragma unroll
      for (int l = 0; l < XL; l++) b.x[l] = *reinterpret_cast<const u32x4_t*>(x[l] + min(k0 + k_x, K - 8));
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
      load_bytes<DW>(w.s[r], s_at[r] + k0 / kBlock<FMT>, w.s_left[r], near_end, (K - k0) / kBlock<FMT>, b.s[r]);
      if (!near_end) {
#pragma unroll
        for (int i = 0; i < SB; i++) b.q[r][i] = load_codes<FMT>(w.q[r], q_at[r] + (k0 + k_lane) / 2 + i * (kStep / 2));
      } else {
#pragma unroll
        for (int i = 0; i < SB; i++)
          b.q[r][i] = load_codes<FMT>(w.q[r], q_at[r] + min(k0 + i * kStep + k_lane, K - 32) / 2);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // the loads go out before anything waits for one
  };
  f32x4_t acc[R][FEW ? 4 : 1] = {};
  auto work = [&](Block& b, int k0) {
#pragma unroll
    for (int l = 0; l < XL; l++) {
      if (k0 + kB > K) {  // past K: zeros
#pragma unroll
        for (int i = 0; i < 4; i++) b.x[l][i] = k0 + k_x < K ? b.x[l][i] : 0;
      }
      if (XR >= RPL || lane / PR < XR) *reinterpret_cast<u32x4_t*>(xput + l * RPL * kPitch) = b.x[l];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < SB; i++) {
      u32x4_t xv[FEW ? 1 : 4];
#pragma unroll
      for (int j = 0; j < (FEW ? 1 : 4); j++) xv[j] = *reinterpret_cast<const u32x4_t*>(xget + i * kStep + j * 8);
#pragma unroll
      for (int r = 0; r < R; r++) {
        float s0, s1;
        if (FMT == MXFP4_FMT_MXFP4) {  // the conversion reads the exponent field
          s0 = s1 = __uint_as_float(__builtin_amdgcn_ubfe(b.s[r][i], 8 * quarter, 8) << 23);
        } else {
          const uint32_t two = (quarter & 2 ? b.s[r][2 * i + 1 < DW ? 2 * i + 1 : 0] : b.s[r][2 * i < DW ? 2 * i : 0]) >>
                               (16 * (quarter & 1));
          s0 = __builtin_amdgcn_cvt_f32_fp8((int)two, 0);
          s1 = __builtin_amdgcn_cvt_f32_fp8((int)two, 1);
        }
        settle<FMT>(b.q[r][i], k0 + i * kStep + k_lane, K);
#pragma unroll
        for (int j = 0; j < 4; j++)
          acc[r][FEW ? j : 0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              dequant8<FMT>(b.q[r][i][j], j < 2 ? s0 : s1), __builtin_bit_cast(bf16x8_t, xv[FEW ? 0 : j]),
              acc[r][FEW ? j : 0], 0, 0, 0);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  const int stride = waves * kB;
  int k0 = wave * kB;
  for (; k0 < K; k0 += stride) {
    Block b;
    load(b, k0);
    work(b, k0);
  }
  // lane: column rc, rows quarter * 4 + i of the tile
#pragma unroll
  for (int r = 0; r < R; r++) {
    f32x4_t v = acc[r][0];
    if (FEW) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
#pragma unroll
        for (int f = 1; f < 4; f++) v[i] = (rc & 3) == f ? acc[r][FEW ? f : 0][i] : v[i];
        v[i] += dpp<0xB1>(v[i]);  // lane ^ 1
        v[i] += dpp<0x4E>(v[i]);  // lane ^ 2
      }
    }
    const int col = FEW ? rc >> 2 : rc;
    if (!FEW || (rc & 3) == 0) *reinterpret_cast<f32x4_t*>(part + r * 256 + col * 16 + quarter * 4) = v;
  }
}

// The same for NVFP4 weights and up to four rows of x, with the scales behind the matrix instruction: of a product's 16
// columns, four belong to a row of x and hold one quarter of the wave's elements each (zeros for the others), so what
// comes out of two instructions is a sum over the 16 elements of one block at a time, which takes its scale in binary32.
// A lane then has 16 conversions, 8 multiply-adds and 8 scales (4 instructions) for its 32 elements of a step, where scaled
// weights take 64 instructions.  1 x 7168 x 7168: 10.5 -> 9.6 us, 1 x 28672 x 7168: 28.6 -> 25 us; 1536 x 2048 with SwiGLU,
// 16 tokens, top-8 of 128: 44 -> 38 us.  The same for 5 to 8 rows (two sets of columns) spilled: 2048 x 768, 64 tokens, 33 -> 40 us.
// kDown on the codes keeps the sums below the scaled ones' (2^-9 is E4M3's least scale); the result takes it back.
// LDS of the wave: rows of x, a row of zeros, the scales turned into the columns' layout.
constexpr float kDown = 0x1p-9f;
constexpr int nv_x_bytes(int xr, int sb) { return (xr + 1) * (sb * kStep + 8) * 2; }
constexpr int nv_bytes(int R, int xr, int sb) { return nv_x_bytes(xr, sb) + R * sb * 128; }

template <int R, int XR, int SB, typename RowX>
MX_DEV void tile_sums_nv(const Tiles<R>& w, int K, int wave, int waves, RowX row_of, uint16_t* xs, float* part) {
  constexpr int kB = SB * kStep, DW = SB / 2;
  constexpr int PR = kB / 8, RPL = 64 / PR;
  constexpr int XL = XR > RPL ? XR / RPL : 1;
  constexpr int kPitch = kB + 8;
  const int lane = threadIdx.x & 63, rc = lane & 15, quarter = lane >> 4, f = rc & 3;
  const int k_lane = quarter * 32, k_x = lane % PR * 8;
  const uint16_t* x[XL];
#pragma unroll
  for (int l = 0; l < XL; l++) x[l] = row_of(l * RPL + lane / PR);
  uint16_t* xput = xs + lane / PR * kPitch + k_x;
  uint16_t* zeros = xs + XR * kPitch;
  if (lane * 8 < kB) *reinterpret_cast<u32x4_t*>(zeros + lane * 8) = u32x4_t{0, 0, 0, 0};
  const uint16_t* xget = (quarter == f ? xs + (rc >> 2) % XR * kPitch : zeros) + k_lane;
  // scales: [quarter of the elements][row][step], two bytes each
  uint8_t* scales = (uint8_t*)xs + nv_x_bytes(XR, SB);
  uint8_t* sput = scales + (SB == 4 ? rc * 8 + quarter * 2 : (quarter & 1) * 128 + rc * 4 + (quarter >> 1) * 2);
  const uint8_t* sget = scales + f * (SB * 32) + quarter * (SB * 8);
  uint32_t q_at[R], s_at[R];
#pragma unroll
  for (int r = 0; r < R; r++) {
    q_at[r] = w.row[r] * (uint32_t)(K / 2);
    s_at[r] = w.row[r] * (uint32_t)(K / 16) + quarter * (2 * SB);
  }
  f32x4_t acc[R] = {};
  for (int k0 = wave * kB; k0 < K; k0 += waves * kB) {
    const bool near_end = k0 + kB > K;
    u32x4_t q[R][SB], xl[XL];
    uint32_t s[R][DW];
#pragma unroll
    for (int l = 0; l < XL; l++) xl[l] = *reinterpret_cast<const u32x4_t*>(x[l] + (near_end ? min(k0 + k_x, K - 8) : k0 + k_x));
#pragma unroll
    for (int r = 0; r < R; r++) {
      load_bytes<DW>(w.s[r], s_at[r] + k0 / 16, w.s_left[r], near_end, (K - k0) / 16 - quarter * (2 * SB), s[r]);
      if (!near_end) {
#pragma unroll
        for (int i = 0; i < SB; i++) q[r][i] = load_codes<MXFP4_FMT_NVFP4>(w.q[r], q_at[r] + (k0 + k_lane) / 2 + i * (kStep / 2));
      } else {
#pragma unroll
        for (int i = 0; i < SB; i++)
          q[r][i] = load_codes<MXFP4_FMT_NVFP4>(w.q[r], q_at[r] + min(k0 + i * kStep + k_lane, K - 32) / 2);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // the loads go out before anything waits for one
#pragma unroll
    for (int l = 0; l < XL; l++) {
      if (near_end) {  // past K: zeros
#pragma unroll
        for (int i = 0; i < 4; i++) xl[l][i] = k0 + k_x < K ? xl[l][i] : 0;
      }
      if (XR >= RPL || lane / PR < XR) *reinterpret_cast<u32x4_t*>(xput + l * RPL * kPitch) = xl[l];
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
      // SB == 4: the lane has a step's four pairs of scales; SB == 2: half of a step's
#pragma unroll
      for (int h = 0; h < SB; h++)
        *reinterpret_cast<uint16_t*>(sput + r * (SB * 128) + h * (SB == 4 ? 128 : 64)) = (uint16_t)(s[r][h / 2] >> (16 * (h & 1)));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    uint32_t sc[R][4][DW];  // rows 4 * quarter + i: two bytes a step
#pragma unroll
    for (int r = 0; r < R; r++) {
#pragma unroll
      for (int h = 0; h < DW; h++) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(sget + r * (SB * 128) + h * 16);
#pragma unroll
        for (int i = 0; i < 4; i++) sc[r][(h * 4 + i) / DW][(h * 4 + i) % DW] = v[i];
      }
    }
#pragma unroll
    for (int i = 0; i < SB; i++) {
      bf16x8_t xv[4];
#pragma unroll
      for (int j = 0; j < 4; j++) xv[j] = *reinterpret_cast<const bf16x8_t*>(xget + i * kStep + j * 8);
#pragma unroll
      for (int r = 0; r < R; r++) {
        settle<MXFP4_FMT_NVFP4>(q[r][i], k0 + i * kStep + k_lane, K);
#pragma unroll
        for (int h = 0; h < 2; h++) {  // the two blocks of the lane's 32 elements
          f32x4_t t = {0, 0, 0, 0};
#pragma unroll
          for (int j = 2 * h; j < 2 * h + 2; j++)
            t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dequant8<MXFP4_FMT_MXFP4>(q[r][i][j], kDown), xv[j], t, 0, 0, 0);
#pragma unroll
          for (int o = 0; o < 4; o++) {
            const f32x2_t two = i % 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)sc[r][o][i / 2], true)
                                      : __builtin_amdgcn_cvt_pk_f32_fp8((int)sc[r][o][i / 2], false);
            acc[r][o] = fmaf(t[o], two[h], acc[r][o]);
          }
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
#pragma unroll
  for (int r = 0; r < R; r++) {
    f32x4_t v = acc[r];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[i] += dpp<0xB1>(v[i]);  // lane ^ 1
      v[i] += dpp<0x4E>(v[i]);  // lane ^ 2
      v[i] *= 1.0f / kDown;
    }
    if (f == 0) *reinterpret_cast<f32x4_t*>(part + r * 256 + (rc >> 2) * 16 + quarter * 4) = v;
  }
}

constexpr int kFew = 4;
constexpr int kManySteps = 2;  // steps of a block for more rows: their x takes registers and LDS
// Where tile_sums_nv takes up to four rows.  Not beside the body for 16 rows with short blocks (64 tokens, top-8 of 128,
// 2048 x 768: 33 us, with it 35 us), nor with four tiles (no faster).
constexpr bool scales_behind(int fmt, int R, int xr, int sb) {
  return fmt == MXFP4_FMT_NVFP4 && R < 4 && (xr <= kFew || sb == 4);
}
// LDS of a wave: its piece of x (and what tile_sums_nv adds), then its sums.
constexpr int wave_bytes(int fmt, int R, int xr, int few_steps) {
  const int f = xr < kFew ? xr : kFew;
  const int few = scales_behind(fmt, R, xr, few_steps) ? nv_bytes(R, f, few_steps) : f * (few_steps * kStep + 8) * 2;
  const int many = xr > kFew ? xr * (kManySteps * kStep + 8) * 2 : 0;
  const int x = few > many ? few : many, sums = R * 1024;
  return x > sums ? x : sums;
}

// Waves per SIMD that the registers are made to fit: four tiles need more of them than four waves leave.
constexpr int waves_a_simd(int R) { return R == 4 ? 3 : 4; }

// One workgroup: a tile of 16 outputs (SWIGLU: 16 gate rows and the 16 up rows), its waves sharing the blocks of K,
// against up to 16 rows of x at a time.  XR: the most rows there are (1, 4 or 16); SB: steps of a block for up to four.
// R: tiles of 16 rows of W (SWIGLU: the gate's and the up projection's).
template <int FMT, bool EXPERT, bool SWIGLU, int XR, int R, int SB>
__global__ __launch_bounds__(XR > kFew ? 512 : 1024, waves_a_simd(R)) void matvec_kernel(MatvecArgs a) {
  constexpr int OT = SWIGLU ? R / 2 : R;  // tiles of outputs
  constexpr int kWave = wave_bytes(FMT, R, XR, SB);
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int K = (int)a.K;
  const int64_t n_out = SWIGLU ? a.N / 2 : a.N;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * OT);
  int64_t e = 0, first = 0, count = a.M;
  if (EXPERT) {
    e = blockIdx.y;
    if (gridDim.y < (unsigned)a.E) {  // fewer pairs than experts: the blockIdx.y-th expert that has any, once clamped
      const int pairs = (int)a.M;  // < E
      int seen = 0;
      e = -1;
      for (int base = 0; base < a.E && e < 0; base += 64) {
        const int i = base + lane;
        const bool has = i < a.E && min(a.offsets[i + 1], pairs) > max(a.offsets[i], 0);
        uint64_t m = __ballot(has);
        const int n = __popcll(m);
        if (seen + n > (int)blockIdx.y) {
          for (int s = seen; s < (int)blockIdx.y; s++) m &= m - 1;
          e = base + __ffsll((unsigned long long)m) - 1;
        }
        seen += n;
      }
      if (e < 0) return;
    }
    const int64_t lo = a.offsets[e], hi = a.offsets[e + 1];
    first = lo < 0 ? 0 : lo;
    count = (hi > a.M ? a.M : hi) - first;
    if (count <= 0) return;
  }
  const float gs = EXPERT && FMT == MXFP4_FMT_NVFP4 ? a.gscales[e] : a.gscale;
  const int KQ = K / 2, KS = K / kBlock<FMT>;
  Tiles<R> w;
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int64_t first_row = min(n0 + 16 * (r % OT), n_out - 1);
    const int64_t row = e * a.N + first_row + r / OT * n_out;
    w.q[r] = a.wq + row * KQ;
    w.s[r] = a.ws + row * KS;
    w.s_left[r] = (int32_t)min(((int64_t)a.E * a.N - row) * KS, (int64_t)1 << 30);
    w.row[r] = (uint32_t)min((int64_t)(lane & 15), n_out - 1 - first_row);
  }
  uint8_t* mine = smem + wave * kWave;
  const int64_t m_step = EXPERT ? 16 : (int64_t)gridDim.y * 16;
  for (int64_t m0 = EXPERT ? 0 : (int64_t)blockIdx.y * 16; m0 < count; m0 += m_step) {
    const int cols = (int)min((int64_t)16, count - m0);
    auto pair_of = [&](int c) -> int64_t {  // column c's row of y, -1: none
      if (!EXPERT) return m0 + c;
      const int64_t p = a.pairs[first + m0 + c];
      return p < a.M ? p : -1;
    };
    auto row_of = [&](int c) {
      const int64_t p = pair_of(min(c, cols - 1));
      return a.x + (p < 0 ? 0 : EXPERT ? (int64_t)((uint32_t)p / (uint32_t)a.top_k) : p) * a.ldx;
    };
    uint16_t* xs = (uint16_t*)mine;
    float* part = (float*)mine;
    if (scales_behind(FMT, R, XR, SB) && (XR == 1 || (EXPERT && cols == 1)))
      tile_sums_nv<R, 1, SB>(w, K, wave, waves, row_of, xs, part);
    else if (scales_behind(FMT, R, XR, SB) && (XR == 4 || cols <= kFew))
      tile_sums_nv<R, 4, SB>(w, K, wave, waves, row_of, xs, part);
    else if (R < 4 && (XR == 1 || (EXPERT && cols == 1)))
      tile_sums<FMT, R, 1, SB, true>(w, K, wave, waves, row_of, xs, part);
    else if (R < 4 && (XR == 4 || cols <= kFew))
      tile_sums<FMT, R, 4, SB, true>(w, K, wave, waves, row_of, xs, part);
    else if (R == 4 && cols <= 4)
      tile_sums<FMT, R, 4, kManySteps, false>(w, K, wave, waves, row_of, xs, part);
    else if (cols <= 8)
      tile_sums<FMT, R, 8, kManySteps, false>(w, K, wave, waves, row_of, xs, part);
    else
      tile_sums<FMT, R, 16, kManySteps, false>(w, K, wave, waves, row_of, xs, part);
    __syncthreads();
    for (int o = tid; o < cols * 16 * OT; o += blockDim.x) {
      const int at = o % (16 * OT), col = o / (16 * OT), tile = at / 16;
      float v[SWIGLU ? 2 : 1];
#pragma unroll
      for (int r = 0; r < (SWIGLU ? 2 : 1); r++) {
        v[r] = 0.0f;
        for (int g = 0; g < waves; g++)
          v[r] += reinterpret_cast<const float*>(smem + g * kWave)[(tile + r * OT) * 256 + col * 16 + at % 16];
      }
      const int64_t n = n0 + at, out_row = pair_of(col);
      if (n < n_out && out_row >= 0) {
#pragma unroll
        for (int r = 0; r < (SWIGLU ? 2 : 1); r++) {
          if (FMT == MXFP4_FMT_NVFP4) v[r] /= gs;  // (its reciprocal may overflow)
          if (a.bias) v[r] += bias_at(a.bias, a.bias_fp32, e * a.N + n + r * n_out);
        }
        const float y = SWIGLU ? v[0] / (1.0f + __expf(-v[0])) * v[SWIGLU ? 1 : 0] : v[0];
        if (a.out_fp32)
          ((float*)a.y)[out_row * a.ldy + n] = y;
        else
          ((uint16_t*)a.y)[out_row * a.ldy + n] = to_bf16(y);
      }
    }
    __syncthreads();
  }
}

template <int FMT, bool EXPERT, bool SWIGLU, int XR, int R, int SB>
int launch_rows(const MatvecArgs& a, hipStream_t stream) {
  constexpr int kRows = 16 * (SWIGLU ? R / 2 : R);
  const int64_t n_out = SWIGLU ? a.N / 2 : a.N;
  const int64_t groups = EXPERT ? (a.M < a.E ? a.M : a.E) : (a.M + 15) / 16;
  const int64_t tiles = (n_out + kRows - 1) / kRows;
  const int kB = (XR > kFew ? kManySteps : SB) * kStep;
  const int64_t blocks = (a.K + kB - 1) / kB;
  // blocks of K a wave works through: as few as leave waves to fill the chip, and 16 waves a workgroup (8 for many rows
  // of x, whose LDS they share); a wave less where the last round would be less than half full (one row of 14000 x 5120,
  // 9600 x 7168, 24000 x 1536: MXFP4 9.9 -> 9.1, 10.6 -> 10.1, 6.8 -> 6.7 us, but NVFP4 11.6 -> 12.0, 11.9 -> 12.3, 7.8 -> 8.2;
  // 16 rows: no difference)
  int64_t each = tiles * groups * blocks / (R == 4 ? kFullWide : kFull);
  each = each < 1 ? 1 : each;
  const int64_t most = XR > kFew ? 8 : 16;
  if ((blocks + each - 1) / each > most) each = (blocks + most - 1) / most;
  int waves = (int)((blocks + each - 1) / each);
  if (waves > 1 && (waves - blocks % waves) % waves * 2 >= waves) waves--;
  const dim3 grid((unsigned)tiles, (unsigned)(groups < 65535 ? groups : 65535));
  const int lds = waves * wave_bytes(FMT, R, XR, SB);
  hipLaunchKernelGGL((matvec_kernel<FMT, EXPERT, SWIGLU, XR, R, SB>), grid, dim3(64 * waves), lds, stream, a);
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

template <int FMT, bool EXPERT, bool SWIGLU, int SB>
int launch_steps(const MatvecArgs& a, hipStream_t stream) {
  constexpr int kOne = SWIGLU ? 2 : 1;
  if (a.M == 1) return launch_rows<FMT, EXPERT, SWIGLU, 1, kOne, SB>(a, stream);
  return a.M <= kFew ? launch_rows<FMT, EXPERT, SWIGLU, 4, kOne, SB>(a, stream)
                     : launch_rows<FMT, EXPERT, SWIGLU, 16, 2, SB>(a, stream);
}

template <int FMT, bool EXPERT, bool SWIGLU>
int launch_waves(const MatvecArgs& a, hipStream_t stream) {
  const int64_t n_out = SWIGLU ? a.N / 2 : a.N;
  // Four tiles a wave, which share its rows of x, where experts have three pairs on average and K is long: 1536 x 2048 with
  // SwiGLU, four pairs an expert, NVFP4 64 -> 56 us.  With two pairs (4000 x 1600) two tiles take 59 us, four 71 us.
  if (EXPERT && a.M >= 3 * (int64_t)a.E && a.K >= 6 * kManySteps * kStep && (n_out + 15) / 16 * a.E >= kWide)
    return launch_rows<FMT, EXPERT, SWIGLU, 16, EXPERT ? 4 : 2, kManySteps>(a, stream);
  // Blocks of four steps, or of two where those would be more than a fifth padding (K = 768: 38 -> 35 us; K = 7168: 10.4
  // and 10.7 us).
  const int64_t padded = (a.K + 4 * kStep - 1) / (4 * kStep) * (4 * kStep);
  return padded * 4 > a.K * 5 ? launch_steps<FMT, EXPERT, SWIGLU, 2>(a, stream)
                              : launch_steps<FMT, EXPERT, SWIGLU, 4>(a, stream);
}

template <int FMT>
int launch_fmt(const MatvecArgs& a, hipStream_t stream) {
  if (!a.offsets) return launch_waves<FMT, false, false>(a, stream);
  return a.swiglu ? launch_waves<FMT, true, true>(a, stream) : launch_waves<FMT, true, false>(a, stream);
}

}  // namespace

int launch_matvec(int fmt, const MatvecArgs& a, hipStream_t stream) {
  return fmt == MXFP4_FMT_NVFP4 ? launch_fmt<MXFP4_FMT_NVFP4>(a, stream) : launch_fmt<MXFP4_FMT_MXFP4>(a, stream);
}
