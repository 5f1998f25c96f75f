// Matrix-vector products with 4-bit weights in the standard layout: y = x W^T (/ global scale) + b for a few
// rows of x, and the same product of every routed pair with its expert's matrix (with SwiGLU on request).
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

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 128;  // K elements of one step: 32 for each quarter of the wave

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

// What a lane holds of one row for one step: 32 codes and their scale bytes.
struct Chunk {
  u32x4_t q;
  uint32_t s;
};

// k: first of the lane's 32 elements; K - k elements are there (K % 16 == 0).
template <int FMT>
MX_DEV Chunk load_chunk(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int64_t k, int64_t K) {
  Chunk c = {u32x4_t{0, 0, 0, 0}, 0};
  if (FMT == MXFP4_FMT_MXFP4) {
    if (k < K) {
      c.q = *reinterpret_cast<const u32x4_t*>(q + k / 2);
      c.s = s[k / 32];
    }
  } else {
    if (k + 32 <= K) {
      c.q = *reinterpret_cast<const u32x4_a8*>(q + k / 2);
      c.s = (uint32_t)s[k / 16] | ((uint32_t)s[k / 16 + 1] << 8);
    } else if (k < K) {
      const u32x2_t h = *reinterpret_cast<const u32x2_t*>(q + k / 2);
      c.q = u32x4_t{h[0], h[1], 0, 0};
      c.s = s[k / 16];
    }
  }
  return c;
}

template <int FMT>
MX_DEV float chunk_scale(uint32_t s, int half) {
  if (FMT == MXFP4_FMT_MXFP4) return __uint_as_float(s << 23);  // the conversion reads the exponent field
  return half ? __builtin_amdgcn_cvt_f32_fp8((int)s, 1) : __builtin_amdgcn_cvt_f32_fp8((int)s, 0);
}

MX_DEV float bias_at(const void* b, int fp32, int64_t i) {
  return fp32 ? ((const float*)b)[i] : __uint_as_float((uint32_t)((const uint16_t*)b)[i] << 16);
}

MX_DEV uint16_t to_bf16(float f) {  // round to nearest even; infinities pass, NaN stays NaN
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// One workgroup: 16 rows of W (SWIGLU: 16 gate rows and the 16 up rows), up to 16 rows of x at a time, the
// whole of K split over the waves, which join through LDS.
template <int FMT, bool EXPERT, bool SWIGLU>
__global__ __launch_bounds__(kThreads) void matvec_kernel(MatvecArgs a) {
  constexpr int R = SWIGLU ? 2 : 1;
  constexpr int B = FMT == MXFP4_FMT_NVFP4 ? 16 : 32;
  __shared__ float part[kWaves][R][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rc = lane & 15, quarter = lane >> 4;
  const int64_t n_out = SWIGLU ? a.N / 2 : a.N;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  int64_t e = 0, first = 0, count = a.M;
  if (EXPERT) {
    // the blockIdx.y-th expert that has pairs
    int seen = 0;
    e = -1;
    for (int base = 0; base < a.E && e < 0; base += 64) {
      const int i = base + lane;
      const bool has = i < a.E && a.offsets[i + 1] > a.offsets[i];
      uint64_t m = __ballot(has);
      const int n = __popcll(m);
      if (seen + n > (int)blockIdx.y) {
        for (int s = seen; s < (int)blockIdx.y; s++) m &= m - 1;
        e = base + __ffsll((unsigned long long)m) - 1;
      }
      seen += n;
    }
    if (e < 0) return;
    const int64_t lo = a.offsets[e], hi = a.offsets[e + 1];
    first = lo < 0 ? 0 : lo;
    count = (hi > a.M ? a.M : hi) - first;
  }
  const int64_t KQ = a.K / 2, KS = a.K / B;
  const uint8_t* wq = a.wq + e * a.N * KQ;
  const uint8_t* ws = a.ws + e * a.N * KS;
  const int64_t row = min(n0 + rc, n_out - 1);  // rows past the last repeat it and are not stored
  const float gs = EXPERT && FMT == MXFP4_FMT_NVFP4 ? a.gscales[e] : a.gscale;

  const int64_t m_step = EXPERT ? 16 : (int64_t)gridDim.y * 16;
  for (int64_t m0 = EXPERT ? 0 : (int64_t)blockIdx.y * 16; m0 < count; m0 += m_step) {
    // the row of x of this lane's column
    int64_t m = m0 + rc;
    bool have = m < count;
    if (EXPERT && have) {
      const int64_t p = a.pairs[first + m];
      have = p >= 0 && p < a.M;
      m = p / a.top_k;
    }
    const uint16_t* x = a.x + m * a.ldx;
    f32x4_t acc[R] = {};
    for (int64_t k0 = (int64_t)wave * kStep; k0 < a.K; k0 += kWaves * kStep) {
      const int64_t k = k0 + quarter * 32;
      Chunk c[R];
#pragma unroll
      for (int r = 0; r < R; r++)
        c[r] = load_chunk<FMT>(wq + (row + r * n_out) * KQ, ws + (row + r * n_out) * KS, k, a.K);
      u32x4_t xv[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        xv[j] = u32x4_t{0, 0, 0, 0};
        if (have && k + j * 8 < a.K) xv[j] = *reinterpret_cast<const u32x4_t*>(x + k + j * 8);
      }
#pragma unroll
      for (int r = 0; r < R; r++)
#pragma unroll
        for (int j = 0; j < 4; j++)
          acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dequant8<FMT>(c[r].q[j], chunk_scale<FMT>(c[r].s, j / 2)),
                                                           __builtin_bit_cast(bf16x8_t, xv[j]), acc[r], 0, 0, 0);
    }
    // lane: column rc of x, rows quarter * 4 + i of W
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
      for (int i = 0; i < 4; i++) part[wave][r][rc * 16 + quarter * 4 + i] = acc[r][i];
    __syncthreads();
    const int t = threadIdx.x;
    if (t < 256) {
      float v[R];
#pragma unroll
      for (int r = 0; r < R; r++) {
        v[r] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; w++) v[r] += part[w][r][t];
      }
      const int64_t n = n0 + (t & 15), mm = m0 + (t >> 4);
      if (n < n_out && mm < count) {
        int64_t out_row = mm;
        bool store = true;
        if (EXPERT) {
          out_row = a.pairs[first + mm];
          store = out_row >= 0 && out_row < a.M;
        }
        if (store) {
#pragma unroll
          for (int r = 0; r < R; r++) {
            if (FMT == MXFP4_FMT_NVFP4) v[r] /= gs;
            if (a.bias) v[r] += bias_at(a.bias, a.bias_fp32, e * a.N + n + r * n_out);
          }
          const float y = SWIGLU ? v[0] / (1.0f + __expf(-v[0])) * v[R - 1] : v[0];
          if (a.out_fp32)
            ((float*)a.y)[out_row * a.ldy + n] = y;
          else
            ((uint16_t*)a.y)[out_row * a.ldy + n] = to_bf16(y);
        }
      }
    }
    __syncthreads();
  }
}

template <int FMT>
int launch_fmt(const MatvecArgs& a, hipStream_t stream) {
  const int64_t n_out = a.swiglu ? a.N / 2 : a.N;
  const unsigned gx = (unsigned)((n_out + 15) / 16);
  if (a.offsets) {
    const dim3 grid(gx, (unsigned)(a.M < a.E ? a.M : a.E));
    if (a.swiglu)
      hipLaunchKernelGGL((matvec_kernel<FMT, true, true>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((matvec_kernel<FMT, true, false>), grid, dim3(kThreads), 0, stream, a);
  } else {
    const int64_t gy = (a.M + 15) / 16;
    hipLaunchKernelGGL((matvec_kernel<FMT, false, false>), dim3(gx, (unsigned)(gy < 65535 ? gy : 65535)),
                       dim3(kThreads), 0, stream, a);
  }
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

}  // namespace

int launch_matvec(int fmt, const MatvecArgs& a, hipStream_t stream) {
  return fmt == MXFP4_FMT_NVFP4 ? launch_fmt<MXFP4_FMT_NVFP4>(a, stream) : launch_fmt<MXFP4_FMT_MXFP4>(a, stream);
}
