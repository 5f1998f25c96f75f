// Attention over the block-quantized paged cache: rows see the positions before their sequence's drafts, and of the
// drafts those that a mask or their order leaves.
//
//   out[t, h] = sum_j p_j V[j, g] / sum_j p_j,  p_j = exp(scale q[t, h] . K[j, g] - m),  m = max_j of the exponent
//
// One wave a row and query head; a lane has a position of 64 at a time.
#include <hip/hip_runtime.h>

#include "cache_slots.h"
#include "drafts.h"

#define MX_DEV __device__ __forceinline__

namespace {

MX_DEV float code_value(int fmt, const uint8_t* q, int i) {
  if (fmt == MXFP4_FMT_MXFP8) return __builtin_amdgcn_cvt_f32_fp8((int)q[i], 0);
  const uint32_t c = (q[i >> 1] >> (4 * (i & 1))) & 15u;
  const uint32_t m = c & 7u, e = m >> 1;
  const float v = e ? ldexpf(1.0f + 0.5f * (m & 1u), (int)e - 1) : 0.5f * m;
  return c & 8u ? -v : v;
}

MX_DEV float scale_value(int fmt, uint8_t s) {
  return fmt == MXFP4_FMT_NVFP4 ? __builtin_amdgcn_cvt_f32_fp8((int)s, 0) : ldexpf(1.0f, (int)s - 127);
}

__global__ __launch_bounds__(64) void attend_kernel(int fmt, AttendArgs a) {
  __shared__ float p[64];
  __shared__ int64_t slot[64];
  const CacheArgs& c = a.cache;
  const int lane = threadIdx.x, h = blockIdx.y, g = h / (a.q_heads / c.heads);
  const int64_t t = blockIdx.x;
  int lo = 0, hi = c.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)c.cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
  }
  if (lo >= c.n_seqs || t < (int64_t)c.cu[lo]) return;
  const int block = fmt == MXFP4_FMT_NVFP4 ? 16 : 32, per = fmt == MXFP4_FMT_MXFP8 ? 1 : 2;
  const int64_t start = c.start ? c.start[lo] : 0, n = (int64_t)c.cu[lo + 1] - c.cu[lo], draft = t - c.cu[lo];
  const int kd = c.plane[0].dim, vd = c.plane[1].dim;
  const uint16_t* q = (const uint16_t*)c.plane[0].rows + t * c.plane[0].ldt + h * c.plane[0].ldh;
  const float scale = a.scale / (fmt == MXFP4_FMT_NVFP4 ? c.plane[0].gs : 1.0f);
  float m = -INFINITY, sum = 0.0f, acc[4] = {0, 0, 0, 0};
  const int64_t end = min(a.mask ? start + n : start + draft + 1, (int64_t)c.max_pages * c.page_size);
  for (int64_t p0 = 0; p0 < end; p0 += 64) {
    const int64_t pos = p0 + lane;
    int64_t at = -1;
    if (pos < end) {
      const int64_t j = pos - start;
      const bool sees = j < 0 || !a.mask || (j < a.mask_cols && a.mask[t * a.ld_mask + j]);
      const int64_t page = sees ? c.table[(int64_t)lo * c.ld_table + pos / c.page_size] : -1;
      if (page >= 0 && page < c.num_pages) at = page * c.page_size + pos % c.page_size;
    }
    float s = -INFINITY;
    if (at >= 0) {
      s = 0.0f;
      const int64_t vec = at * c.heads + g;
      for (int b = 0; b < kd / block; b++) {
        const float f = scale_value(fmt, c.plane[0].s[vec * (kd / block) + b]);
        for (int i = 0; i < block; i++) {
          const int e = b * block + i;
          s += __uint_as_float((uint32_t)q[e] << 16) * (code_value(fmt, c.plane[0].q + vec * (kd / per), e) * f);
        }
      }
      s *= scale;
    }
    float top = s;
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float now = fmaxf(m, top);
    if (now == -INFINITY) continue;
    const float keep = expf(m - now), w = expf(s - now);
    float all = w;
    for (int x = 1; x < 64; x <<= 1) all += __shfl_xor(all, x);
    sum = sum * keep + all;
    m = now;
    __syncthreads();
    p[lane] = w;
    slot[lane] = at;
    __syncthreads();
    for (int d = 0; d < 4; d++) {
      const int e = d * 64 + lane;
      acc[d] *= keep;
      if (e >= vd) continue;
      for (int j = 0; j < 64; j++) {
        if (slot[j] < 0) continue;
        const int64_t vec = slot[j] * c.heads + g;
        acc[d] += p[j] * (code_value(fmt, c.plane[1].q + vec * (vd / per), e) *
                          scale_value(fmt, c.plane[1].s[vec * (vd / block) + e / block]));
      }
    }
  }
  const float r = sum > 0.0f ? 1.0f / (sum * (fmt == MXFP4_FMT_NVFP4 ? c.plane[1].gs : 1.0f)) : 0.0f;
  const int64_t to = t * c.plane[1].ldt + h * c.plane[1].ldh;
  for (int d = 0; d < 4; d++) {
    const int e = d * 64 + lane;
    if (e >= vd) continue;
    if (a.out_fp32)
      ((float*)c.plane[1].rows)[to + e] = acc[d] * r;
    else
      ((__bf16*)c.plane[1].rows)[to + e] = (__bf16)(acc[d] * r);
  }
}

}  // namespace

uint64_t attend_workspace(const mxfp4_cache_dims*, int32_t, int64_t, int32_t) { return 256; }

int launch_attend(int fmt, const AttendArgs& a, void*, hipStream_t stream) {
  hipLaunchKernelGGL(attend_kernel, dim3((unsigned)a.cache.rows, a.q_heads), dim3(64), 0, stream, fmt, a);
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}
