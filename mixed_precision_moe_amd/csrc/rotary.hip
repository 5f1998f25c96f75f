// Rotary positions: pairs of each query and key vector turned by position * frequency.
//
//   a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t),  t = 2 pi position turns[i]
//
// Bound by memory: each element is read once and written once.  A workgroup takes a few tokens, has the sine and cosine of
// their angles in LDS first (one a thread, shared by all heads), then runs over the vectors of both tensors in 16-byte
// accesses.  The angle is formed in binary64 and loses its whole turns there (a far position times a frequency has
// no place left for the fraction in binary32); what rounding the fraction to binary32 loses is put back to first order.
#include <hip/hip_runtime.h>

#include "drafts.h"

#define MX_DEV __device__ __forceinline__

namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 1024;  // in LDS: tokens of a workgroup times pairs
constexpr int64_t kMaxGrid = 1 << 20;

template <typename T, int V, int ALIGN>
struct alignas(ALIGN) Vec {
  T v[V];
};

MX_DEV float2 cos_sin(double turns, float magnitude, float sign) {
  const double f = turns - rint(turns);  // [-1/2, 1/2]
  const float hi = (float)(2.0 * f);
  const float lo = (float)(2.0 * f - (double)hi) * 3.14159274f;
  float s, c;
  sincospif(hi, &s, &c);
  return float2{magnitude * (c - s * lo), magnitude * sign * (s + c * lo)};
}

// WIDE: 16 bytes an access, which everything is aligned to; else single elements.
template <typename T, bool WIDE, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, int tokens) {
  constexpr int V = WIDE ? 16 / sizeof(T) : INTERLEAVED ? 2 : 1;  // turned elements of an access
  constexpr int R = WIDE ? V : 1;                                 // and others
  using W = Vec<T, V, WIDE ? 16 : sizeof(T)>;
  using C = Vec<T, R, WIDE ? 16 : sizeof(T)>;
  __shared__ float2 cs[kAngles];
  const int pairs = a.rot_dim / 2;
  for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.rows; t0 += (int64_t)gridDim.x * tokens) {
    const int n = (int)min((int64_t)tokens, a.rows - t0);
    if (t0 >= (int64_t)gridDim.x * tokens) __syncthreads();  // the angles before are done with
    for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
      const int t = i / pairs;
      cs[i] = cos_sin((double)a.positions[t0 + t] * a.turns[i - t * pairs], a.magnitude, a.sign);
    }
    __syncthreads();
    // units of a head: accesses of turned elements (pairs of accesses with the halves apart), then those of the rest
    const uint32_t turned = INTERLEAVED ? a.rot_dim / V : pairs / V;
    const uint32_t rest = (a.head_dim - a.rot_dim) / R;
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const RotaryRows& r = a.x[x];
      const bool in_place = r.in == r.out && r.in_ldt == r.out_ldt && r.in_ldh == r.out_ldh;
      const uint32_t per_head = turned + (in_place ? 0 : rest), per_token = per_head * (uint32_t)r.heads;
      for (uint32_t u = threadIdx.x; u < per_token * (uint32_t)n; u += kThreads) {
        const uint32_t t = u / per_token, in_token = u - t * per_token;
        const uint32_t head = in_token / per_head, k = in_token - head * per_head;
        const T* src = (const T*)r.in + (t0 + t) * r.in_ldt + (int64_t)head * r.in_ldh;
        T* dst = (T*)r.out + (t0 + t) * r.out_ldt + (int64_t)head * r.out_ldh;
        if (k >= turned) {
          uint32_t e = (k - turned) * R;
          if (e >= (uint32_t)a.offset) e += a.rot_dim;
          *reinterpret_cast<C*>(dst + e) = *reinterpret_cast<const C*>(src + e);
          continue;
        }
        const float2* angle = cs + t * pairs;
        if (INTERLEAVED) {
          const uint32_t e = a.offset + k * V;
          const W in = *reinterpret_cast<const W*>(src + e);
          W out;
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float2 c = angle[(k * V + i) / 2];
            const float p = (float)in.v[i], q = (float)in.v[i + 1];
            out.v[i] = (T)(p * c.x - q * c.y);
            out.v[i + 1] = (T)(q * c.x + p * c.y);
          }
          *reinterpret_cast<W*>(dst + e) = out;
        } else {
          const uint32_t e = a.offset + k * V;
          const W lo = *reinterpret_cast<const W*>(src + e), hi = *reinterpret_cast<const W*>(src + e + pairs);
          W out_lo, out_hi;
#pragma unroll
          for (int i = 0; i < V; i++) {
            const float2 c = angle[k * V + i];
            const float p = (float)lo.v[i], q = (float)hi.v[i];
            out_lo.v[i] = (T)(p * c.x - q * c.y);
            out_hi.v[i] = (T)(q * c.x + p * c.y);
          }
          *reinterpret_cast<W*>(dst + e) = out_lo;
          *reinterpret_cast<W*>(dst + e + pairs) = out_hi;
        }
      }
    }
  }
}

template <typename T, bool INTERLEAVED>
int launch_type(const RotaryArgs& a, hipStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const int pairs = a.rot_dim / 2;
  bool wide = (INTERLEAVED ? a.rot_dim : pairs) % V == 0 && a.offset % V == 0 && a.head_dim % V == 0;
  for (const RotaryRows& r : a.x) {
    if (!r.heads) continue;
    // (the stride of a dimension of one entry is used for entry 0 alone)
    const uint64_t strides = (a.rows > 1 ? (uint64_t)r.in_ldt | (uint64_t)r.out_ldt : 0) |
                             (r.heads > 1 ? (uint64_t)r.in_ldh | (uint64_t)r.out_ldh : 0);
    wide = wide && strides % V == 0 && ((uint64_t)(uintptr_t)r.in | (uint64_t)(uintptr_t)r.out) % 16 == 0;
  }
  int tokens = kAngles / pairs;
  tokens = tokens > 4 ? 4 : tokens;  // pairs <= kAngles
  const int64_t n = (a.rows + tokens - 1) / tokens;
  const dim3 grid((unsigned)(n < kMaxGrid ? n : kMaxGrid));
  if (wide)
    hipLaunchKernelGGL((rotary_kernel<T, true, INTERLEAVED>), grid, dim3(kThreads), 0, stream, a, tokens);
  else
    hipLaunchKernelGGL((rotary_kernel<T, false, INTERLEAVED>), grid, dim3(kThreads), 0, stream, a, tokens);
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

}  // namespace

int launch_rotary(bool fp32, bool interleaved, const RotaryArgs& a, hipStream_t stream) {
  if (fp32) return interleaved ? launch_type<float, true>(a, stream) : launch_type<float, false>(a, stream);
  return interleaved ? launch_type<__bf16, true>(a, stream) : launch_type<__bf16, false>(a, stream);
}
