// Rotary positions: pairs of each query and key vector turned by position * frequency.
//
//   a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t),  t = 2 pi position turns[i]
//
// Bound by memory: each element is read once and written once.  A workgroup takes a few tokens, has the sine and cosine of
// their angles in LDS first (one a thread, shared by all heads), then runs over the vectors of both tensors in the widest
// accesses that everything divides by.  8192 x 40 heads of 128 elements, bf16: 31 us, 5.4 TB/s (4 tokens a workgroup; 2: 33,
// 8: 35); 4099 x 32 heads of 192 with a third turned, fp32: 43 us, 4.7 TB/s (45, 52); 4096 x 32 heads of 128, bf16, with
// accesses of 16, 8, 4 and 2 bytes: 4.8, 4.7, 4.1 and 2.9 TB/s (passes of 14 to 23 us).  The angle is formed in binary64 and loses
// its whole turns there (a far position times a frequency has no place left for the fraction in binary32); what rounding
// the fraction to binary32 loses is put back to first order.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "drafts.h"

#define MX_DEV __device__ __forceinline__

namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 1024;  // in LDS: tokens of a workgroup times pairs
constexpr int64_t kMaxGrid = 1 << 20;

// An access of N bytes, and what it holds.
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
template <int N>
using Access = std::conditional_t<N == 16, u32x4_t, std::conditional_t<N == 8, uint64_t, std::conditional_t<N == 4, uint32_t, uint16_t>>>;
template <typename T, int V>
struct Vec {
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

// V: elements of an access, which divides everything.
template <typename T, int V, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, int tokens) {
  constexpr bool ONE = INTERLEAVED && V > 1;  // an access has both elements of its pairs
  using A = Access<V * sizeof(T)>;
  using W = Vec<T, V>;
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
    // Units of a head: accesses in order where they have whole pairs, else the pairs' two accesses, then the others by two,
    // the last of an odd number twice.  Turned and other elements, side by side in a wave, take the same loads.
    const uint32_t turned = (uint32_t)pairs / V, begin = (uint32_t)a.offset, end = begin + a.rot_dim;
    const uint32_t rest = (a.head_dim - a.rot_dim) / V, half = (rest + 1) / 2;
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const RotaryRows& r = a.x[x];
      if (r.heads == 0) continue;  // no such tensor
      const bool in_place = r.in == r.out && r.in_ldt == r.out_ldt && r.in_ldh == r.out_ldh;
      const uint32_t per_head = ONE ? (in_place ? a.rot_dim : a.head_dim) / V : turned + (in_place ? 0 : half);
      const uint32_t heads = (uint32_t)r.heads;
      // a thread's unit k of head h of token t, and what a step of all threads adds to them
      uint32_t k = threadIdx.x % per_head, h = threadIdx.x / per_head, t = h / heads;
      h -= t * heads;
      const uint32_t step_k = kThreads % per_head, step_h = kThreads / per_head % heads, step_t = kThreads / per_head / heads;
      const auto step = [&] {
        k += step_k;
        h += step_h;
        t += step_t;
        if (k >= per_head) k -= per_head, h++;
        if (h >= heads) h -= heads, t++;
      };
      for (; t < (uint32_t)n; step()) {
        const T* src = (const T*)r.in + (t0 + t) * r.in_ldt + (int64_t)h * r.in_ldh;
        T* dst = (T*)r.out + (t0 + t) * r.out_ldt + (int64_t)h * r.out_ldh;
        if (ONE) {
          const uint32_t at = k * V + (in_place ? begin : 0);
          W x = __builtin_bit_cast(W, *reinterpret_cast<const A*>(src + at));
          if (at >= begin && at < end) {
            const float2* angle = cs + t * pairs + (at - begin) / 2;
#pragma unroll
            for (int i = 0; i < V; i += 2) {
              const float2 c = angle[i / 2];
              const float p = (float)x.v[i], q = (float)x.v[i + 1];
              x.v[i] = (T)(p * c.x - q * c.y);
              x.v[i + 1] = (T)(q * c.x + p * c.y);
            }
          }
          *reinterpret_cast<A*>(dst + at) = __builtin_bit_cast(A, x);
          continue;
        }
        uint32_t at = begin + (INTERLEAVED ? 2 * k : k * V), other = at + (INTERLEAVED ? 1 : pairs);
        if (k >= turned) {
          at = (k - turned) * V;
          other = min(k - turned + half, rest - 1) * V;
          at += at >= begin ? a.rot_dim : 0;
          other += other >= begin ? a.rot_dim : 0;
        }
        const A at_lo = *reinterpret_cast<const A*>(src + at), at_hi = *reinterpret_cast<const A*>(src + other);
        if (k >= turned) {
          *reinterpret_cast<A*>(dst + at) = at_lo;
          *reinterpret_cast<A*>(dst + other) = at_hi;
          continue;
        }
        const float2* angle = cs + t * pairs + k * V;
        const W lo = __builtin_bit_cast(W, at_lo), hi = __builtin_bit_cast(W, at_hi);
        W out_lo, out_hi;
#pragma unroll
        for (int i = 0; i < V; i++) {
          const float2 c = angle[i];
          const float p = (float)lo.v[i], q = (float)hi.v[i];
          out_lo.v[i] = (T)(p * c.x - q * c.y);
          out_hi.v[i] = (T)(q * c.x + p * c.y);
        }
        *reinterpret_cast<A*>(dst + at) = __builtin_bit_cast(A, out_lo);
        *reinterpret_cast<A*>(dst + other) = __builtin_bit_cast(A, out_hi);
      }
    }
  }
}

template <typename T, int V, bool INTERLEAVED>
int launch_width(const RotaryArgs& a, uint64_t sizes, uint64_t pointers, hipStream_t stream) {
  if constexpr (V > 1)
    if (sizes % V || pointers % (V * sizeof(T))) return launch_width<T, V / 2, INTERLEAVED>(a, sizes, pointers, stream);
  int tokens = kAngles / (a.rot_dim / 2);
  tokens = tokens > 4 ? 4 : tokens;  // pairs <= kAngles
  const int64_t n = (a.rows + tokens - 1) / tokens;
  const dim3 grid((unsigned)(n < kMaxGrid ? n : kMaxGrid));
  hipLaunchKernelGGL((rotary_kernel<T, V, INTERLEAVED>), grid, dim3(kThreads), 0, stream, a, tokens);
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

// The widest accesses that sizes, strides and pointers allow, up to 16 bytes.
template <typename T, bool INTERLEAVED>
int launch_type(const RotaryArgs& a, hipStream_t stream) {
  uint64_t sizes = (uint64_t)(INTERLEAVED ? a.rot_dim : a.rot_dim / 2) | (uint64_t)a.offset | (uint64_t)a.head_dim, pointers = 0;
  for (const RotaryRows& r : a.x) {
    if (!r.heads) continue;
    // (the stride of a dimension of one entry is used for entry 0 alone)
    if (a.rows > 1) sizes |= (uint64_t)r.in_ldt | (uint64_t)r.out_ldt;
    if (r.heads > 1) sizes |= (uint64_t)r.in_ldh | (uint64_t)r.out_ldh;
    pointers |= (uint64_t)(uintptr_t)r.in | (uint64_t)(uintptr_t)r.out;
  }
  return launch_width<T, 16 / sizeof(T), INTERLEAVED>(a, sizes, pointers, stream);
}

}  // namespace

int launch_rotary(bool fp32, bool interleaved, const RotaryArgs& a, hipStream_t stream) {
  if (fp32) return interleaved ? launch_type<float, true>(a, stream) : launch_type<float, false>(a, stream);
  return interleaved ? launch_type<__bf16, true>(a, stream) : launch_type<__bf16, false>(a, stream);
}
