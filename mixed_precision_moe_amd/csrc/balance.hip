// Balance loss of the router: per-expert counts, the loss and its gradient.
//
//   p_t = softmax(l_t),  S_e = sum_t p_te,  n_e = pairs of expert e,  V = tokens that count
//   loss = E / (k V^2) * sum_e n_e S_e
//   dl_te = g p_te (d_e - sum_e' d_e' p_te'),  d_e = E / (k V^2) (n_e - mean n)
//
// Both passes stream the logits once and are bound by that; everything about a token stays in registers.
// A token's row lies across LPR lanes with VPL values each, so a wave holds 64 / LPR rows and a lane keeps
// the same columns from row to row: S_e needs no exchange inside the loop.  The forward pass runs as
// partial sums of up to 256 workgroups and a second launch that joins them (8 columns a workgroup, binary64, fixed
// order); the workgroup that is last to finish adds up the loss.  Few logits take one workgroup and one launch.
// Measured (averages): 65533 x 384 with a fifth of the rows masked: forward 22.6 us (80 MB of rows that count, 3.6 TB/s),
// join 9.4 us, backward 34.5 us (181 MB, 5.3 TB/s); one row instead of two on its way 29.5 us; 8192 x 128: 5, 7 and 5.3 us.
// The join is four dependent trips to memory (partial sums, publishing, the number, the columns); with 512 partial sums and
// 32 columns a workgroup it took 14 us.
#include <hip/hip_runtime.h>

#include "ops.h"

#define MX_DEV __device__ __forceinline__

namespace {

constexpr int kThreads = 1024;  // of the first launch and the backward pass
constexpr int kWaves = kThreads / 64;
constexpr int kJoin = 256;  // threads of the second launch
constexpr int kJoinCols = 8;
// Rounds of rows that one workgroup takes by itself: eight rounds (512 x 128, 2048 x 4) take 10.8 and 8.6 us, with two
// launches 16.4 and 20.7 us; four (128 x 384) 8.6 and 24.6 us.
constexpr int64_t kSingleRounds = 8;
constexpr int kMaxBlocks = 256;    // workgroups of the first launch
constexpr int kMaxBackward = 512;  // and of the backward pass

typedef float f4_t __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------------------------
// Reductions over the LPR consecutive lanes of a row (4 <= LPR <= 64): every lane gets the same bits,
// since each step adds a pair of values that both partners hold.
template <int CTRL>
MX_DEV float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int LPR, typename F>
MX_DEV float across(float v, F f) {
  v = f(v, dpp<0xB1>(v));                    // lane ^ 1
  v = f(v, dpp<0x4E>(v));                    // lane ^ 2
  if (LPR == 8) v = f(v, __shfl_xor(v, 4));  // an 8-lane rotation is no DPP move
  if (LPR >= 16) {
    v = f(v, dpp<0x128>(v));  // rotate by 8 within 16 lanes
    v = f(v, dpp<0x124>(v));  // rotate by 4
  }
  if (LPR >= 32) v = f(v, __shfl_xor(v, 16));
  if (LPR >= 64) v = f(v, __shfl_xor(v, 32));
  return v;
}
struct Add { MX_DEV float operator()(float a, float b) const { return a + b; } };
struct Max { MX_DEV float operator()(float a, float b) const { return fmaxf(a, b); } };

// Column of value i of the lane lr of its row.
template <int LPR, int VPL, int VEC>
MX_DEV int column(int lr, int i) {
  return VEC == 4 ? ((i / 4) * LPR + lr) * 4 + (i & 3) : i * LPR + lr;
}

// One row's softmax in place: v holds the logits (-inf past E), then the probabilities.
template <int LPR, int VPL>
MX_DEV void softmax_row(float* v) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < VPL; i++) m = fmaxf(m, v[i]);
  m = across<LPR>(m, Max());
  const bool any = m > -INFINITY;  // no logit but -inf: nothing to share out
  if (!any) m = 0.0f;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; i++) {
    v[i] = __expf(v[i] - m);
    s += v[i];
  }
  s = across<LPR>(s, Add());
  const float r = any ? 1.0f / s : 0.0f;
#pragma unroll
  for (int i = 0; i < VPL; i++) v[i] *= r;
}

template <int LPR, int VPL, int VEC>
MX_DEV void load_row(const float* __restrict__ l, int E, int lr, float* v) {
  if (VEC == 4) {
#pragma unroll
    for (int c = 0; c < VPL / 4; c++) {
      const int col = (c * LPR + lr) * 4;
      f4_t x = f4_t{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (col < E) x = *reinterpret_cast<const f4_t*>(l + col);
#pragma unroll
      for (int j = 0; j < 4; j++) v[4 * c + j] = x[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; i++) {
      const int col = i * LPR + lr;
      v[i] = -INFINITY;
      if (col < E) v[i] = l[col];
    }
  }
}

// Sums of a and b over the workgroup, to every thread; red: 2 * 16 values.
MX_DEV void block_sums(double& a, double& b, double* red) {
#pragma unroll
  for (int h = 1; h < 64; h <<= 1) {
    a += __shfl_xor(a, h);
    b += __shfl_xor(b, h);
  }
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    red[wave] = a;
    red[16 + wave] = b;
  }
  __syncthreads();
  a = b = 0.0;
  for (int w = 0; w < waves; w++) {
    a += red[w];
    b += red[16 + w];
  }
}

// loss and coef from the joined sums; one workgroup, all threads.  n and S may be global or LDS.
MX_DEV void finish(int E, int k, const int32_t* n, const double* S, int64_t V, float* loss, float* coef, double* red) {
  const int t = threadIdx.x, nt = blockDim.x;
  double dot = 0.0, pairs = 0.0;
  for (int e = t; e < E; e += nt) {
    dot += (double)n[e] * S[e];
    pairs += (double)n[e];
  }
  block_sums(dot, pairs, red);
  const double each = V > 0 ? (double)E / ((double)k * (double)V * (double)V) : 0.0;
  const double mean = pairs / (double)E;
  if (t == 0) *loss = (float)(each * dot);
  for (int e = t; e < E; e += nt) coef[e] = (float)(each * ((double)n[e] - mean));
}

// What a workgroup found about a column: the sum of its probabilities, its pairs.
struct Part {
  float p;
  int32_t n;
};

template <int LPR, int VPL, int VEC>
__global__ __launch_bounds__(kThreads) void balance_forward_kernel(BalanceArgs a, Part* __restrict__ parts,
                                                                   int32_t* __restrict__ part_v, uint32_t* ticket) {
  constexpr int RPW = 64 / LPR;
  constexpr int GROUPS = kWaves * RPW;  // rows in flight in the workgroup
  constexpr int COLS = LPR * VPL;
  __shared__ float cols[kWaves * COLS];
  __shared__ int32_t hist[COLS];
  __shared__ int32_t live_in[kWaves];
  const int t = threadIdx.x, E = a.E;
  const int lr = t & (LPR - 1), group = t / LPR;
  for (int e = t; e < E; e += kThreads) hist[e] = 0;
  __syncthreads();

  // the pairs' experts: a contiguous range of pairs a workgroup
  const int64_t pairs = a.T * a.k, per = (pairs + gridDim.x - 1) / gridDim.x;
  const int64_t p1 = min(pairs, (int64_t)(blockIdx.x + 1) * per);
  for (int64_t p = (int64_t)blockIdx.x * per + t; p < p1; p += kThreads) {
    const int32_t e = a.ids[p];
    const bool counts = !a.mask || a.mask[(uint32_t)p / (uint32_t)a.k];  // T * k < 2^31
    if (counts && e >= 0 && e < E) atomicAdd(&hist[e], 1);
  }

  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; i++) acc[i] = 0.0f;
  int32_t live = 0;
  // two rows at a time: the loads of both are on their way before either is worked on
  const int64_t stride = (int64_t)gridDim.x * GROUPS;
  for (int64_t r = (int64_t)blockIdx.x * GROUPS + group; r < a.T; r += 2 * stride) {
    // uniform over a row's lanes, which exchange among themselves alone
    const bool second = r + stride < a.T;
    const bool live0 = !a.mask || a.mask[r], live1 = second && (!a.mask || a.mask[r + stride]);
    float v[2][VPL];
    if (live0) load_row<LPR, VPL, VEC>(a.logits + r * a.ldl, E, lr, v[0]);
    if (live1) load_row<LPR, VPL, VEC>(a.logits + (r + stride) * a.ldl, E, lr, v[1]);
    if (live0) {
      softmax_row<LPR, VPL>(v[0]);
#pragma unroll
      for (int i = 0; i < VPL; i++) acc[i] += v[0][i];
      live++;
    }
    if (live1) {
      softmax_row<LPR, VPL>(v[1]);
#pragma unroll
      for (int i = 0; i < VPL; i++) acc[i] += v[1][i];
      live++;
    }
  }
  // the wave's rows first, by their lanes, then the waves in LDS
  const int wave = t >> 6;
#pragma unroll
  for (int h = LPR; h < 64; h <<= 1) {
#pragma unroll
    for (int i = 0; i < VPL; i++) acc[i] += __shfl_xor(acc[i], h);
    live += __shfl_xor(live, h);
  }
  if ((t & 63) < LPR) {
#pragma unroll
    for (int i = 0; i < VPL; i++) cols[wave * COLS + column<LPR, VPL, VEC>(lr, i)] = acc[i];
  }
  if ((t & 63) == 0) live_in[wave] = live;
  __syncthreads();

  if (gridDim.x > 1) {
    for (int e = t; e < E; e += kThreads) {
      float s = 0.0f;
      for (int w = 0; w < kWaves; w++) s += cols[w * COLS + e];
      parts[(int64_t)blockIdx.x * E + e] = Part{s, hist[e]};
    }
    if (t == 0) {
      int32_t v = 0;
      for (int w = 0; w < kWaves; w++) v += live_in[w];
      part_v[blockIdx.x] = v;
      if (blockIdx.x == 0) *ticket = 0;  // for the second launch
    }
    return;
  }
  __shared__ double sums[COLS];
  __shared__ double red[32];
  for (int e = t; e < E; e += kThreads) {
    double s = 0.0;
    for (int w = 0; w < kWaves; w++) s += (double)cols[w * COLS + e];
    sums[e] = s;
    a.counts[e] = hist[e];
  }
  int64_t V = 0;
  for (int w = 0; w < kWaves; w++) V += live_in[w];
  __syncthreads();
  finish(E, a.k, hist, sums, V, a.loss, a.coef, red);
}

// Joins the partial sums of `blocks` <= kMaxBlocks workgroups: kJoinCols columns a workgroup, the blocks spread over
// its groups of kJoinCols threads.  The last workgroup to finish has the loss.
__global__ __launch_bounds__(kJoin) void balance_join_kernel(BalanceArgs a, int32_t blocks,
                                                             const Part* __restrict__ parts,
                                                             const int32_t* __restrict__ part_v, double* sums,
                                                             uint32_t* ticket) {
  constexpr int SPLIT = kJoin / kJoinCols, LOADS = kMaxBlocks / SPLIT;
  __shared__ double reds[kJoin / 64][kJoinCols];
  __shared__ int32_t redn[kJoin / 64][kJoinCols];
  __shared__ double red[32];
  __shared__ bool last;
  const int t = threadIdx.x, E = a.E;
  const int c = t % kJoinCols, part = t / kJoinCols, e = blockIdx.x * kJoinCols + c;
  Part p[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; i++) {
    const int b = part + i * SPLIT;
    p[i] = Part{0.0f, 0};
    if (b < blocks && e < E) p[i] = parts[(int64_t)b * E + e];
  }
  double s = 0.0;
  int32_t n = 0;
#pragma unroll
  for (int i = 0; i < LOADS; i++) {
    s += (double)p[i].p;
    n += p[i].n;
  }
#pragma unroll
  for (int h = kJoinCols; h < 64; h <<= 1) {
    s += __shfl_xor(s, h);
    n += __shfl_xor(n, h);
  }
  if ((t & 63) < kJoinCols) {
    reds[t >> 6][c] = s;
    redn[t >> 6][c] = n;
  }
  __syncthreads();
  if (t < 64) {  // the first wave: it publishes the columns and takes a number
    if (t < kJoinCols && e < E) {
      for (int w = 1; w < kJoin / 64; w++) {
        s += reds[w][c];
        n += redn[w][c];
      }
      sums[e] = s;
      a.counts[e] = n;
    }
    __threadfence();
    if (t == 0)
      last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double v = 0.0, none = 0.0;  // the tokens that count
  for (int b = t; b < blocks; b += kJoin) v += (double)part_v[b];
  block_sums(v, none, red);
  __syncthreads();
  finish(E, a.k, a.counts, sums, (int64_t)v, a.loss, a.coef, red);
}

template <int LPR, int VPL, int VEC>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(const float* __restrict__ logits, int64_t T, int E,
                                                                    int64_t ldl, const uint8_t* __restrict__ mask,
                                                                    const float* __restrict__ coef,
                                                                    const float* __restrict__ grad_loss,
                                                                    float* __restrict__ grad) {
  constexpr int GROUPS = kWaves * (64 / LPR);
  const int lr = threadIdx.x & (LPR - 1), group = threadIdx.x / LPR;
  const float g = *grad_loss;
  float d[VPL];
#pragma unroll
  for (int i = 0; i < VPL; i++) {
    const int col = column<LPR, VPL, VEC>(lr, i);
    d[i] = col < E ? coef[col] : 0.0f;
  }
  for (int64_t r = (int64_t)blockIdx.x * GROUPS + group; r < T; r += (int64_t)gridDim.x * GROUPS) {
    float v[VPL];
    if (!mask || mask[r]) {
      load_row<LPR, VPL, VEC>(logits + r * ldl, E, lr, v);
      softmax_row<LPR, VPL>(v);
      // the weighted mean of d, taken off twice: where one expert holds nearly all of the row, its own d
      // less the mean is small, and what the first mean's rounding left would be all of it
      float mean = 0.0f, rest = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; i++) mean += v[i] * d[i];
      mean = across<LPR>(mean, Add());
#pragma unroll
      for (int i = 0; i < VPL; i++) rest += v[i] * (d[i] - mean);
      rest = across<LPR>(rest, Add());
#pragma unroll
      for (int i = 0; i < VPL; i++) v[i] = g * v[i] * ((d[i] - mean) - rest);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; i++) v[i] = 0.0f;
    }
    float* out = grad + r * E;
    if (VEC == 4) {
#pragma unroll
      for (int c = 0; c < VPL / 4; c++) {
        const int col = (c * LPR + lr) * 4;
        if (col < E) *reinterpret_cast<f4_t*>(out + col) = f4_t{v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; i++) {
        const int col = i * LPR + lr;
        if (col < E) out[col] = v[i];
      }
    }
  }
}

// Lanes and values per row: VPL * LPR >= E, short reductions for few experts, at most 16 values a lane.
// f is called with the constants of the variant.
template <int L, int V>
struct RowShape { static constexpr int LPR = L, VPL = V; };
template <typename F>
int with_shape(int E, F f) {
  if (E <= 16) return f(RowShape<4, 4>());
  if (E <= 32) return f(RowShape<8, 4>());
  if (E <= 64) return f(RowShape<16, 4>());
  if (E <= 128) return f(RowShape<16, 8>());
  if (E <= 256) return f(RowShape<32, 8>());
  if (E <= 384) return f(RowShape<32, 12>());
  if (E <= 512) return f(RowShape<32, 16>());
  if (E <= 768) return f(RowShape<64, 12>());
  return f(RowShape<64, 16>());
}
template <typename R>
constexpr int rows_in_flight() { return kWaves * (64 / R::LPR); }

bool vec4(const void* p, int64_t ld, int E) { return E % 4 == 0 && ld % 4 == 0 && ((uintptr_t)p & 15) == 0; }

int status() { return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE; }

}  // namespace

int32_t balance_blocks(int64_t T, int32_t E) {
  return with_shape(E, [&](auto r) {
    const int64_t n = (T + rows_in_flight<decltype(r)>() - 1) / rows_in_flight<decltype(r)>();
    return n <= kSingleRounds ? 1 : (int)(n < kMaxBlocks ? n : kMaxBlocks);
  });
}

int launch_balance_forward(const BalanceArgs& a, const BalanceWs& w, uint8_t* ws, hipStream_t stream) {
  Part* parts = (Part*)(ws + w.parts);
  int32_t* pv = (int32_t*)(ws + w.part_v);
  uint32_t* ticket = (uint32_t*)(ws + w.ticket);
  const int st = with_shape(a.E, [&](auto r) {
    using R = decltype(r);
    if (vec4(a.logits, a.ldl, a.E))
      hipLaunchKernelGGL((balance_forward_kernel<R::LPR, R::VPL, 4>), dim3(w.blocks), dim3(kThreads), 0, stream, a, parts,
                         pv, ticket);
    else
      hipLaunchKernelGGL((balance_forward_kernel<R::LPR, R::VPL, 1>), dim3(w.blocks), dim3(kThreads), 0, stream, a, parts,
                         pv, ticket);
    return status();
  });
  if (st || w.blocks == 1) return st;
  hipLaunchKernelGGL(balance_join_kernel, dim3((a.E + kJoinCols - 1) / kJoinCols), dim3(kJoin), 0, stream, a, w.blocks,
                     parts, pv, (double*)(ws + w.sums), ticket);
  return status();
}

int launch_balance_backward(const float* logits, int64_t T, int32_t E, int64_t ldl, const uint8_t* mask,
                            const float* coef, const float* grad_loss, float* grad, hipStream_t stream) {
  return with_shape(E, [&](auto r) {
    using R = decltype(r);
    const int64_t n = (T + rows_in_flight<R>() - 1) / rows_in_flight<R>();
    const dim3 grid((unsigned)(n < kMaxBackward ? n : kMaxBackward));
    if (vec4(logits, ldl, E) && vec4(grad, E, E))
      hipLaunchKernelGGL((balance_backward_kernel<R::LPR, R::VPL, 4>), grid, dim3(kThreads), 0, stream, logits, T, E,
                         ldl, mask, coef, grad_loss, grad);
    else
      hipLaunchKernelGGL((balance_backward_kernel<R::LPR, R::VPL, 1>), grid, dim3(kThreads), 0, stream, logits, T, E,
                         ldl, mask, coef, grad_loss, grad);
    return status();
  });
}
