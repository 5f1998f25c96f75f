// The join of parts and the choice of the kernel: see attend_common.h.
#pragma once

#include "attend_shared.h"
#include "attend_split.h"

namespace {

// Joins the parts of the item that a worker begins and others go on with: a wave a row, blockIdx.y: rows of the tile.
template <int FMT, int DV, int NT>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(AttendArgs a, const float* __restrict__ part,
                                                               const float2* __restrict__ part_ml,
                                                               const Open* __restrict__ open,
                                                               const int64_t* __restrict__ totals, int workers) {
  constexpr int MT = 16 * NT, LANES = DV / 8, SIDES = 64 / LANES;  // lanes of a row of a part, parts side by side
  const Open it = open[blockIdx.x];
  if (it.rest <= 0) return;
  const int g = blockIdx.x / workers, worker = blockIdx.x % workers;
  const int lane = threadIdx.x & 63, e = lane % LANES * 8, side = lane / LANES;
  const Seq s = sequence(a, it.seq);
  const int there = min(MT, s.rows * a.group - it.tile * MT);
  // the worker of the item's last unit
  int64_t u0, u1;
  worker_range(*totals, workers, worker, u0, u1);
  const int64_t used = min((int64_t)workers, *totals);
  const int last = (int)(((u1 + it.rest) * used - 1) / *totals), n = last - worker + 1;
  // the first part is the second of its worker's two, the others are the first of theirs
  const auto slot = [&](int i) { return 2 * ((int64_t)g * workers + worker + i) + (i == 0 ? 1 : 0); };
  for (int r = blockIdx.y * (kThreads / 64) + (threadIdx.x >> 6); r < there; r += gridDim.y * (kThreads / 64)) {
    float top = -INFINITY;
    for (int i = lane; i < n; i += 64) top = fmaxf(top, part_ml[slot(i) * MT + r].x);
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) top = fmaxf(top, __shfl_xor(top, h));
    f32x4_t x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
    float sum = 0.0f;
    if (top > -INFINITY) {
#pragma unroll 4
      for (int i = side; i < n; i += SIDES) {
        const float2 ml = part_ml[slot(i) * MT + r];
        const f32x4_t* src = reinterpret_cast<const f32x4_t*>(part + (slot(i) * MT + r) * DV + e);
        const float f = __builtin_amdgcn_exp2f(ml.x - top);
        const f32x4_t p = src[0], q = src[1];
        sum += f * ml.y;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          x[j] += f * p[j];
          y[j] += f * q[j];
        }
      }
    }
#pragma unroll
    for (int h = LANES; h < 64; h <<= 1) {
      sum += __shfl_xor(sum, h);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        x[j] += __shfl_xor(x[j], h);
        y[j] += __shfl_xor(y[j], h);
      }
    }
    if (side == 0 && e < a.cache.plane[1].dim) write_row<FMT>(a, s, it.tile * MT + r, g, e, x, y, sum);
  }
}

// ---------------------------------------------------------------------------------------------

template <int FMT, int DV, int NT, typename F>
int launch_both(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream, F kernel) {
  float* part = (float*)(ws + p.part);
  float2* ml = (float2*)(ws + p.ml);
  Open* open = (Open*)(ws + p.open);
  int64_t* totals = (int64_t*)(ws + p.totals);
  const unsigned n = (unsigned)p.workers * (unsigned)a.cache.heads;
  hipLaunchKernelGGL(kernel, dim3(n), dim3(kThreads), 0, stream, a, part, ml, open, totals, p.workers);
  if (hipGetLastError() != hipSuccess) return MXFP4_ERR_DEVICE;
  // one unit holds the longest context that the table can: nothing to join
  if ((int64_t)a.cache.max_pages * a.cache.page_size <= p.unit) return MXFP4_OK;
  hipLaunchKernelGGL((attend_join_kernel<FMT, DV, NT>), dim3(n, 2 * NT), dim3(kThreads), 0, stream, a, part, ml, open, totals, p.workers);
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

template <int FMT, int DK, int DV>
int launch_dims(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  const CacheArgs& c = a.cache;
  const bool paged = c.page_size % kTile == 0 && c.plane[0].dim == DK && c.plane[1].dim == DV;
  if (p.nt == 1)
    return launch_both<FMT, DV, 1>(a, p, ws, stream, paged ? attend_split_kernel<FMT, DK, DV, 1, attend_waves(DK, 1), true>
                                                           : attend_split_kernel<FMT, DK, DV, 1, attend_waves(DK, 1), false>);
  if (p.nt == 2)
    return launch_both<FMT, DV, 2>(a, p, ws, stream, paged ? attend_split_kernel<FMT, DK, DV, 2, attend_waves(DK, 2), true>
                                                           : attend_split_kernel<FMT, DK, DV, 2, attend_waves(DK, 2), false>);
  constexpr int KEYS = attend_keys(DK);
  if constexpr (KEYS == 64)
    if (p.nt == 4) return launch_both<FMT, DV, 4>(a, p, ws, stream, attend_shared_kernel<FMT, DK, DV, 2, KEYS, attend_waves(DK, 4)>);
  return launch_both<FMT, DV, 8>(a, p, ws, stream, attend_shared_kernel<FMT, DK, DV, 4, KEYS, attend_waves(DK, 8)>);
}

template <int FMT>
int launch_format(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  if (p.dk == 64) return launch_dims<FMT, 64, 64>(a, p, ws, stream);
  if (p.dk == 128) return launch_dims<FMT, 128, 128>(a, p, ws, stream);
  if (p.dk == 192) return launch_dims<FMT, 192, 128>(a, p, ws, stream);
  return launch_dims<FMT, 256, 256>(a, p, ws, stream);
}

}  // namespace
