// The join of parts and the choice of the kernel: see attend_common.h.
#pragma once

#include "attend_shared.h"
#include "attend_split.h"

namespace {

// Joins the parts of the item that a worker begins and another ends; blockIdx.y: sixteen of its rows.
template <int FMT, int DV, int NT>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(AttendArgs a, const float* __restrict__ part,
                                                               const float2* __restrict__ part_ml,
                                                               const Open* __restrict__ open, int workers) {
  constexpr int MT = 16 * NT;
  const Open it = open[blockIdx.x];
  if (it.last < 0) return;
  const int g = blockIdx.x / workers, worker = blockIdx.x % workers;
  const Seq s = sequence(a, it.seq);
  const int there = min(MT, s.rows * a.group - it.tile * MT);
  for (int id = threadIdx.x; id < 16 * (DV / 8); id += kThreads) {
    const int r = 16 * blockIdx.y + id / (DV / 8), e = id % (DV / 8) * 8;
    if (r >= there || e >= a.cache.plane[1].dim) continue;
    // the first part is the second of its worker's two, the others are the first of theirs
    auto slot = [&](int w) { return 2 * ((int64_t)g * workers + w) + (w == worker ? 1 : 0); };
    float top = -INFINITY;
    for (int w = worker; w <= it.last; w++) top = fmaxf(top, part_ml[slot(w) * MT + r].x);
    f32x4_t x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
    float sum = 0.0f;
    if (top > -INFINITY) {
#pragma unroll 4
      for (int w = worker; w <= it.last; w++) {
        const float2 ml = part_ml[slot(w) * MT + r];
        const f32x4_t* src = reinterpret_cast<const f32x4_t*>(part + (slot(w) * MT + r) * DV + e);
        const float f = __builtin_amdgcn_exp2f(ml.x - top);
        const f32x4_t p = src[0], q = src[1];
        sum += f * ml.y;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          x[i] += f * p[i];
          y[i] += f * q[i];
        }
      }
    }
    write_row<FMT>(a, s, it.tile * MT + r, g, e, x, y, sum);
  }
}

// ---------------------------------------------------------------------------------------------

template <int FMT, int DV, int NT, typename F>
int launch_both(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream, F kernel) {
  float* part = (float*)(ws + p.part);
  float2* ml = (float2*)(ws + p.ml);
  Open* open = (Open*)(ws + p.open);
  const unsigned n = (unsigned)p.workers * (unsigned)a.cache.heads;
  hipLaunchKernelGGL(kernel, dim3(n), dim3(kThreads), 0, stream, a, part, ml, open, p.workers);
  if (hipGetLastError() != hipSuccess) return MXFP4_ERR_DEVICE;
  // one unit holds the longest context that the table can: nothing to join
  if ((int64_t)a.cache.max_pages * a.cache.page_size <= p.unit) return MXFP4_OK;
  hipLaunchKernelGGL((attend_join_kernel<FMT, DV, NT>), dim3(n, NT), dim3(kThreads), 0, stream, a, part, ml, open, p.workers);
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
