// The join of parts and the choice of the kernel: see attend_common.h.
#pragma once

#include "attend_shared.h"
#include "attend_split.h"

namespace {

// Joins the parts of the items that a worker begins and others go on with.  blockIdx.x: entry of `open`, blockIdx.y: rows of
// the tile, blockIdx.z: the head in the worker's group.  A row of a part is LANES lanes; the rest of the wave's have other
// rows where the parts are few, else other parts of the same row; kAhead parts are asked for at a time.  Bound by the parts'
// trip: 67 MB of 2 x 1024 rows of 8 x 4 heads join in 14 us, 64 parts of one context's 35 rows a head in 7.7 (22 with a
// workgroup for each of a tile's rows that takes a part after the other).
template <int FMT, int DV, int NT>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(AttendArgs a, const float* __restrict__ part,
                                                               const float2* __restrict__ part_ml,
                                                               const Open* __restrict__ open,
                                                               const Totals* __restrict__ totals, int workers) {
  constexpr int MT = 16 * NT, LANES = DV / 8, SIDES = 64 / LANES, kFew = 8, kAhead = 4;
  const int entries = a.open_items ? a.open_items : workers;
  if (a.open_items && blockIdx.x % entries >= totals->items) return;
  const Open it = open[blockIdx.x];
  if (it.rest <= 0) return;
  const int g = (blockIdx.x / entries << a.heads_log) + blockIdx.z;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = lane % LANES * 8, side = lane / LANES;
  const Seq s = sequence(a, it.seq);
  const int there = min(MT, s.rows * a.group - it.tile * MT);
  // the worker of the item's last unit
  const int64_t all = totals->units, used = min((int64_t)workers, all);
  int64_t u0, u1;
  worker_range(all, workers, it.worker, u0, u1);
  const int n = (int)(((u1 + it.rest) * used - 1) / all) - it.worker + 1;
  const bool few = n <= kFew;
  const int per_wave = few ? SIDES : 1, step = few ? 1 : SIDES;
  for (int r0 = (blockIdx.y * (kThreads / 64) + wave) * per_wave; r0 < there; r0 += gridDim.y * (kThreads / 64) * per_wave) {
    const int r = few ? min(r0 + side, there - 1) : r0;
    // the first part is the second of its worker's two, the others are the first of theirs
    const int64_t first = 2 * ((int64_t)g * workers + it.worker);
    f32x4_t x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
    float sum = 0.0f, top = -INFINITY;
    for (int i = few ? 0 : side; i < n; i += kAhead * step) {
      float2 ml[kAhead];
      f32x4_t p[kAhead], q[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; j++) {
        const int k = min(i + j * step, n - 1);
        const int64_t at = (k == 0 ? first + 1 : first + 2 * k) * MT + r;
        ml[j] = part_ml[at];
        const f32x4_t* src = reinterpret_cast<const f32x4_t*>(part + at * DV + e);
        p[j] = src[0];
        q[j] = src[1];
        if (i + j * step >= n) ml[j] = float2{-INFINITY, 0.0f};
      }
      float now = top;
#pragma unroll
      for (int j = 0; j < kAhead; j++) now = fmaxf(now, ml[j].x);
      const float by = now > -INFINITY ? now : 0.0f, keep = __builtin_amdgcn_exp2f(top - by);
      top = now;
      sum *= keep;
#pragma unroll
      for (int c = 0; c < 4; c++) {
        x[c] *= keep;
        y[c] *= keep;
      }
#pragma unroll
      for (int j = 0; j < kAhead; j++) {
        const float f = __builtin_amdgcn_exp2f(ml[j].x - by);  // 0 too: a part's NaN stays one
        sum += f * ml[j].y;
#pragma unroll
        for (int c = 0; c < 4; c++) {
          x[c] += f * p[j][c];
          y[c] += f * q[j][c];
        }
      }
    }
    if (!few) {
#pragma unroll
      for (int h = LANES; h < 64; h <<= 1) {
        const float other = __shfl_xor(top, h), now = fmaxf(top, other), by = now > -INFINITY ? now : 0.0f;
        const float f = __builtin_amdgcn_exp2f(top - by), o = __builtin_amdgcn_exp2f(other - by);
        top = now;
        sum = sum * f + __shfl_xor(sum, h) * o;
#pragma unroll
        for (int c = 0; c < 4; c++) {
          x[c] = x[c] * f + __shfl_xor(x[c], h) * o;
          y[c] = y[c] * f + __shfl_xor(y[c], h) * o;
        }
      }
    }
    if ((few ? r0 + side < there : side == 0) && e < a.cache.plane[1].dim)
      write_row<FMT>(a, s, it.tile * MT + r, g, e, x, y, sum);
  }
}

// ---------------------------------------------------------------------------------------------

template <int FMT, int DV, int NT, typename F>
int launch_both(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream, F kernel, int threads = kThreads) {
  float* part = (float*)(ws + p.part);
  float2* ml = (float2*)(ws + p.ml);
  Open* open = (Open*)(ws + p.open);
  Totals* totals = (Totals*)(ws + p.totals);
  const unsigned n = (unsigned)p.workers * ((unsigned)a.cache.heads >> p.heads_log);
  hipLaunchKernelGGL(kernel, dim3(n), dim3(threads), 0, stream, a, part, ml, open, totals, p.workers);
  if (hipGetLastError() != hipSuccess) return MXFP4_ERR_DEVICE;
  // one unit holds the longest context that the table can: nothing to join
  if ((int64_t)a.cache.max_pages * a.cache.page_size <= 1 << p.unit_log) return MXFP4_OK;
  // at most `workers` items are in parts; enough workgroups to have their rows side by side
  const unsigned groups = (unsigned)a.cache.heads >> p.heads_log, heads = 1u << p.heads_log;
  const unsigned entries = groups * (unsigned)(a.open_items ? a.open_items : p.workers);
  const unsigned rows = min(4u * NT, max((unsigned)NT, 2048u / (entries * heads)));
  hipLaunchKernelGGL((attend_join_kernel<FMT, DV, NT>), dim3(entries, rows, heads), dim3(kThreads), 0, stream, a, part, ml, open,
                     totals, p.workers);
  return hipGetLastError() == hipSuccess ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

template <int FMT, bool FINE, int DK, int DV>
int launch_dims(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  const CacheArgs& c = a.cache;
  const bool paged = c.page_size % kTile == 0 && c.plane[0].dim == DK && c.plane[1].dim == DV;
  if constexpr (!FINE)  // with two terms of the weights whatever the result's type is
    if (p.nt == 1)
      return launch_both<FMT, DV, 1>(a, p, ws, stream, paged ? attend_split_kernel<FMT, DK, DV, 1, attend_waves(DK, 1), true, true>
                                                             : attend_split_kernel<FMT, DK, DV, 1, attend_waves(DK, 1), false, true>);
  if (p.nt == 2)
    return launch_both<FMT, DV, 2>(a, p, ws, stream, paged ? attend_split_kernel<FMT, DK, DV, 2, attend_waves(DK, 2), true, FINE>
                                                           : attend_split_kernel<FMT, DK, DV, 2, attend_waves(DK, 2), false, FINE>);
  if constexpr (DK <= 128)
    if (p.nt == 4) return launch_both<FMT, DV, 4>(a, p, ws, stream, attend_shared_kernel<FMT, DK, DV, 2, 4, 2, attend_waves(DK, 4), FINE>);
  constexpr int W8 = attend_size(DK, 8), W16 = attend_size(DK, 16);
  if constexpr (DK <= 192)
    if (p.nt == 16)
      return launch_both<FMT, DV, 16>(a, p, ws, stream, attend_shared_kernel<FMT, DK, DV, 2, W16, 8, attend_waves(DK, 16), FINE>, 64 * W16);
  constexpr int NT = attend_columns(DK);
  return launch_both<FMT, DV, 8>(a, p, ws, stream, attend_shared_kernel<FMT, DK, DV, NT, W8, 8 / NT, attend_waves(DK, 8), FINE>, 64 * W8);
}

// FINE: for results in fp32 and more than 16 rows a key head.
template <int FMT, bool FINE>
int launch_format(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  if (p.dk == 64) return launch_dims<FMT, FINE, 64, 64>(a, p, ws, stream);
  if (p.dk == 128) return launch_dims<FMT, FINE, 128, 128>(a, p, ws, stream);
  if (p.dk == 192) return launch_dims<FMT, FINE, 192, 128>(a, p, ws, stream);
  return launch_dims<FMT, FINE, 256, 256>(a, p, ws, stream);
}

}  // namespace
