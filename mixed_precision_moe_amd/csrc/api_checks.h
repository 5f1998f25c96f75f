// What the argument checks of the operators' C entry points share: limits, alignment, formats, the cache's sizes.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/mxfp4moe.h"

#define MX_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31;   // tokens, pairs
constexpr int64_t kMaxWidth = int64_t(1) << 20;  // N, K, heads * dim
constexpr int64_t kMaxLd = int64_t(1) << 40;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline hipStream_t S(void* s) { return (hipStream_t)s; }
inline uint64_t up256(uint64_t v) { return (v + 255) & ~uint64_t(255); }

// positive and finite (the comparison also rejects NaN)
inline bool good_scale(float g) { return g > 0.0f && g <= 3.40282347e38f; }

inline int group_of(int32_t fmt) {
  return fmt == MXFP4_FMT_MXFP4 || fmt == MXFP4_FMT_MXFP8 ? 32 : fmt == MXFP4_FMT_NVFP4 ? 16 : 0;
}

inline int check_flags(int32_t a, int32_t b, int32_t c) {
  return ((a | b | c) & ~1) ? MXFP4_ERR_SHAPE : MXFP4_OK;
}

inline int check_cache(const mxfp4_cache_dims* d, bool v) {
  if (!d) return MXFP4_ERR_NULL;
  const int g = group_of(d->fmt);
  if (!g) return MXFP4_ERR_LAYOUT;
  if (d->heads < 1 || d->page_size < 1 || d->num_pages < 0 || d->k_dim < g || d->k_dim % g || d->v_dim < 0 ||
      d->v_dim % g || (int64_t)d->heads * d->k_dim > kMaxWidth || (int64_t)d->heads * d->v_dim > kMaxWidth)
    return MXFP4_ERR_SHAPE;
  // keeps byte offsets into a plane in 63 bits, with room
  if (d->num_pages > kMaxRows || d->num_pages * d->page_size > kMaxLd) return MXFP4_ERR_SHAPE;
  if (d->fmt == MXFP4_FMT_NVFP4 && (!good_scale(d->k_global_scale) || (v && !good_scale(d->v_global_scale))))
    return MXFP4_ERR_SHAPE;
  return MXFP4_OK;
}

}  // namespace
