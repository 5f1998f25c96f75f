// Launchers of the balance loss, the 4-bit matrix-vector products and the block-quantized paged cache
// (each defined next to its kernels), and the argument structures they share with ops_api.cpp, which
// validates.  Host C++ and device code.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/mxfp4moe.h"

// ---------------------------------------------------------------------------------------------
// Balance loss (balance.hip).  Workspace: per-workgroup partial column sums and counts, the joined
// column sums and a ticket.
struct BalanceWs {
  uint64_t parts, part_v, sums, ticket, total;
  int32_t blocks;  // workgroups of the first launch
};
// Workgroups of the forward pass over T tokens and E experts; 1: it finishes by itself.
int32_t balance_blocks(int64_t T, int32_t E);

struct BalanceArgs {
  const float* logits;
  int64_t T, ldl;
  int32_t E, k;
  const int32_t* ids;
  const uint8_t* mask;  // may be NULL
  int32_t* counts;
  float *loss, *coef;
};
int launch_balance_forward(const BalanceArgs& a, const BalanceWs& w, uint8_t* ws, hipStream_t stream);
int launch_balance_backward(const float* logits, int64_t T, int32_t E, int64_t ldl, const uint8_t* mask,
                            const float* coef, const float* grad_loss, float* grad, hipStream_t stream);

// ---------------------------------------------------------------------------------------------
// Matrix-vector products (matvec.hip).  The dense form is the expert form with one expert whose rows are
// the M rows of x: offsets and pairs are then NULL.
struct MatvecArgs {
  const uint8_t *wq, *ws;   // [E, N, K/2], [E, N, K/B]
  const float* gscales;     // device [E] (expert form), or NULL: gscale
  float gscale;
  const void* bias;         // [E, N] or NULL
  int32_t bias_fp32;
  const uint16_t* x;
  int64_t ldx;
  void* y;
  int64_t ldy;
  int32_t out_fp32, swiglu;
  int32_t E, top_k;
  int64_t N, K, M;          // M: rows of x (dense) or pairs (expert form)
  const int32_t *offsets, *pairs;
};
int launch_matvec(int fmt, const MatvecArgs& a, hipStream_t stream);

// ---------------------------------------------------------------------------------------------
// Paged cache (cache.hip).
struct CachePlane {
  void* rows;       // bf16: read by the write, written by the read
  int64_t ldt, ldh;  // elements between tokens and between heads
  uint8_t *q, *s;
  int32_t dim;
  float gs;
};
struct CacheArgs {
  CachePlane plane[2];  // plane[1].dim == 0: one plane
  int64_t rows, num_pages, ld_table;
  const int32_t *cu, *start, *table;
  int32_t n_seqs, max_pages, page_size, heads;
};
int launch_cache_write(int fmt, const CacheArgs& a, hipStream_t stream);
int launch_cache_read(int fmt, const CacheArgs& a, hipStream_t stream);
