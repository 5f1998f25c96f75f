// C ABI of the balance loss, the 4-bit matrix-vector products and the block-quantized paged cache:
// argument validation before any device work, then the launches.  Declarations and contracts are in
// include/mxfp4moe.h.
#include <hip/hip_runtime_api.h>

#include "api_checks.h"
#include "ops.h"

namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxTopK = 32;

int check_balance(int64_t T, int32_t E, int32_t top_k, int64_t ldl) {
  if (T < 0 || E < 1 || E > kMaxE || top_k < 1 || top_k > E || top_k > kMaxTopK) return MXFP4_ERR_SHAPE;
  if (T * top_k >= kMaxRows || T >= kMaxRows || ldl < E || ldl > kMaxLd) return MXFP4_ERR_SHAPE;
  return MXFP4_OK;
}

BalanceWs balance_ws(int64_t T, int32_t E) {
  BalanceWs w;
  w.blocks = balance_blocks(T, E);
  uint64_t p = 0;
  auto take = [&](uint64_t bytes) { uint64_t o = p; p = up256(p + bytes); return o; };
  const uint64_t cells = (uint64_t)w.blocks * (uint64_t)E;
  w.parts = take(8 * cells);
  w.part_v = take(4 * (uint64_t)w.blocks);
  w.sums = take(8 * (uint64_t)E);
  w.ticket = take(4);
  w.total = p;
  return w;
}

int check_matvec(int32_t fmt, int64_t N, int64_t K) {
  if (fmt != MXFP4_FMT_MXFP4 && fmt != MXFP4_FMT_NVFP4) return MXFP4_ERR_LAYOUT;
  if (N < 1 || N > kMaxWidth || K < 32 || K > kMaxWidth || K % group_of(fmt)) return MXFP4_ERR_SHAPE;
  return MXFP4_OK;
}

int cache_args(CacheArgs& a, const mxfp4_cache_dims* d, const void* k, int64_t k_ldt, int64_t k_ldh, const void* v,
               int64_t v_ldt, int64_t v_ldh, int64_t rows, const int32_t* cu_rows, const int32_t* start,
               const int32_t* page_table, int64_t ld_table, int32_t n_seqs, int32_t max_pages, const void* k_q,
               const void* k_s, const void* v_q, const void* v_s) {
  int st = check_cache(d, d && d->v_dim > 0);
  if (st) return st;
  const bool two = d->v_dim > 0;
  if (rows < 0 || rows >= kMaxRows || n_seqs < 0 || max_pages < 0 || ld_table < max_pages || ld_table > kMaxLd)
    return MXFP4_ERR_SHAPE;
  auto bad_ld = [&](int64_t ldt, int64_t ldh, int32_t dim) {
    return ldt < 0 || ldt % 8 || ldt > kMaxLd || ldh < 0 || ldh % 8 || ldh > kMaxLd || (d->heads > 1 && ldh < dim) ||
           (rows > 1 && ldt < dim);
  };
  if (bad_ld(k_ldt, k_ldh, d->k_dim) || (two && bad_ld(v_ldt, v_ldh, d->v_dim))) return MXFP4_ERR_SHAPE;
  a = CacheArgs{};
  a.rows = n_seqs == 0 ? 0 : rows;
  if (a.rows == 0) return MXFP4_OK;
  // memory of no pages and a table of no columns may be NULL
  if (!k || !cu_rows || (!page_table && max_pages > 0) || (two && !v)) return MXFP4_ERR_NULL;
  if (d->num_pages > 0 && (!k_q || !k_s || (two && (!v_q || !v_s)))) return MXFP4_ERR_NULL;
  if (!aligned(k, 16) || !aligned(k_q, 8) || !aligned(cu_rows, 4) || !aligned(start, 4) || !aligned(page_table, 4) ||
      (two && (!aligned(v, 16) || !aligned(v_q, 8))))
    return MXFP4_ERR_ALIGN;
  a.plane[0] = CachePlane{(void*)k, k_ldt, k_ldh, (uint8_t*)k_q, (uint8_t*)k_s, d->k_dim, d->k_global_scale};
  if (two) a.plane[1] = CachePlane{(void*)v, v_ldt, v_ldh, (uint8_t*)v_q, (uint8_t*)v_s, d->v_dim, d->v_global_scale};
  a.num_pages = d->num_pages;
  a.ld_table = ld_table;
  a.cu = cu_rows;
  a.start = start;
  a.table = page_table;
  a.n_seqs = n_seqs;
  a.max_pages = max_pages;
  a.page_size = d->page_size;
  a.heads = d->heads;
  return MXFP4_OK;
}

}  // namespace

// ------------------------------------------------------------------------------------------------
// Balance loss.

MX_API size_t moe_balance_workspace_bytes(int64_t T, int32_t E) {
  if (check_balance(T, E, 1, E) != MXFP4_OK) return 0;
  return (size_t)balance_ws(T, E).total;
}

MX_API int moe_balance_forward(const float* router_logits, int64_t T, int32_t E, int64_t ldl, const int32_t* topk_ids,
                               int32_t top_k, const uint8_t* token_mask, float* loss, int32_t* counts, float* coef,
                               void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_balance(T, E, top_k, ldl);
  if (st) return st;
  if (!loss || !counts || !coef || !workspace) return MXFP4_ERR_NULL;
  if (T > 0 && (!router_logits || !topk_ids)) return MXFP4_ERR_NULL;
  if (!aligned(router_logits, 4) || !aligned(topk_ids, 4) || !aligned(loss, 4) || !aligned(counts, 4) ||
      !aligned(coef, 4) || !aligned(workspace, 256))
    return MXFP4_ERR_ALIGN;
  const BalanceWs w = balance_ws(T, E);
  if (workspace_bytes < w.total) return MXFP4_ERR_WORKSPACE;
  const BalanceArgs a = {router_logits, T, ldl, E, top_k, topk_ids, token_mask, counts, loss, coef};
  return launch_balance_forward(a, w, (uint8_t*)workspace, S(stream));
}

MX_API int moe_balance_backward(const float* router_logits, int64_t T, int32_t E, int64_t ldl,
                                const uint8_t* token_mask, const float* coef, const float* grad_loss,
                                float* grad_logits, void* stream) {
  int st = check_balance(T, E, 1, ldl);
  if (st) return st;
  if (T == 0) return MXFP4_OK;
  if (!router_logits || !coef || !grad_loss || !grad_logits) return MXFP4_ERR_NULL;
  if (!aligned(router_logits, 4) || !aligned(coef, 4) || !aligned(grad_loss, 4) || !aligned(grad_logits, 4))
    return MXFP4_ERR_ALIGN;
  return launch_balance_backward(router_logits, T, E, ldl, token_mask, coef, grad_loss, grad_logits, S(stream));
}

// ------------------------------------------------------------------------------------------------
// Matrix-vector products.

MX_API int fp4_matvec(int32_t fmt, const void* w_q, const void* w_s, float global_scale, int64_t N, int64_t K,
                      const void* bias, int32_t bias_is_fp32, const void* x_bf16, int64_t M, int64_t ldx, void* y,
                      int64_t ldy, int32_t out_is_fp32, void* stream) {
  int st = check_matvec(fmt, N, K);
  if (st || (st = check_flags(bias_is_fp32, out_is_fp32, 0))) return st;
  if (fmt == MXFP4_FMT_NVFP4 && !good_scale(global_scale)) return MXFP4_ERR_SHAPE;
  if (M < 0 || M > kMaxWidth || ldx < K || ldx % 8 || ldx > kMaxLd || ldy < N || ldy > kMaxLd) return MXFP4_ERR_SHAPE;
  if (M == 0) return MXFP4_OK;
  if (!w_q || !w_s || !x_bf16 || !y) return MXFP4_ERR_NULL;
  if (!aligned(w_q, 16) || !aligned(x_bf16, 16) || !aligned(y, out_is_fp32 ? 4 : 2) ||
      !aligned(bias, bias_is_fp32 ? 4 : 2))
    return MXFP4_ERR_ALIGN;
  MatvecArgs a = {};
  a.wq = (const uint8_t*)w_q;
  a.ws = (const uint8_t*)w_s;
  a.gscale = fmt == MXFP4_FMT_NVFP4 ? global_scale : 1.0f;
  a.bias = bias;
  a.bias_fp32 = bias_is_fp32;
  a.x = (const uint16_t*)x_bf16;
  a.ldx = ldx;
  a.y = y;
  a.ldy = ldy;
  a.out_fp32 = out_is_fp32;
  a.E = 1;
  a.top_k = 1;
  a.N = N;
  a.K = K;
  a.M = M;
  return launch_matvec(fmt, a, S(stream));
}

MX_API int fp4_expert_matvec(int32_t fmt, const void* w_q, const void* w_s, const float* global_scales, int32_t E,
                             int64_t N, int64_t K, const void* bias, int32_t bias_is_fp32, const void* x_bf16,
                             int64_t ldx, int32_t top_k, const int32_t* expert_offsets, const int32_t* sorted_pairs,
                             int64_t n_pairs, int32_t swiglu, void* y, int32_t out_is_fp32, void* stream) {
  int st = check_matvec(fmt, N, K);
  if (st || (st = check_flags(bias_is_fp32, out_is_fp32, swiglu))) return st;
  if (E < 1 || E > kMaxE || top_k < 1 || top_k > kMaxE || (swiglu && N % 2)) return MXFP4_ERR_SHAPE;
  if (n_pairs < 0 || n_pairs >= kMaxRows || n_pairs % top_k || ldx < K || ldx % 8 || ldx > kMaxLd)
    return MXFP4_ERR_SHAPE;
  if (n_pairs == 0) return MXFP4_OK;
  if (!w_q || !w_s || !x_bf16 || !y || !expert_offsets || !sorted_pairs) return MXFP4_ERR_NULL;
  if (fmt == MXFP4_FMT_NVFP4 && !global_scales) return MXFP4_ERR_NULL;
  if (!aligned(w_q, 16) || !aligned(x_bf16, 16) || !aligned(y, out_is_fp32 ? 4 : 2) ||
      !aligned(bias, bias_is_fp32 ? 4 : 2) || !aligned(expert_offsets, 4) || !aligned(sorted_pairs, 4) ||
      !aligned(global_scales, 4))
    return MXFP4_ERR_ALIGN;
  MatvecArgs a = {};
  a.wq = (const uint8_t*)w_q;
  a.ws = (const uint8_t*)w_s;
  a.gscales = fmt == MXFP4_FMT_NVFP4 ? global_scales : nullptr;
  a.gscale = 1.0f;
  a.bias = bias;
  a.bias_fp32 = bias_is_fp32;
  a.x = (const uint16_t*)x_bf16;
  a.ldx = ldx;
  a.y = y;
  a.ldy = swiglu ? N / 2 : N;
  a.out_fp32 = out_is_fp32;
  a.swiglu = swiglu;
  a.E = E;
  a.top_k = top_k;
  a.N = N;
  a.K = K;
  a.M = n_pairs;
  a.offsets = expert_offsets;
  a.pairs = sorted_pairs;
  return launch_matvec(fmt, a, S(stream));
}

// ------------------------------------------------------------------------------------------------
// Paged cache.

MX_API int mxfp4_cache_bytes(const mxfp4_cache_dims* d, size_t bytes_out[4]) {
  int st = check_cache(d, d && d->v_dim > 0);
  if (st) return st;
  if (!bytes_out) return MXFP4_ERR_NULL;
  const size_t slots = (size_t)d->num_pages * (size_t)d->page_size * (size_t)d->heads;
  const size_t per = d->fmt == MXFP4_FMT_MXFP8 ? 1 : 2, g = (size_t)group_of(d->fmt);
  const size_t dims[2] = {(size_t)d->k_dim, (size_t)d->v_dim};
  for (int i = 0; i < 2; i++) {
    bytes_out[2 * i] = slots * (dims[i] / per);
    bytes_out[2 * i + 1] = slots * (dims[i] / g);
  }
  return MXFP4_OK;
}

MX_API int mxfp4_cache_write(const mxfp4_cache_dims* d, const void* k_bf16, int64_t k_ldt, int64_t k_ldh,
                             const void* v_bf16, int64_t v_ldt, int64_t v_ldh, int64_t rows, const int32_t* cu_rows,
                             const int32_t* start, const int32_t* page_table, int64_t ld_table, int32_t n_seqs,
                             int32_t max_pages, void* k_q, void* k_s, void* v_q, void* v_s, void* stream) {
  CacheArgs a;
  int st = cache_args(a, d, k_bf16, k_ldt, k_ldh, v_bf16, v_ldt, v_ldh, rows, cu_rows, start, page_table, ld_table,
                      n_seqs, max_pages, k_q, k_s, v_q, v_s);
  if (st || a.rows == 0) return st;
  return launch_cache_write(d->fmt, a, S(stream));
}

MX_API int mxfp4_cache_read(const mxfp4_cache_dims* d, const void* k_q, const void* k_s, const void* v_q,
                            const void* v_s, int64_t rows, const int32_t* cu_rows, const int32_t* start,
                            const int32_t* page_table, int64_t ld_table, int32_t n_seqs, int32_t max_pages,
                            void* k_bf16, int64_t k_ldt, int64_t k_ldh, void* v_bf16, int64_t v_ldt, int64_t v_ldh,
                            void* stream) {
  CacheArgs a;
  int st = cache_args(a, d, k_bf16, k_ldt, k_ldh, v_bf16, v_ldt, v_ldh, rows, cu_rows, start, page_table, ld_table,
                      n_seqs, max_pages, k_q, k_s, v_q, v_s);
  if (st || a.rows == 0) return st;
  return launch_cache_read(d->fmt, a, S(stream));
}
