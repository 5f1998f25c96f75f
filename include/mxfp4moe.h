/*
 * mxfp4moe.h -- C ABI of the gfx950 (MI355X) MXFP4 quantization and MXFP4-weight MoE library.
 *
 * Page tags used in the citations below:
 *   [P1] prhub summary of vLLM PR #46915 (weight/scale interleave fix in the SM90 MXFP4 fused-MoE test)
 *   [P2] prhub report of vLLM PR #51038 "[Bugfix][Quantization] Fix MXFP4 conversion for FlashInfer CUTLASS"
 *   [P3] prhub summary of vLLM PR #43557 (E8M0 scale fix in the MXFP4 MoE CUTLASS kernel)
 *   [DEF] definitions this library adopts where the pages name a step without spelling it out: the
 *        OCP Microscaling MXFP4 format (32-element blocks, E2M1 round-to-nearest-even saturating at
 *        +-6, two nibbles per byte), top-k routing over softmax(logits), SwiGLU = silu(w1 half) *
 *        (w3 half), grouped GEMMs and a routing-weighted combine.
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are HIP device pointers owned by the caller; the library never
 *     allocates, frees or keeps them.  Host pointers ("host") are read during the call only.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).  All device work is
 *     enqueued on it; the calls return without synchronizing unless stated otherwise.
 *   - Arguments are validated before any device work; on failure nothing is written and a status
 *     below is returned.  Launch failures return MXFP4_ERR_DEVICE.  NaN/Inf inputs are outside the
 *     contract (no device-side checks).
 *   - Device pointers must be 16-byte aligned unless stated otherwise.
 */
#ifndef MXFP4MOE_H
#define MXFP4MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  MXFP4_OK = 0,
  MXFP4_ERR_NULL = 1,      /* a required pointer is NULL */
  MXFP4_ERR_SHAPE = 2,     /* a size or dimension is out of range */
  MXFP4_ERR_ALIGN = 3,     /* a pointer or stride breaks the alignment rule */
  MXFP4_ERR_WORKSPACE = 4, /* workspace or output buffer too small */
  MXFP4_ERR_LAYOUT = 5,    /* unknown layout flag, or a packed blob whose header does not match */
  MXFP4_ERR_DEVICE = 6     /* a HIP call or kernel launch failed */
};

/* Static, NUL-terminated description of a status code (unknown codes get a generic string). */
const char* mxfp4_status_str(int status);

/* Library version, (major << 16) | minor. */
uint32_t mxfp4_version(void);

/* ------------------------------------------------------------------------------------------------
 * MXFP4 block quantization.  [P3 Implementation breakdown item 1; Key source snippets: the E8M0
 * reference helper and the UE8M0_SF branch of the FP16/BF16 -> FP4 converter; DEF element rule]
 *
 * For each row of x and each 32-element block along K:
 *   amax = max |x| over the block (bf16 magnitudes, exact);
 *   e    = 0 if amax == 0, else B - 2 clamped to [0, 254], with B the biased exponent of the binary32
 *          bits of amax after adding 2^21 (significands >= 1.75 round up);
 *   code = E2M1 of |x| * 2^(127 - e), round to nearest even, saturating at 6; sign bit 0x8 copied
 *          from x (also when the magnitude code is 0);
 *   q[row][j] = code[2j] | code[2j+1] << 4  (element 2j in the low nibble).
 * x_bf16        device, bf16 [M, ldx] row-major; K % 32 == 0, ldx >= K, ldx % 8 == 0.
 *               Strided (ldx > K) input is read correctly: the pages' linear path had to force a
 *               contiguous copy before quantizing [P3 Implementation breakdown item 2]; here the
 *               stride is explicit.
 * q_u8          device, uint8 [M, K/2], required.
 * scale_flat_u8 device, uint8 [M, K/32], may be NULL; any alignment (byte stores are used unless the
 *               pointer is 4-byte aligned and K/32 is a multiple of 4, then whole dwords).
 * scale_tiled_u8 device, uint8 [ceil(M/128), ceil(K/128), 32, 4, 4], 16-byte aligned (each
 *               [mT][kT][oM] group of 16 bytes is written with one store), may be NULL: the byte at
 *               [mT][kT][oM][iM][iK] is the scale of row mT*128 + iM*32 + oM and scale column
 *               kT*4 + iK; padding bytes are written as 0.  [P3 Key source snippets, the untile
 *               helper's permute (0, 3, 2, 1, 4)]
 * M >= 0 (M == 0 is a no-op), K >= 32.
 */
int mxfp4_quantize(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, void* q_u8, void* scale_flat_u8,
                   void* scale_tiled_u8, void* stream);

/* Bytes of the tiled scale output for an [M, K] matrix: ceil(M/128) * ceil(K/128) * 512. */
size_t mxfp4_tiled_scale_bytes(int64_t M, int64_t K);

/* ------------------------------------------------------------------------------------------------
 * NVFP4 block quantization, the converter's other scale format.  [P3 Implementation breakdown item 1
 * and Key source snippets: the branch taken without UE8M0 scales (max / 6 stored as E4M3, times a
 * global scale); Review highlights item 2: elements are scaled by the dequantized stored scale]
 * For each row of x and each 16-element block along K, in binary32:
 *   SF   = global_scale * (amax * r6), r6 the binary32 nearest to 1/6, amax = max |x| (exact);
 *   s    = SF as E4M3 (round to nearest even; above 448 -> 448), the stored scale byte;
 *   code = E2M1 of |x| * (global_scale / value(s)) (quotient and product rounded to binary32, then
 *          nearest even, saturating at 6; 0 when value(s) is 0), sign bit 0x8 copied from x;
 *   q[row][j] = code[2j] | code[2j+1] << 4.
 * A value decodes as E2M1(code) * value(s) / global_scale.
 * x_bf16 device bf16 [M, ldx]; K % 16 == 0, K >= 16, ldx >= K, ldx % 8 == 0.
 * global_scale: host binary32, positive and finite (else MXFP4_ERR_SHAPE).
 * q_u8 device uint8 [M, K/2], required.  scale_flat_u8 device uint8 [M, K/16], may be NULL, any
 * alignment.  scale_tiled_u8 device, 16-byte aligned, may be NULL: [ceil(M/128), ceil(K/64), 32, 4, 4],
 * the byte at [mT][kT][oM][iM][iK] the scale of row mT*128 + iM*32 + oM and scale column kT*4 + iK
 * (the tiling of mxfp4_quantize over 16-element scale columns), padding bytes 0.
 * M >= 0 (M == 0 is a no-op). */
int nvfp4_quantize(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, float global_scale, void* q_u8,
                   void* scale_flat_u8, void* scale_tiled_u8, void* stream);

/* Bytes of nvfp4_quantize's tiled scale output: ceil(M/128) * ceil(K/64) * 512; 0 for invalid sizes. */
size_t nvfp4_tiled_scale_bytes(int64_t M, int64_t K);

/* ------------------------------------------------------------------------------------------------
 * MoE weight set.  The standard checkpoint layout [P2 Implementation breakdown item 2]:
 *   w13_q uint8 [E, 2I, H/2]  rows [w1 (gate); w3 (up)]     w13_s uint8 [E, 2I, H/32]  E8M0
 *   w2_q  uint8 [E, H, I/2]                                 w2_s  uint8 [E, H, I/32]   E8M0
 *   b13 [E, 2I], b2 [E, H] optional, fp32 or bf16; converted to bf16 (round to nearest even).
 * Requirements: E >= 1, H % 32 == 0, I % 32 == 0, H >= 32, I >= 32.
 */
typedef struct {
  int32_t E, H, I, has_bias;
} mxfp4_moe_dims;

enum {
  MXFP4_LAYOUT_GFX950 = 0,      /* this library's execution layout (opaque blob with a header) */
  MXFP4_LAYOUT_STD_W31 = 1,     /* checked conversion: standard tensors with w13 as [w3; w1] */
  MXFP4_LAYOUT_SCALE_TILED = 2  /* checked conversion flag: scales in the tiled layout above */
};

/* Output bytes of mxfp4_repack_weights for `layout`; 0 for invalid dims or layout. */
size_t mxfp4_repack_bytes(const mxfp4_moe_dims* d, uint32_t layout);

/* Byte offsets of the six tensors inside a checked-conversion output (layout != GFX950), in the
 * order w13_q, w2_q, w13_s, w2_s, b13, b2: the order in which the pages' conversion returns
 * (w13 weight, w2 weight, w13 scale, w2 scale, w13 bias, w2 bias) [P2 Key source snippets, the
 * conversion branch's return tuple and the test's converted[0..5]]; each offset is 256-byte aligned.
 * Returns a status. */
int mxfp4_repack_offsets(const mxfp4_moe_dims* d, uint32_t layout, size_t offsets_out[6]);

/* Weight conversion at load time.  [P2 Implementation breakdown items 1-3, Key source snippets]
 * Inputs are the standard tensors above (device).  b13/b2 are read only when d->has_bias (then
 * required); bias_is_fp32 selects fp32 (else bf16) input, 4-byte/2-byte aligned.
 * layout = MXFP4_LAYOUT_GFX950: writes the execution blob consumed by moe_mxfp4_forward.
 * layout = MXFP4_LAYOUT_STD_W31 [| MXFP4_LAYOUT_SCALE_TILED], or MXFP4_LAYOUT_SCALE_TILED alone:
 *   writes the six standard tensors at mxfp4_repack_offsets() (w13_q, w2_q, w13_s, w2_s, b13, b2 in
 *   that order): w13_q and w13_s with their row halves exchanged ([w1; w3] -> [w3; w1]) when
 *   STD_W31 is set, w2 unchanged, b13 halves exchanged
 *   likewise, both biases as bf16; with SCALE_TILED both scale tensors are written per expert in the
 *   tiled layout [E, ceil(rows/128), ceil(K/128), 32, 4, 4] instead of flat.  These conversions
 *   exist to check this library against the pages' layouts; the forward pass does not use them.
 * Unknown layout bits -> MXFP4_ERR_LAYOUT.  out_bytes < mxfp4_repack_bytes() -> MXFP4_ERR_WORKSPACE.
 */
int mxfp4_repack_weights(const mxfp4_moe_dims* d, const void* w13_q, const void* w13_s, const void* w2_q,
                         const void* w2_s, const void* b13, const void* b2, int32_t bias_is_fp32, uint32_t layout,
                         void* out, size_t out_bytes, void* stream);

/* Inverse of mxfp4_repack_weights(GFX950): writes the standard tensors back (biases as bf16 bit
 * patterns).  Round trip is the identity on q and scales.  Reads the blob header with a
 * synchronous device-to-host copy and returns MXFP4_ERR_LAYOUT if it does not match *d. */
int mxfp4_unpack_weights(const mxfp4_moe_dims* d, const void* packed, void* w13_q, void* w13_s, void* w2_q,
                         void* w2_s, void* b13_bf16, void* b2_bf16, void* stream);

/* Checks a GFX950 blob's header against *d (synchronous device-to-host copy of 256 bytes).
 * MXFP4_OK or MXFP4_ERR_LAYOUT.  moe_mxfp4_forward itself does not read the header. */
int mxfp4_check_packed(const mxfp4_moe_dims* d, const void* packed, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Routing.  [DEF: router logits -> softmax -> top-k, renormalized over the selected experts]
 *   topk_ids[t] = the top_k largest logits of token t in descending order, equal logits in
 *                 increasing expert index (-0.0 equals +0.0);
 *   topk_w[t,j] = exp(l_j - l_max) / S, S summed over the selected experts (renormalize != 0) or
 *                 over all E experts (renormalize == 0), computed in fp32;
 *   expert_offsets [E+1] = exclusive prefix sum of per-expert pair counts;
 *   sorted_pairs [T*top_k]: pairs p = t*top_k + j grouped by expert, increasing p within an expert.
 * router_logits device fp32 [T, E] contiguous; 1 <= top_k <= min(E, 32); 1 <= E <= 1024; T >= 0.
 * Outputs device int32/fp32 (4-byte alignment suffices).  workspace: device,
 * >= moe_mxfp4_route_workspace_bytes(T, E, top_k), 256-byte aligned.
 */
size_t moe_mxfp4_route_workspace_bytes(int64_t T, int32_t E, int32_t top_k);
int moe_mxfp4_route(const float* router_logits, int64_t T, int32_t E, int32_t top_k, int32_t renormalize,
                    int32_t* topk_ids, float* topk_w, int32_t* expert_offsets, int32_t* sorted_pairs, void* workspace,
                    size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * The MoE layer.  [DEF; P1 Implementation breakdown: the fused-MoE call takes packed 4-bit weights
 * with per-32 group scales and 16-bit activations]
 *   y[t] = sum_j topk_w[t,j] * ( W2_e (silu(h_g) * h_u) + b2_e ),  e = topk_ids[t,j],
 *   h = W13_e x_t + b13_e, h_g = rows [0, I) (w1), h_u = rows [I, 2I) (w3),
 * with W13_e, W2_e the dequantized MXFP4 weights.  Routing as moe_mxfp4_route.
 * packed_gfx950 device blob from mxfp4_repack_weights(GFX950) for the same *d (not re-checked here;
 *   see mxfp4_check_packed).
 * x_bf16  device bf16 [T, ldx], ldx >= H, ldx % 8 == 0.   y_bf16 device bf16 [T, H].
 * router_logits device fp32 [T, E].  topk_ids / topk_w: optional device outputs [T, top_k].
 * workspace device, >= moe_mxfp4_workspace_bytes(d, T, top_k), 256-byte aligned.
 * Size limit: the split activations of the first GEMM (T * H * 2.25 bytes) and of the second (about
 * 2 bytes per padded pair row and I element) must each stay below 4 GiB, else MXFP4_ERR_SHAPE.
 * Arithmetic: activations enter the block-scaled MFMA as three terms with E8M0 scales per 32
 * elements, x = t0 + t1 + t2 (E2M3, E2M3 of the remainder, E2M1 of what is left; each scale from the
 * rule above), weights as E2M1 with their E8M0 scales, fp32 accumulation; the SwiGLU output stays
 * fp32 and is split into three terms the same way; each pair's weighted expert output is kept as
 * integers with a power-of-two scale per 16 columns (at most 2^-14 of the block maximum off), and
 * the combine sums a token's k rows in fp32 in slot order, then rounds to bf16.  The result is
 * deterministic: repeated calls give the same bits.
 */
size_t moe_mxfp4_workspace_bytes(const mxfp4_moe_dims* d, int64_t T, int32_t top_k);

/* Activation formats of moe_mxfp4_forward_act. */
enum {
  MXFP4_ACT_BF16 = 0,  /* bf16 activations, as moe_mxfp4_forward */
  MXFP4_ACT_MXFP8 = 1, /* both GEMM inputs quantized to MXFP8 */
  MXFP4_ACT_MXFP4 = 2  /* both GEMM inputs quantized to MXFP4 */
};
int moe_mxfp4_forward(const mxfp4_moe_dims* d, const void* packed_gfx950, const void* x_bf16, int64_t T, int64_t ldx,
                      const float* router_logits, int32_t top_k, int32_t renormalize, void* y_bf16, int32_t* topk_ids,
                      float* topk_w, void* workspace, size_t workspace_bytes, void* stream);

/* The MoE layer with quantized activations, or bf16 ones (act_format = MXFP4_ACT_BF16 is exactly
 * moe_mxfp4_forward).  [P2 Implementation breakdown item 3: the MXFP8-activation variant of the MXFP4
 * MoE backend; P3 Implementation breakdown item 3: the experts-quant step, MoE activations quantized to
 * MXFP4 with the same E8M0 rule]
 * With MXFP4_ACT_MXFP8 / MXFP4_ACT_MXFP4 the layer input x (each token row, per 32-element block) and
 * the SwiGLU output (fp32, per 32-element block of I) are quantized before the two products and enter
 * the MFMA as one term:
 *   MXFP8: E4M3 elements (round to nearest even) with e = B - 8, B the rounded biased exponent of the
 *          block maximum as in mxfp4_quantize (the pages' rule with E4M3's largest exponent 8 in place
 *          of E2M1's 2), so the maximum maps into [224, 448) and nothing saturates;
 *   MXFP4: exactly the element and scale rule of mxfp4_quantize.
 * Arguments, workspace and errors as moe_mxfp4_forward; an unknown act_format -> MXFP4_ERR_LAYOUT. */
int moe_mxfp4_forward_act(const mxfp4_moe_dims* d, int32_t act_format, const void* packed_gfx950, const void* x_bf16,
                          int64_t T, int64_t ldx, const float* router_logits, int32_t top_k, int32_t renormalize,
                          void* y_bf16, int32_t* topk_ids, float* topk_w, void* workspace, size_t workspace_bytes,
                          void* stream);

/* Same as moe_mxfp4_forward_act, and records events[i] (hipEvent_t passed as void*, created by the caller)
 * on `stream` at stage boundaries: events[0] before the first launch, then after each stage in the
 * order activation split and routing (one launch), pair placement/tile schedule, first GEMM (+SwiGLU),
 * second GEMM (weighted rows), combine (bf16 output) -- 6 events in all.  Only the first n_events are
 * recorded.
 * For per-stage timing (measurement); the computation is identical. */
int moe_mxfp4_forward_profiled(const mxfp4_moe_dims* d, int32_t act_format, const void* packed_gfx950,
                               const void* x_bf16, int64_t T, int64_t ldx, const float* router_logits, int32_t top_k,
                               int32_t renormalize, void* y_bf16, int32_t* topk_ids, float* topk_w, void* workspace,
                               size_t workspace_bytes, void* stream, void* const* events, int32_t n_events);

/* ------------------------------------------------------------------------------------------------
 * Dense MXFP4-weight linear layer (W4A16): y = x W^T + b, W dequantized MXFP4.  [P3 Implementation
 * breakdown item 2: the MXFP4 linear path; DEF: a MoE layer of one expert without routing or
 * activation function]
 * Weights in the standard layout: w_q uint8 [N, K/2] (element 2j in the low nibble), w_s uint8 [N, K/32]
 * E8M0; bias [N] fp32 or bf16 (converted to bf16, round to nearest even), optional.
 * Requirements: N, K multiples of 32, 32 <= N, K <= 2^20.
 * Arithmetic as the second product of moe_mxfp4_forward: x enters as three terms per 32 elements, fp32
 * accumulation, bias added in fp32, one rounding to bf16.
 */
/* Output bytes of mxfp4_linear_pack; 0 for invalid sizes. */
size_t mxfp4_linear_pack_bytes(int64_t N, int64_t K, int32_t has_bias);

/* Weight conversion at load time into this library's layout (opaque, 256-byte header).  w_q, w_s,
 * bias (may be NULL) device; out device, 256-byte aligned, >= mxfp4_linear_pack_bytes (else
 * MXFP4_ERR_WORKSPACE). */
int mxfp4_linear_pack(int64_t N, int64_t K, const void* w_q, const void* w_s, const void* bias, int32_t bias_is_fp32,
                      void* out, size_t out_bytes, void* stream);

/* Workspace bytes of mxfp4_linear_forward for M rows; 0 for invalid sizes. */
size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* y_bf16 device bf16 [M, N] (row-major, contiguous, 16-byte aligned) = x_bf16 (device bf16 [M, ldx],
 * ldx >= K, ldx % 8 == 0) times the packed weights (has_bias as packed).  workspace device, 256-byte
 * aligned, >= mxfp4_linear_workspace_bytes(M, N, K).  M == 0 is a no-op; M * K * 2 bytes of split
 * activations must stay below 4 GiB (else MXFP4_ERR_SHAPE).  Deterministic. */
int mxfp4_linear_forward(const void* packed, int64_t N, int64_t K, int32_t has_bias, const void* x_bf16, int64_t M,
                         int64_t ldx, void* y_bf16, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * The MoE layer without a workspace argument, for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc).  Same arguments,
 * arithmetic and result as moe_mxfp4_forward, whose kernels it shares; the workspace is a device
 * array of MXFP4_NOALLOC_SCRATCH_BYTES inside the library (one per device, held until the process
 * ends), so the call allocates nothing.
 * Limit: moe_mxfp4_workspace_bytes(d, T, top_k) must not exceed MXFP4_NOALLOC_SCRATCH_BYTES, else
 *   MXFP4_ERR_WORKSPACE (nothing is launched).  It covers e.g. E = 128, H = 2048, I = 768, top-8 up
 *   to about 200 tokens.
 * The array of the current device is used (make the stream's device current).  Every call on a
 * device shares that device's array: calls that may overlap on one device (streams without ordering
 * between them) race and must not be issued.  Its address is looked up on the first call on each
 * device (MXFP4_ERR_DEVICE if that fails).
 */
#define MXFP4_NOALLOC_SCRATCH_BYTES (32u << 20)
int moe_mxfp4_forward_noalloc(const mxfp4_moe_dims* d, const void* packed_gfx950, const void* x_bf16, int64_t T,
                              int64_t ldx, const float* router_logits, int32_t top_k, int32_t renormalize,
                              void* y_bf16, int32_t* topk_ids, float* topk_w, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Balance loss of the router, with the per-expert counts it is made of and its gradient.  [DEF]
 *   p_t   = softmax of token t's logits over the E experts;
 *   n_e   = number of pairs (t, j) with topk_ids[t, j] = e over the tokens that count;
 *   loss  = E / (k V^2) * sum_e n_e * sum_t p_{t,e},  V = number of tokens that count
 *           (1 when pairs and probabilities are spread evenly; 0 when V = 0);
 *   dloss/dlogits_{t,e} = p_{t,e} * (d_e - sum_e' d_e' p_{t,e'}),  d_e = E / (k V^2) * (n_e - mean n).
 * The counts are constants of the gradient.  d_e is taken less its mean, which drops out of the bracket.
 * router_logits device fp32 [T, ldl], ldl >= E; E, top_k and T as in moe_mxfp4_route.  topk_ids device
 *   int32 [T, top_k] contiguous; an id outside [0, E) is a dropped pair and is not counted.
 * token_mask device uint8 [T] or NULL: a token counts when its byte is not 0.  The logits and ids of
 *   other tokens are not looked at (any bits), and their gradient is 0.  A logit of -inf has p = 0; a
 *   token whose logits are all -inf has p = 0 throughout and a gradient of 0.
 * loss device fp32 [1], counts device int32 [E], coef device fp32 [E] (d_e, for the backward pass).
 * workspace device, >= moe_balance_workspace_bytes(T, E), 256-byte aligned; nothing in it is kept
 * between calls.  Sums over tokens run in binary32 inside a workgroup and in binary64 across
 * workgroups, in a fixed order: repeated calls give the same bits.  Exponentials are the hardware's: a probability
 * is off by about |logit - maximum| 2^-23 of itself besides its roundings.  T == 0 writes loss 0 and counts 0.
 * moe_balance_backward: grad_loss device fp32 [1]; grad_logits device fp32 [T, E] contiguous, every
 * element written.  Pointers of both need 4-byte alignment only (workspace aside).
 */
size_t moe_balance_workspace_bytes(int64_t T, int32_t E);
int moe_balance_forward(const float* router_logits, int64_t T, int32_t E, int64_t ldl, const int32_t* topk_ids,
                        int32_t top_k, const uint8_t* token_mask, float* loss, int32_t* counts, float* coef,
                        void* workspace, size_t workspace_bytes, void* stream);
int moe_balance_backward(const float* router_logits, int64_t T, int32_t E, int64_t ldl, const uint8_t* token_mask,
                         const float* coef, const float* grad_loss, float* grad_logits, void* stream);

/* Block formats of the entry points below. */
enum {
  MXFP4_FMT_MXFP4 = 0, /* E2M1, an E8M0 scale per 32 elements, as mxfp4_quantize writes it */
  MXFP4_FMT_NVFP4 = 1, /* E2M1, an E4M3 scale per 16 elements and a global scale, as nvfp4_quantize */
  MXFP4_FMT_MXFP8 = 2  /* E4M3, an E8M0 scale per 32 elements, as MXFP4_ACT_MXFP8 (the cache only) */
};

/* ------------------------------------------------------------------------------------------------
 * Matrix-vector products with 4-bit weights: y = x W^T (/ global_scale) + b for one or a few rows of x.
 * [DEF: the W4A16 linear layer, for NVFP4 weights too, in the form that decoding a token needs]
 * Weights in the standard layout, as the quantizers write them (no pack): w_q uint8 [N, K/2] (16-byte
 * aligned), w_s uint8 [N, K/32] E8M0 (MXFP4) or [N, K/16] E4M3 (NVFP4), any alignment.  K is a multiple of the block
 * (32 or 16), 32 <= K <= 2^20, 1 <= N <= 2^20.  global_scale host, positive and finite (NVFP4; MXFP4 ignores it).
 * bias [N] fp32 or bf16 or NULL.  x_bf16 device bf16 [M, ldx], ldx >= K, ldx % 8 == 0, 0 <= M <= 2^20.
 * y device [M, ldy], ldy >= N, bf16 or fp32 (out_is_fp32).
 * Arithmetic: a weight times its scale is exact in bf16 (at most six significant bits) and the products
 * accumulate in fp32, or (NVFP4, up to four rows) x times the codes of a block of 16 accumulates in fp32 and
 * then takes the scale in fp32; the global scale divides and the bias is added in fp32, one rounding to bf16.
 * Products of x and an NVFP4 code below 2^-117 may be lost.
 * Weights of 2^128 and more, or of less than 2^-126, are outside the contract.
 * Deterministic: repeated calls give the same bits (other numbers of rows may sum in another order).  The weights
 * are read once per 16 rows of x: for many rows mxfp4_linear_forward is the faster layer. */
int fp4_matvec(int32_t fmt, const void* w_q, const void* w_s, float global_scale, int64_t N, int64_t K,
               const void* bias, int32_t bias_is_fp32, const void* x_bf16, int64_t M, int64_t ldx, void* y,
               int64_t ldy, int32_t out_is_fp32, void* stream);

/* The same product of every routed pair with its expert's matrix.  [DEF: the experts' products of the MoE
 * layer, on weights in the standard layout]
 *   y[p] = W_e x[p / top_k] / global_scales[e] + b_e   for p in sorted_pairs[offsets[e], offsets[e+1]);
 *   swiglu != 0: the first N/2 rows of W_e are the gate, the others the up projection, and
 *   y[p] = silu(gate) * up has N/2 columns (rows [w1; w3], as in the MoE layer; the hardware's exponential: silu is off
 *   by about |gate| 2^-24 of itself, and 0 for gates below -88.7, where it is less than 2^-121).
 * w_q [E, N, K/2], w_s [E, N, K/B], bias [E, N] or NULL, global_scales device fp32 [E] (NVFP4).
 * expert_offsets device int32 [E + 1] and sorted_pairs device int32 [n_pairs]: moe_mxfp4_route's outputs
 *   (offsets outside [0, n_pairs] are clamped, pairs outside it passed over; a pair that is not
 *   listed keeps its row of y).  x has n_pairs / top_k rows: top_k as routed when the pairs of a token
 *   share its row, 1 when every pair has a row of its own (the second product).
 * y device [n_pairs, N or N/2] contiguous.  1 <= E, top_k <= 1024. */
int fp4_expert_matvec(int32_t fmt, const void* w_q, const void* w_s, const float* global_scales, int32_t E, int64_t N,
                      int64_t K, const void* bias, int32_t bias_is_fp32, const void* x_bf16, int64_t ldx,
                      int32_t top_k, const int32_t* expert_offsets, const int32_t* sorted_pairs, int64_t n_pairs,
                      int32_t swiglu, void* y, int32_t out_is_fp32, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Paged cache in a block format: rows are quantized as they are written and read back as bf16.
 * [DEF: the quantizers' element and scale rules, applied to the cached rows of an attention layer]
 * A cache holds num_pages pages of page_size tokens; a token has `heads` vectors of k_dim elements, and
 * of v_dim elements in a second plane (v_dim = 0: one plane).  Caller-owned memory, per plane:
 *   q uint8 [num_pages, page_size, heads, dim/2] (MXFP8: dim), 8-byte aligned;
 *   s uint8 [num_pages, page_size, heads, dim/B], B the format's block (32; NVFP4: 16), dim % B == 0.
 * Rows are ragged: rows [cu_rows[b], cu_rows[b + 1]) belong to sequence b and hold its positions
 * start[b], start[b] + 1, ... (start NULL: from 0).  Position i lives in page page_table[b][i / page_size],
 * slot i % page_size.  cu_rows device int32 [n_seqs + 1], non-decreasing; start device int32 [n_seqs] or
 * NULL; page_table device int32 [n_seqs, ld_table], max_pages <= ld_table columns used.
 * `rows` is the number of rows that k and v hold; rows before cu_rows[0] or from cu_rows[n_seqs] on are not
 * read by the write and are left as they were by the read.  A position below 0, past max_pages or in a
 * page outside [0, num_pages) is not written, and is read as zeros.
 * The write quantizes each block of each row: MXFP4 and NVFP4 bit for bit as mxfp4_quantize and
 * nvfp4_quantize, MXFP8 as MXFP4_ACT_MXFP8 quantizes activations.  Two rows of one call must not share a
 * slot: what such a slot then holds is not specified.  The read returns code * scale, rounded once to bf16
 * (NVFP4: the scale divided by the plane's global scale and multiplied by the code in binary32, then rounded; where
 * the quotient alone would overflow, codes whose value does not still have it).
 * k / v device bf16, element (row, head, i) at row * ldt + head * ldh + i; ldt, ldh multiples of 8, ldh >= dim,
 * ldt >= dim; the vectors that the read writes must not overlap.  heads * dim <= 2^20.  Neither call uses a
 * workspace.  The cache's pointers may be NULL when num_pages is 0, the table when max_pages is 0. */
typedef struct {
  int32_t fmt, heads, k_dim, v_dim, page_size;
  int64_t num_pages;
  float k_global_scale, v_global_scale; /* NVFP4: host, positive and finite */
} mxfp4_cache_dims;

/* Bytes of the four cache tensors, in the order k_q, k_s, v_q, v_s. */
int mxfp4_cache_bytes(const mxfp4_cache_dims* d, size_t bytes_out[4]);
int mxfp4_cache_write(const mxfp4_cache_dims* d, const void* k_bf16, int64_t k_ldt, int64_t k_ldh, const void* v_bf16,
                      int64_t v_ldt, int64_t v_ldh, int64_t rows, const int32_t* cu_rows, const int32_t* start,
                      const int32_t* page_table, int64_t ld_table, int32_t n_seqs, int32_t max_pages, void* k_q,
                      void* k_s, void* v_q, void* v_s, void* stream);
int mxfp4_cache_read(const mxfp4_cache_dims* d, const void* k_q, const void* k_s, const void* v_q, const void* v_s,
                     int64_t rows, const int32_t* cu_rows, const int32_t* start, const int32_t* page_table,
                     int64_t ld_table, int32_t n_seqs, int32_t max_pages, void* k_bf16, int64_t k_ldt, int64_t k_ldh,
                     void* v_bf16, int64_t v_ldt, int64_t v_ldh, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Attention over the paged cache, for rows whose keys and values the cache holds already: one new token, a
 * chunk of a prompt, or a tree of drafted tokens.  [DEF]
 *   out[t, h] = sum_j p_j V[j, g],  p = softmax over the positions j that row t sees of scale * q[t, h] . K[j, g],
 *   g = h / (q_heads / heads), K and V the cache's values (code * scale, NVFP4: / global scale; not rounded to bf16).
 * Rows are ragged as for mxfp4_cache_write, and given the same cu_rows, start and page_table: row t of sequence b is
 * its draft i = t - cu_rows[b], at position start[b] + i.  It sees the positions below start[b], and of its sequence's
 * n drafts those j with tree_mask[t * ld_mask + j] != 0 (j >= mask_cols: none), or, tree_mask NULL, those with j <= i.
 * A position without a page (mxfp4_cache_write) is not seen; what lies there or in places that the mask hides is not
 * looked at.  A row that sees nothing gets zeros.  Rows outside every sequence are not read and keep their output.
 * q device bf16, element (row, head, i) at row * q_ldt + head * q_ldh + i, strides multiples of 8, 16-byte aligned,
 *   q_heads a multiple of heads, q_heads <= 2^16.  k_dim and v_dim at most 256, v_dim > 0.  scale finite, log2(e) times
 *   it too (NVFP4: divided by the keys' global scale).
 *   max_pages * page_size <= 2^31 - 256, rows * q_heads / heads < 2^31 - 256.
 * out device bf16 or fp32 (out_is_fp32), element (row, head, i) at row * out_ldt + head * out_ldh + i, strides multiples
 *   of 8, 16-byte aligned; its vectors must not overlap each other or q.
 * tree_mask device uint8, row t of mask_cols entries at t * ld_mask, or NULL.
 * Arithmetic: values are exact in bf16 (code * scale), products accumulate in fp32, the maximum and the sum of the
 * softmax are fp32, the weights p are rounded to bf16 before the second product (2^-8 of each; for results in fp32, and
 * where a sequence has up to 16 rows a key head on average, to two terms in bf16, 2^-16 of each); parts of a long context are joined in fp32 in a fixed order, and the result is rounded
 * once: repeated calls give the same bits.  Exponentials are the hardware's.  A NaN in a query or in a key that it sees
 * makes the result NaN, one in a value that it sees at least the element it is in.  Outside the contract are keys of 2^128
 * and more, scores past fp32's range, and values of 2^88 and more (NVFP4: before the division by the global scale, so
 * none): their sums over up to 2^31 positions, with weights below 2^9, are formed before they are divided.
 * workspace device, 256-byte aligned, >= mxfp4_cache_attend_workspace_bytes (0: invalid sizes); nothing in it is kept
 * between calls. */
size_t mxfp4_cache_attend_workspace_bytes(const mxfp4_cache_dims* d, int32_t q_heads, int64_t rows, int32_t n_seqs);
int mxfp4_cache_attend(const mxfp4_cache_dims* d, const void* k_q, const void* k_s, const void* v_q, const void* v_s,
                       const void* q_bf16, int64_t q_ldt, int64_t q_ldh, int32_t q_heads, int64_t rows,
                       const int32_t* cu_rows, const int32_t* start, const int32_t* page_table, int64_t ld_table,
                       int32_t n_seqs, int32_t max_pages, const uint8_t* tree_mask, int64_t ld_mask, int32_t mask_cols,
                       float scale, void* out, int64_t out_ldt, int64_t out_ldh, int32_t out_is_fp32, void* workspace,
                       size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Compaction: the accepted drafts of each sequence are moved together.  [DEF]
 * path device int32 [n_seqs, ld_path], path_cols columns used: path[b] = the accepted drafts of sequence b in increasing
 * order, ended by a negative entry, by one that does not increase, or by the last column.  Position start[b] + i takes the
 * codes and scales of position start[b] + path[b][i], as they were before the call.  A position without a page is not
 * written, and one whose source has no page keeps what it holds.  lengths device int32 [n_seqs] gets start[b] + the
 * number of accepted drafts (may be NULL; must not be start).  Sequences must not share the slots that are moved. */
int mxfp4_cache_compact(const mxfp4_cache_dims* d, const int32_t* start, const int32_t* path, int64_t ld_path,
                        int32_t path_cols, const int32_t* page_table, int64_t ld_table, int32_t n_seqs,
                        int32_t max_pages, int32_t* lengths, void* k_q, void* k_s, void* v_q, void* v_s, void* stream);

/* The first rows[i] tokens (rows NULL: all) of page src[i] are copied to page dst[i], i < n.  A pair with a page outside
 * [0, num_pages) is passed over.  No page may be the destination of two pairs, or a source and another pair's
 * destination. */
int mxfp4_cache_copy_pages(const mxfp4_cache_dims* d, const int32_t* src, const int32_t* dst, const int32_t* rows,
                           int32_t n, void* k_q, void* k_s, void* v_q, void* v_s, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Page pool: which pages of a cache are in use, on the device.  [DEF]
 * refs device int32 [num_pages]: how many rows of the page tables hold the page; a page with refs <= 0 is free.  The pages
 * that row b of a table holds are its leading entries in [0, num_pages); the other entries are -1.
 * Free pages are handed out in increasing order, to rows (pairs) in increasing order.
 *
 * mxfp4_pool_resize: row b then holds the ceil(lengths[b] / page_size) pages of lengths[b] tokens (at most max_pages;
 * lengths[b] < 0: the row is left alone).  Pages past them are given back, missing ones are taken.  Where lengths[b] ends
 * inside a page that the row held already and that is shared (refs > 1 after what this call gives back), the row gets a
 * page of its own in its place.
 *
 * mxfp4_pool_fork: for each pair i < n, row dst[i] gives back its pages and gets the first lengths[i] tokens of row
 * src[i]: whole pages are shared, the page that lengths[i] ends in, where row src[i] holds it, becomes a page of its own.
 * A pair is passed over when a row is outside the table, lengths[i] < 0, dst[i] is a source of any pair, or an earlier
 * pair has the same dst.
 *
 * copies device int32 [3, n_rows] (fork: [3, n]): the source page, new page and tokens of each row (pair) whose page has
 * to be copied, as mxfp4_cache_copy_pages takes them; -1, -1, 0 where there is none.
 * missing device int32 [1]: pages that were wanted when no page was free any more; their entries are -1.  So is that of a
 * shared page that was to be replaced: the row lets go of it, and of its tokens in it, and the other rows keep them.  Where
 * every row that held such a page let go of it or got a copy, the last of those that could not be given one keeps it as its
 * own, and none is missing there.
 * workspace device, 256-byte aligned, >= mxfp4_pool_workspace_bytes(num_pages, n_rows or n, max_pages).
 * num_pages < 2^31, page_size >= 1, n_rows <= 2^24, n <= 2^16, n_rows * max_pages and n * max_pages < 2^31. */
size_t mxfp4_pool_workspace_bytes(int64_t num_pages, int32_t n, int32_t max_pages);
int mxfp4_pool_resize(int64_t num_pages, int32_t page_size, int32_t* refs, int32_t* page_table, int64_t ld_table,
                      int32_t n_rows, int32_t max_pages, const int32_t* lengths, int32_t* copies, int32_t* missing,
                      void* workspace, size_t workspace_bytes, void* stream);
int mxfp4_pool_fork(int64_t num_pages, int32_t page_size, int32_t* refs, int32_t* page_table, int64_t ld_table,
                    int32_t n_rows, int32_t max_pages, const int32_t* src, const int32_t* dst, const int32_t* lengths,
                    int32_t n, int32_t* copies, int32_t* missing, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Rotary positions, on queries and keys at once.  [DEF]
 * Elements [offset, offset + rot_dim) of each head_dim vector are pairs (a, b), pair i turned by the angle
 * 2 pi positions[row] turns[i]:  a' = m (a cos - b sin), b' = m (b cos + a sin), m = magnitude; pair i is elements
 * (i, i + rot_dim / 2), or (2i, 2i + 1) with interleaved.  The other elements are copied (not where input and output are
 * the same memory).  inverse != 0 turns by the negative angle: with the same magnitude, the gradient.
 * turns device double [rot_dim / 2]: turns per position.  positions device int32 [rows].
 * q, k device bf16 or fp32 (is_fp32), element (row, head, i) at row * ldt + head * ldh + i; k NULL: queries only.  Output
 * vectors must not overlap each other, nor an input but that of the same place.  rot_dim even, 2 <= rot_dim <= 2048,
 * offset >= 0, offset + rot_dim <= head_dim <= 2^16, heads * head_dim <= 2^20.  Element alignment suffices.
 * Arithmetic: the angle in binary64, less its whole turns; sine, cosine, magnitude and the sums in binary32; one rounding
 * to the type. */
int mxfp4_rotary(const double* turns, const int32_t* positions, int64_t rows, int32_t head_dim, int32_t rot_dim,
                 int32_t offset, int32_t interleaved, float magnitude, int32_t inverse, int32_t is_fp32, const void* q,
                 int64_t q_ldt, int64_t q_ldh, int32_t q_heads, void* q_out, int64_t q_out_ldt, int64_t q_out_ldh,
                 const void* k, int64_t k_ldt, int64_t k_ldh, int32_t k_heads, void* k_out, int64_t k_out_ldt,
                 int64_t k_out_ldh, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4MOE_H */
