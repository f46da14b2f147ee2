/* ffn_ops.h -- C ABI of the operators around the sparse FFN layer of sparse_ffn.h, in the same
 * library (libsparse_ffn.so, MI355X / gfx950): the root-mean-square norm and the layer norm before
 * the layer with the residual stream's sum (also with an 8-bit output for serving), their gradients,
 * products with 4-bit weights for batches of few tokens and, with the tokens in 4 bits too, for
 * prompts, the norm of all gradients and clipping by it, and the AdamW step over the layer's tensors.
 * All declarations here are interface of the library.
 *
 * Conventions are those of sparse_ffn.h: device pointers unless marked (host), row-major
 * layouts, status codes only, arguments checked on the host before any launch, asynchronous on
 * `stream`, no device memory allocated, nothing kept between calls.  Besides:
 *   - A row stride counts elements from one row to the next (>= the row's length); the elements
 *     of a row are contiguous.  Pointers need only their element's alignment.
 *   - Zero rows (or elements, or tensors) are valid and launch nothing.
 *   - No output may overlap an input or another output (SFFN_ERR_INVALID_ARGUMENT), except where
 *     a call says that it updates in place, and a norm's h, and its y in dtype, which may be x
 *     or the residual itself (same address and stride).
 *   - Non-finite values follow the formulas: they reach the outputs that depend on them.
 *   - Results do not depend on timing: no call adds with atomics.
 *   - Kernel names for sffn_profile_read: rms_norm, rms_norm_fp8, rms_norm_grad,
 *     rms_norm_grad_sum, layer_norm, layer_norm_fp8, layer_norm_grad, layer_norm_grad_sum,
 *     mx4_quantize, mx4_tile, mx4_linear, mx4_tokens, mx4_matmul, grad_norm, grad_norm_sum, grad_scale, adamw. */
#ifndef FFN_OPS_H_
#define FFN_OPS_H_

#include "sparse_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type code beside SFFN_F32 and SFFN_BF16: 8-bit e4m3 (OCP: largest value 448, no
 * infinities), where a call accepts it. */
#define SFFN_E4M3 2

/* Largest row length of the norm calls (SFFN_ERR_UNSUPPORTED beyond it): a row is held in the
 * registers of at most 16 waves. */
#define SFFN_NORM_MAX_D 32768

/* Weights that share a scale in the 4-bit format, and values that share a scale in an 8-bit
 * optimizer state. */
#define SFFN_MX4_GROUP 32
#define SFFN_ADAMW_BLOCK 256

/* Root-mean-square norm of the residual stream, for `rows` tokens of length d:
 *   h = x + residual  (h = x without one),  rstd = 1 / sqrt(mean(h^2) + eps),
 *   y = h * rstd * gain
 * with h, its squares' sum and the products in fp32 (y is computed from the unrounded h).
 * x, residual, h [rows, d] and y [rows, d] are dtype (SFFN_F32 or SFFN_BF16); gain [d] is dtype
 * or SFFN_F32 (gain_dtype).  residual may be NULL, then h must be NULL too; otherwise h may be
 * NULL if the sum is not wanted.  rstd [rows] fp32 may be NULL.  h and y have stride d. */
sffn_status_t sffn_rms_norm(int32_t dtype, int32_t gain_dtype, const void *x, int64_t x_stride,
                            const void *residual, int64_t residual_stride, const void *gain,
                            float eps, int64_t rows, int32_t d, void *y, float *rstd, void *h,
                            void *stream);

/* The same norm with its output in 8 bits and one scale a row, the form sffn_mx4_linear takes:
 *   scale = max(max_i |y_i| / 448, 2^-126),  q = e4m3(y / scale)
 * (the quotient rounded to fp32, then to nearest-even).  q [rows, d] bytes, scale [rows] fp32.
 * A row of zeros gives zeros; a NaN or an infinity in a row gives a scale that is not finite. */
sffn_status_t sffn_rms_norm_fp8(int32_t dtype, int32_t gain_dtype, const void *x,
                                int64_t x_stride, const void *residual, int64_t residual_stride,
                                const void *gain, float eps, int64_t rows, int32_t d, void *q,
                                float *scale, void *h, void *stream);

/* (host only) Bytes of scratch sffn_rms_norm_backward needs for these sizes with dgain: 0 for few
 * rows, which are summed without it. */
sffn_status_t sffn_rms_norm_backward_workspace(int64_t rows, int32_t d, size_t *bytes);

/* Gradient of sffn_rms_norm.  With xh = h * rstd and t = dy * gain:
 *   dx = rstd * (t - xh * mean(t * xh)) + dres,   dgain = sum over rows of dy * xh
 * h and rstd are the forward's (h = x where there was no residual); dres, the gradient that
 * reaches h past the norm, may be NULL.  dx [rows, d] (stride d, dtype) is the gradient of both
 * x and the residual; dgain [d] is fp32 and may be NULL; with zero rows it is cleared.  dx may be dres
 * itself.  Sums are in fp32 in an order that depends on the sizes alone.  workspace: as many
 * bytes as sffn_rms_norm_backward_workspace says, 16-byte aligned (NULL for 0). */
sffn_status_t sffn_rms_norm_backward(int32_t dtype, int32_t gain_dtype, const void *dy,
                                     int64_t dy_stride, const void *h, int64_t h_stride,
                                     const void *gain, const float *rstd, const void *dres,
                                     int64_t dres_stride, int64_t rows, int32_t d, void *dx,
                                     float *dgain, void *workspace, size_t workspace_bytes,
                                     void *stream);

/* Layer norm of the residual stream, for `rows` tokens of length d:
 *   h = x + residual  (h = x without one),  mean = mean(h),
 *   rstd = 1 / sqrt(mean((h - mean)^2) + eps),  y = (h - mean) * rstd * gain + bias
 * in fp32, from the unrounded h; the deviations are taken from the mean of the row's own values (no
 * difference of two large sums), and their sum corrects that mean.  A row whose sum or whose deviations'
 * squares pass fp32's range has an infinite mean or variance, and what follows from it.  Types, strides and what may be
 * NULL are as in sffn_rms_norm; gain and bias [d] have gain_dtype, bias may be NULL (0).
 * mean and rstd [rows] fp32 may each be NULL. */
sffn_status_t sffn_layer_norm(int32_t dtype, int32_t gain_dtype, const void *x, int64_t x_stride,
                              const void *residual, int64_t residual_stride, const void *gain,
                              const void *bias, float eps, int64_t rows, int32_t d, void *y,
                              float *mean, float *rstd, void *h, void *stream);

/* The same norm with its output in 8 bits and one scale a row, as sffn_rms_norm_fp8 gives it. */
sffn_status_t sffn_layer_norm_fp8(int32_t dtype, int32_t gain_dtype, const void *x,
                                  int64_t x_stride, const void *residual, int64_t residual_stride,
                                  const void *gain, const void *bias, float eps, int64_t rows,
                                  int32_t d, void *q, float *scale, void *h, void *stream);

/* (host only) Bytes of scratch sffn_layer_norm_backward needs for these sizes with dgain or dbias: 0
 * for few rows, which are summed without it. */
sffn_status_t sffn_layer_norm_backward_workspace(int64_t rows, int32_t d, size_t *bytes);

/* Gradient of sffn_layer_norm.  With xh = (h - mean) * rstd and t = dy * gain:
 *   dx = rstd * (t - mean(t) - xh * mean(t * xh)) + dres,
 *   dgain = sum over rows of dy * xh,   dbias = sum over rows of dy
 * h, mean and rstd are the forward's, as stored: in a row whose mean is many times its spread, mean's
 * rounding to fp32 puts xh off by up to 2^-24 |mean| rstd.  dgain and dbias [d] are fp32 and may each be NULL; with zero
 * rows they are cleared.  All else is as in sffn_rms_norm_backward. */
sffn_status_t sffn_layer_norm_backward(int32_t dtype, int32_t gain_dtype, const void *dy,
                                       int64_t dy_stride, const void *h, int64_t h_stride,
                                       const void *gain, const float *mean, const float *rstd,
                                       const void *dres, int64_t dres_stride, int64_t rows,
                                       int32_t d, void *dx, float *dgain, float *dbias,
                                       void *workspace, size_t workspace_bytes, void *stream);

/* 4-bit weights.  Value of weight (n, k): e2m1(code) * 2^(s - 127), s = scales[n, k / 32] (255
 * is NaN), e2m1 codes 0..7 = 0, 0.5, 1, 1.5, 2, 3, 4, 6, bit 3 the sign (the OCP microscaling
 * format MXFP4).  codes [N, 16 * ceil(K / 32)] bytes, the even k in the low half;
 * scales [N, ceil(K / 32)] bytes.  Codes of k >= K are ignored.
 *
 * Quantise a dense matrix W [N, K] (SFFN_F32 or SFFN_BF16) into codes and scales: per group of
 * 32, exponent floor(log2(max |w|)) - 2 (at least -127), values to nearest-even, at most 6.  A
 * group with a value that is not finite gets scale 255. */
sffn_status_t sffn_mx4_quantize(int32_t dtype, const void *W, int64_t w_stride, int32_t N,
                                int32_t K, uint8_t *codes, uint8_t *scales, void *stream);

/* (host only) Bytes of the layout sffn_mx4_linear reads (written by sffn_mx4_tile). */
sffn_status_t sffn_mx4_bytes(int32_t N, int32_t K, size_t *bytes);

/* Lay codes and scales out for sffn_mx4_linear, once for a weight: `tiled` (sffn_mx4_bytes
 * bytes, 16-byte aligned) holds for every 16 rows and 128 columns the 1 KB that one wave loads
 * at once, then the scales in the same order. */
sffn_status_t sffn_mx4_tile(const uint8_t *codes, const uint8_t *scales, int32_t N, int32_t K,
                            void *tiled, void *stream);

/* y = act(x W^T * x_scale + bias) for T tokens, W [N, K] in the layout of sffn_mx4_tile.
 * x [T, K] is SFFN_BF16, SFFN_F32 or SFFN_E4M3; x_scale [T] fp32 multiplies a token's results
 * (required for SFFN_E4M3, otherwise it may be NULL).  bias [N] fp32 may be NULL.  act is
 * max(., 0) if relu is nonzero (NaN stays).  y [T, N] (stride N) is SFFN_F32 or SFFN_BF16.
 * Products are exact and sums in fp32, within fp32's range: a weight of 2^128 or more (scales 253
 * and 254 with a large code, which sffn_mx4_quantize never writes) makes its row's results not
 * finite, also where a small token value would bring the product back.
 * N up to 2^26, K up to 2^30, N K below 2^36.  Every T up to 2^20 is accepted; the kernel is made
 * for T <= 64.  Up to 16 tokens read the weights once, more read them again for every 32 tokens, or
 * with SFFN_BF16 and SFFN_E4M3 tokens for every 64 where that is estimated to be quicker (33 to
 * 64 tokens: once). */
sffn_status_t sffn_mx4_linear(const void *tiled, int32_t N, int32_t K, int32_t x_dtype,
                              const void *x, int64_t x_stride, const float *x_scale, int32_t T,
                              const float *bias, int32_t relu, int32_t y_dtype, void *y,
                              void *stream);

/* (host only) Bytes of the layout of T tokens of K columns that sffn_mx4_matmul reads. */
sffn_status_t sffn_mx4_tokens_bytes(int32_t T, int32_t K, size_t *bytes);

/* Round tokens x [T, K] (SFFN_F32 or SFFN_BF16) to 4 bits as sffn_mx4_quantize rounds weights, into
 * the layout that sffn_mx4_matmul reads: `tokens` (sffn_mx4_tokens_bytes bytes, 16-byte aligned) holds
 * for every 16 tokens and 128 columns 1 KB of codes, then the scales.  Tokens past the last one and
 * columns past K are zeros. */
sffn_status_t sffn_mx4_tokens(int32_t dtype, const void *x, int64_t x_stride, int32_t T, int32_t K,
                              void *tokens, void *stream);

/* y = act(x W^T + bias) for T tokens in 4 bits (the layout of sffn_mx4_tokens for this T and K) and
 * W [N, K] in the layout of sffn_mx4_tile.  bias [N] fp32 may be NULL; act, y and N are as in
 * sffn_mx4_linear; T up to 2^20, K up to 2^28, T K below 2^36, T N up to 2^37.  Products are
 * exact; the sum of 128 columns, and each addition of such sums in fp32, is off by at most two fp32
 * roundings of the absolute values summed, within fp32's range.  Their order depends on T, N, K and
 * y's type alone.  A token group or a weight group with the scale 255 (NaN) makes the results that it
 * reaches NaN. */
sffn_status_t sffn_mx4_matmul(const void *tiled, int32_t N, int32_t K, const void *tokens,
                              int32_t T, const float *bias, int32_t relu, int32_t y_dtype, void *y,
                              void *stream);

/* (host only) Bytes of scratch sffn_mx4_quantized needs for T tokens of K columns: 0 for up to 16. */
sffn_status_t sffn_mx4_quantized_workspace(int32_t T, int32_t K, size_t *bytes);

/* sffn_mx4_tokens and sffn_mx4_matmul in one call, with the same results: x [T, K] (SFFN_F32 or
 * SFFN_BF16) is rounded into the workspace, or up to 16 tokens in the product itself.  workspace: as
 * many bytes as sffn_mx4_quantized_workspace says, 16-byte aligned (NULL for 0). */
sffn_status_t sffn_mx4_quantized(const void *tiled, int32_t N, int32_t K, int32_t x_dtype,
                                 const void *x, int64_t x_stride, int32_t T, const float *bias,
                                 int32_t relu, int32_t y_dtype, void *y, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* One gradient: n elements of its own type (SFFN_F32 or SFFN_BF16). */
typedef struct {
  const void *grad;
  void *out;       /* sffn_grad_clip: where it goes, grad itself to clip in place */
  int64_t n;
  int32_t dtype;
  int32_t zero;    /* 0 */
} sffn_grad_t;

/* (host only) Bytes of scratch sffn_grad_norm and sffn_grad_clip need for these gradients (host
 * array, of which only n is read): at most 8 * (1024 + n_grads). */
sffn_status_t sffn_grad_norm_workspace(const sffn_grad_t *grads, int32_t n_grads, size_t *bytes);

/* Norm of all gradients together (host array, read before the call returns; out is not read):
 *   norm[0] = sqrt(sum of the squares of all elements),
 *   factor[0] = 1 if norm <= max_norm, else max_norm / norm
 * with the squares, exact in 64 bits, summed in 64 bits, so that no square overflows or vanishes;
 * norm is rounded to fp32 once, and so is the quotient, by that norm.  factor is what
 * sffn_adamw_step takes as grad_scale; it may be NULL.  An infinity among the gradients, or a norm
 * beyond fp32's range, gives the norm infinity and, with a finite max_norm, the factor 0; a NaN gives
 * NaN for both.  No gradients, or none with elements, have the norm 0.  The order of the sums depends on the sizes alone.  workspace: as many bytes as
 * sffn_grad_norm_workspace says, 16-byte aligned. */
sffn_status_t sffn_grad_norm(const sffn_grad_t *grads, int32_t n_grads, double max_norm,
                             float *norm, float *factor, void *workspace, size_t workspace_bytes,
                             void *stream);

/* The same, and then out = grad * factor (in fp32, then rounded to the gradient's type) for every gradient.
 * Where out is grad itself and factor is 1, nothing is written.  factor is required.  An out may be
 * its own gradient, and may overlap nothing else of the call. */
sffn_status_t sffn_grad_clip(const sffn_grad_t *grads, int32_t n_grads, double max_norm,
                             float *norm, float *factor, void *workspace, size_t workspace_bytes,
                             void *stream);

/* One tensor of an AdamW step (device pointers, n elements each). */
typedef struct {
  void *param;       /* updated; written only (rounded from master) where master is given */
  const void *grad;
  float *master;     /* fp32 master, updated; NULL: the step is taken on param itself */
  void *m;           /* first moment: fp32, or e4m3 codes */
  void *v;           /* second moment in fp32; with 8-bit states its root, in e4m3 codes */
  float *m_scale;    /* 8-bit states: [ceil(n / 256)] scales (NULL otherwise) */
  float *v_scale;
  int64_t n;
} sffn_adamw_tensor_t;

typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step; /* 1 for the first step */
} sffn_adamw_hyper_t;

/* One AdamW step over n_tensors tensors (host array, read before the call returns), in place:
 *   g = grad * grad_scale[0]  (grad_scale: one fp32 on the device, or NULL for 1)
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = p - lr (weight_decay p + (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps))
 * param is SFFN_F32 or SFFN_BF16, with an fp32 master only where it is SFFN_BF16; grad is
 * SFFN_F32 or SFFN_BF16.  state_bits 32 holds m and v in fp32.  state_bits 8 holds m and
 * r = sqrt(v) as e4m3 codes with one scale per 256 consecutive elements,
 * scale = max(absmax / 448, 2^-126), each code the e4m3 value nearest to the quotient by it; a
 * positive r keeps at least the smallest positive code, since it divides.  The step itself uses
 * the unrounded m and r.  The arrays of a tensor are checked for overlap; different tensors are
 * the caller's to keep apart. */
sffn_status_t sffn_adamw_step(const sffn_adamw_tensor_t *tensors, int32_t n_tensors,
                              int32_t param_dtype, int32_t grad_dtype, int32_t state_bits,
                              const sffn_adamw_hyper_t *hyper, const float *grad_scale,
                              void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FFN_OPS_H_ */
