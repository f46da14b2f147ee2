/* ffn_ops.h -- C ABI of the operators around the sparse FFN layer of sparse_ffn.h, in the same
 * library (libsparse_ffn.so, MI355X / gfx950): the root-mean-square norm before the layer with
 * the residual stream's sum (also with an 8-bit output for serving), its gradient, products
 * with 4-bit weights for batches of few tokens, and the AdamW step over the layer's tensors.
 * All declarations here are interface of the library.
 *
 * Conventions are those of sparse_ffn.h: device pointers unless marked (host), row-major
 * layouts, status codes only, arguments checked on the host before any launch, asynchronous on
 * `stream`, no device memory allocated, nothing kept between calls.  Besides:
 *   - A row stride counts elements from one row to the next (>= the row's length); the elements
 *     of a row are contiguous.  Pointers need only their element's alignment.
 *   - Zero rows (or elements, or tensors) are valid and launch nothing.
 *   - No output may overlap an input or another output (SFFN_ERR_INVALID_ARGUMENT), except where
 *     a call says that it updates in place, and the norm's h, and its y in dtype, which may be x
 *     or the residual itself (same address and stride).
 *   - Non-finite values follow the formulas: they reach the outputs that depend on them.
 *   - Results do not depend on timing: no call adds with atomics.
 *   - Kernel names for sffn_profile_read: rms_norm, rms_norm_fp8, rms_norm_grad,
 *     rms_norm_grad_sum, mx4_quantize, mx4_tile, mx4_linear, adamw. */
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
