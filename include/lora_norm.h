/*
 * lora_norm.h -- root-mean-square norm with the residual's addition, dropout of
 * the branch, and an output in 8 bits for the fp8 layers.
 *
 * ch05 "Acceleration principles: Triton kernels and fused LoRA", §5.4 (fused
 * RMSNorm: one pass over the hidden state).  Per row of `dim` elements:
 *
 *     h = drop(x) + residual           (rounded to the dtype: what is kept)
 *     r = (mean(h^2) + eps)^(-1/2)
 *     y = h r w
 *     codes = e4m3(y / scale), scale = 2^e, e the smallest integer >= -126
 *             with max|y| <= 448 2^e  (y before it is rounded to the dtype)
 *
 * with the rows, scales and saturation of lora_fp8.h (lora_fp8_fwd_rows takes
 * them), and drop as in lora_dropout.h.  Backward, from dy and the gradient dh
 * that reaches h from the stream itself:
 *
 *     g = dy w,  dresidual = r (g - h r mean(g h r)) + dh,  dx = drop(dresidual)
 *     dw = sum over rows of dy h r
 *
 * Sums are fp32 (rows whose squares leave its range, or lose bits below it where
 * eps is as small, are summed again scaled; r itself is an fp32 number: infinite
 * where h is 0 or its root mean square is below 2^-128 and eps is 0); dw adds
 * blocks of rows in a fixed order: the same call gives the same bits.  Errors,
 * streams and the timing hook are those of lora_linear.h.  Nothing is allocated;
 * no host synchronisation.
 */
#ifndef LORA_NORM_H
#define LORA_NORM_H

#include "lora_dropout.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Row (o, i), o < outer, i < inner, begins at o * stride[0] + i * stride[1]
 * elements; the elements of a row are contiguous. */
typedef struct {
    int64_t outer, inner; /* >= 0; outer * inner < 2^31                       */
    int32_t dim;          /* 1 .. 32768                                       */
    int32_t weight_fp32;  /* 1: w and dw are fp32, 0: of the dtype            */
    float eps;            /* >= 0                                             */
    int64_t x[2], residual[2], h[2], y[2];
    int64_t dy[2], dh[2], dx[2], dresidual[2];
} lora_norm_t;

/*
 * Forward.  One launch.
 *   x, w       in.  residual: in, or NULL.  dropout: or NULL.
 *   h          out, or NULL (nothing is kept).  Without residual and dropout
 *              h is x: give NULL.
 *   y          out, or NULL where only the codes are wanted.
 *   rstd       out, r of each row (fp32, contiguous), or NULL.
 *   codes      out, [outer * inner][dim] bytes, and scale, a float a row, or
 *              both NULL.
 * An output may be an input of the same rows (same address and strides: y = x,
 * h = residual); otherwise none may overlap another tensor.
 */
lora_status_t lora_norm_fwd(const lora_norm_t *shape, const void *x, const void *residual,
                            const void *w, const lora_dropout_t *dropout, lora_dtype_t dtype,
                            void *h, void *y, float *rstd, void *codes, float *scale,
                            void *stream);

/* Bytes of device workspace lora_norm_bwd needs for dw (0 without it). */
size_t lora_norm_workspace_bytes(const lora_norm_t *shape, int with_dw);

/*
 * Backward.  One launch, two with dw.
 *   dy, h, w, rstd  in (h: the forward's, or its x where it had none to write).
 *   dh         in, or NULL (0).
 *   dx         out; with dropout, the gradient of the dropped-out branch.
 *   dresidual  out, or NULL.  Without dropout it equals dx: give NULL.
 *   dw         out, or NULL.
 * Gradients are overwritten; dx or dresidual may be dy or dh in place.  With
 * no rows, dw is set to zero.
 */
lora_status_t lora_norm_bwd(const lora_norm_t *shape, const void *dy, const void *h,
                            const void *w, const float *rstd, const void *dh,
                            const lora_dropout_t *dropout, lora_dtype_t dtype, void *dx,
                            void *dresidual, void *dw, void *workspace, size_t workspace_bytes,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_NORM_H */
