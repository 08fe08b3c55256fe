/*
 * lora_loss.h -- softmax cross entropy of a frozen head over a large vocabulary,
 * with the gradient of the hidden states, without keeping the logits.
 *
 * ch05 "Acceleration principles: Triton kernels and fused LoRA", §5.7 (chunked
 * cross entropy: the logits are never materialised).  For token n with target
 * t_n and weight w_n (1 where none are given):
 *
 *     z_nv   = c(X_n . W_v),   c(z) = z, or softcap tanh(z / softcap)
 *     loss_n = log(sum_v exp z_nv) - z_n,t
 *     loss   = sum_n g_n loss_n,   g_n = w_n / sum of the w (mean), or w_n (sum)
 *     dX_n   = g_n sum_v (p_nv - [v = t_n]) c'(X_n . W_v) W_v,   p = softmax(z)
 *
 * over the tokens that count: those with t_n >= 0.  The others (padding,
 * prompts) cost nothing but their line of zeros in `losses` and dX.  Where the
 * weights' sum is 0 the mean is taken as the sum.  A target >= vocab shows as
 * NaN in its token's outputs and in the loss.  W is frozen: it has no gradient.
 *
 * The two products run on the tensor cores (bf16, fp32 accumulators) strip by
 * strip of tokens.  Of a strip's logits only exp(z_nv - z_n,t) is kept between
 * the products, in bf16 (one rounding, to half a step, of each p_nv - [v = t_n];
 * the sums are of the unrounded numbers, in fp32); without dX nothing is kept.
 * Sums have a fixed order: the same call gives the same bits.  Errors, streams,
 * the status word and the timing hook are those of lora_linear.h.  Nothing is
 * allocated; no host synchronisation.
 */
#ifndef LORA_LOSS_H
#define LORA_LOSS_H

#include "lora_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t rows;        /* tokens, 0 .. 2^31 - 65537                         */
    int64_t vocab;       /* 1 .. 2^31 - 512                                   */
    int32_t dim;         /* a multiple of 8, 8 .. 65536                       */
    int32_t target_bits; /* 32 or 64 (signed)                                 */
    int32_t mean;        /* 1: divide by the sum of the weights; 0: do not    */
    float softcap;       /* 0: none; else 2^-100 .. 2^100                     */
    int64_t x, w, dx;    /* row strides in elements: multiples of 8, >= dim   */
} lora_loss_t;

/* Bytes of device workspace lora_loss needs, with dX or without (0 for bad
 * arguments).  It holds a strip of tokens, and four bytes a token: at most 716 MB
 * (of 2^20 bytes) and these where 256 tokens fit (with dX, vocabularies up to a
 * million words), else what 256 tokens take. */
size_t lora_loss_workspace_bytes(const lora_loss_t *shape, int with_dx);

/*
 *   X          in, device, bf16 [rows, dim], 16-byte aligned.
 *   W          in, device, bf16 [vocab, dim], 16-byte aligned.
 *   targets    in, device, one integer a token.
 *   weights    in, device, one float a token, or NULL (all 1).
 *   loss       out, device, one float.
 *   losses     out, device, one float a token (not weighted; 0 where t_n < 0);
 *              not the weights' tensor.
 *   dX         out, device, bf16 [rows, dim], or NULL: the gradient of loss.
 *              It may be X itself (same stride).
 * With no tokens that count, loss is 0.
 */
lora_status_t lora_loss(const lora_loss_t *shape, const void *X, const void *W,
                        const void *targets, const float *weights, float *loss, float *losses,
                        void *dX, void *workspace, size_t workspace_bytes, void *stream);

/* out = factor[0] dX, bf16 [rows, dim] with strides shape->dx and shape->x: the
 * gradient where more follows the loss (factor: fp32, device).  out may be dX
 * (same stride). */
lora_status_t lora_loss_scale(const lora_loss_t *shape, const void *dX, const float *factor,
                              void *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_LOSS_H */
