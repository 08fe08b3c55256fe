/*
 * lora_rotary.h -- rotary positions for the outputs of the q and k LoRA layers.
 *
 * ch05 "Acceleration principles: Triton kernels and fused LoRA", §5.5 (fused
 * RoPE: q and k in one kernel, in place, variable lengths).  Per token with
 * position p, head and pair i < rot / 2 of its elements (x, y):
 *
 *     a = p * w_i
 *     x' = m (x cos a - y sin a)      y' = m (y cos a + x sin a)
 *
 * with m the magnitude.  Pairs are (i, i + rot/2) (half layout) or
 * (2i, 2i + 1) (interleaved); elements from `rot` on are copied.  The
 * backward of the operator is the same with -a (inverse = 1).
 *
 * Frequencies are given in turns per position as 64-bit fractions, turns_i =
 * frac(w_i / 2 pi) * 2^64 to the nearest (lora_rotary_turns; w_i as the double
 * that it is).  Position times turns modulo 2^64 is the reduced angle (negative
 * positions included): off by at most 2^-65 of a turn for every position, below
 * the 2^-24 that the angle is then rounded to up to position 2^41.
 *
 * Errors, streams and the timing hook are those of lora_linear.h.  Nothing
 * is allocated; no host synchronisation.  One launch.
 */
#ifndef LORA_ROTARY_H
#define LORA_ROTARY_H

#include "lora_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes and layouts.  Strides are in elements, for (batch, token, head); the
 * elements of a head are contiguous. */
typedef struct {
    int64_t batch, seq;            /* >= 0                                    */
    int32_t q_heads, k_heads;      /* >= 0; with 0 the pointers may be NULL   */
    int32_t dim, rot;              /* rot even, 2 <= rot <= dim <= 1024       */
    int32_t interleaved, inverse;  /* 0 or 1                                  */
    int32_t position_bits;         /* 32 or 64 (signed)                       */
    float magnitude;
    int64_t q_in[3], k_in[3], q_out[3], k_out[3];
    int64_t position[2];           /* strides of the positions: batch, token  */
} lora_rotary_t;

/* turns[i] = frac(radians[i] / 2 pi) * 2^64, to the nearest, for n finite
 * frequencies, on the host. */
lora_status_t lora_rotary_turns(const double *radians, int n, uint64_t *turns);

/*
 * Turns q and k.
 *   q, k          in, device, bf16 or fp32 by dtype, aligned to their type.
 *   positions     in, device, one integer per token.
 *   turns         in, device, rot / 2 words.
 *   q_out, k_out  out, device, same dtype.  An output may be its input (same
 *                 address and strides: in place); otherwise it must not
 *                 overlap any input.  Not broadcast (strides other than 0).
 * batch * seq == 0 launches nothing; it has to be less than 2^31
 * (LORA_ERR_UNSUPPORTED).
 */
lora_status_t lora_rotary(const lora_rotary_t *shape, const void *q, const void *k,
                          const void *positions, const uint64_t *turns, lora_dtype_t dtype,
                          void *q_out, void *k_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_ROTARY_H */
