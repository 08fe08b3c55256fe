/*
 * lora_dropout.h -- dropout whose mask is never stored.
 *
 * The Unsloth essay's recipe table has a dropout rate beside the rank; where it
 * is not 0, an element of row n and column c is kept if
 *
 *     word(n, c) >= T,   T = round(p 2^32)
 *
 * and then multiplied by 2^32 / (2^32 - T) (the expectation is kept exactly);
 * else it is 0, whatever it was (NaN and infinities too).  The words come from
 * the counter-based generator Philox4x32 with ten rounds (Salmon, Moraes, Dror
 * and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011):
 *
 *     word(n, c) = Philox(counter = (c / 4, n mod 2^32, n / 2^32, offset),
 *                         key = (seed mod 2^32, seed / 2^32)) [c mod 4]
 *
 * so that the backward makes the forward's mask again from (seed, offset), for
 * any strides, type and order of the work.  Give every dropout of a step an
 * offset of its own, and every step another seed (or other offsets).
 *
 * Errors, streams and the timing hook are those of lora_linear.h.  Nothing is
 * allocated; no host synchronisation.  One launch.
 */
#ifndef LORA_DROPOUT_H
#define LORA_DROPOUT_H

#include "lora_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    double p;               /* 0 <= p, and round(p 2^32) < 2^32               */
    uint64_t seed;
    uint32_t offset;
    const uint64_t *state;  /* NULL, or two words on the device, read when the
                               kernel runs: seed = state[0] and offset + state[1]
                               (mod 2^32) take the place of seed and offset, so
                               that a captured graph can be replayed with other
                               masks                                          */
} lora_dropout_t;

/*
 * y = dropout(x); the gradient of x from that of y is the same call.
 *   x, y      device, bf16 or fp32 by dtype, aligned to their type, rows of
 *             `cols` contiguous elements `x_stride` (`y_stride`) apart.  y may
 *             be x (same strides: in place); otherwise they must not overlap.
 * rows, cols >= 0; rows * cols == 0 launches nothing; cols < 2^31, rows <=
 * 2^36, at most 2^40 elements; the rows of y do not overlap (y_stride >= cols
 * where rows > 1).
 */
lora_status_t lora_dropout(const void *x, int64_t rows, int64_t cols, int64_t x_stride,
                           int64_t y_stride, const lora_dropout_t *dropout, lora_dtype_t dtype,
                           void *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_DROPOUT_H */
