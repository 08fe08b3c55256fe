/*
 * lora_clip.h -- the global norm of many gradient tensors, and clipping by it.
 *
 *     n = (sum over all tensors of g^2)^(1/2)     or  n = max |g|
 *     c = min(1, max_norm / (n + 1e-6))           g' = c g
 *
 * A fine-tuning step ends with it over the dA and dB of every LoRA layer
 * (lora_linear.h).  The tensors' addresses, sizes and types are laid out once
 * in a plan, which the caller keeps as long as the tensors stay where they
 * are (a training loop that makes new gradients each step, as PyTorch's
 * zero_grad() does by default, has to make a new plan or clear them in place).  Tensors may mix bf16 and fp32, have any size and any alignment of
 * their type.
 *
 * Sums: at most 33 squares in fp32, then unevaluated pairs of fp32 and fp64;
 * where a partial sum leaves the range fp32 squares can hold, it is taken
 * again in fp64, so that the norm is right over the whole range of the inputs.  The order of
 * every sum is fixed: the same plan and values give the same bits.  NaN or
 * infinite gradients give a NaN or infinite norm, and c as the formula has
 * it (NaN, or 0).
 *
 * Errors, streams and the timing hook are those of lora_linear.h.  Nothing
 * is allocated; no host synchronisation.
 */
#ifndef LORA_CLIP_H
#define LORA_CLIP_H

#include "lora_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void *in; /* device, aligned to its type                          */
    void *out;      /* device; `in` itself (in place), or memory of its own:
                       no other tensor's, in or out                          */
    int64_t count;  /* elements, >= 0 (0: the pointers may be NULL)          */
    int32_t dtype;  /* lora_dtype_t of both                                  */
} lora_clip_tensor_t;

/* Bytes of the plan of these tensors; 0 for bad arguments. */
size_t lora_clip_plan_bytes(const lora_clip_tensor_t *tensors, int n);

/* Writes the plan's image to HOST memory (outputs that share memory are
 * refused).  The caller copies it to a 16-byte
 * aligned device buffer of the same size, which lora_clip_norm and lora_clip
 * take.  The device copy holds scratch too: calls with one plan that overlap
 * on the GPU race on it. */
lora_status_t lora_clip_plan_build(const lora_clip_tensor_t *tensors, int n, void *image,
                                   size_t image_bytes);

/* norm[0] (device, fp32) = the norm of all inputs; largest = 0: the 2-norm,
 * 1: the largest magnitude.  plan_bytes: the size of the plan.  One launch. */
lora_status_t lora_clip_norm(void *plan, size_t plan_bytes, int largest, float *norm,
                             void *stream);

/* The same, then out = c in for every tensor.  max_norm >= 0.  Two launches;
 * in-place tensors are not touched where c is 1. */
lora_status_t lora_clip(void *plan, size_t plan_bytes, float max_norm, int largest, float *norm,
                        void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_CLIP_H */
