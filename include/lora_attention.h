/*
 * lora_attention.h -- attention between the q, k, v and o LoRA layers.
 *
 * Scores may be capped by a tanh, get a bias that falls with distance, and be
 * masked by documents and by a prefix (ch05 "Acceleration principles: Triton
 * kernels and fused LoRA", §5.10, a score and mask function per pair; packed
 * documents as in the padding-free packing of the Unsloth essay).  For query
 * i of q_len and key j of k_len, the queries being the last q_len of k_len
 * positions, p_i = i + k_len - q_len:
 *
 *     z = scale * q_i . k_j
 *     c = cap * tanh(z / cap)                        (softcap > 0; else c = z)
 *     s = c - slope_h * |p_i - j|                    (slopes given)
 *     visible = (not causal or j <= p_i or j < prefix_b)
 *               and (no documents or q_doc_i == k_doc_j >= 0)
 *     P = softmax of s over the visible j,  o_i = sum_j P_ij v_j,
 *     lse_i = log sum_j exp s_ij
 *
 * A row that sees nothing gives o = 0, lse = -inf and zero gradients.  A
 * document below zero is padding: it sees nothing and is not seen, and
 * whatever its q, k, v, o and do hold (NaN included) reaches no result.
 * Elsewhere a masked pair's score is replaced, never added to; its v and k
 * are still multiplied by an exact zero, so they have to be finite.
 *
 * Backward:
 *     dv = P^T do,  dP = do v^T,  delta_i = do_i . o_i,  ds = P (dP - delta),
 *     dz = ds (1 - (c / cap)^2),  dq = scale dz k,  dk = scale dz^T q
 * (dk and dv summed over the query heads that share a key head; slopes are
 * constants).
 *
 * Types: bf16 tensors, fp32 lse.  Scores, softmax statistics and all sums in
 * fp32; P and dz are rounded to bf16 as tensor-core operands (P not with one
 * token), and delta comes from o as it was stored, but from P and dP for queries
 * whose keys lie in one 128-aligned tile of keys (the first of a causal mask,
 * short documents, at most 128 keys): dq and dk are off by 0.0025 to 0.0035 of
 * their norm where rounding them alone takes 0.0017, more in a row of keys in
 * several tiles that looks almost wholly at one of them.
 * Layout: any
 * strides in elements for (batch, token, head), a head's dim elements
 * contiguous; q [batch, q_len, q_heads, dim], k and v [batch, k_len, k_heads,
 * dim], o like q, lse [batch, q_heads, q_len] contiguous.  Query head h reads
 * key head h / (q_heads / k_heads).  Requirements: dim % 8 == 0, 8 <= dim <=
 * 128, q_heads % k_heads == 0, 16-byte aligned pointers, strides of multiples
 * of 8 elements (above 0, but for o in the backward and q, k and v with one
 * token, which may be broadcast), q_len and k_len < 2^24, batch and q_heads <
 * 2^16, at most 2^33 rows (batch * q_heads * (q_len + k_len + 1)) and 2^30 tiles
 * of 128 tokens over all heads.
 *
 * Errors, streams, determinism, the status word and the timing hook are those
 * of lora_linear.h.  Nothing is allocated; no host synchronisation.
 */
#ifndef LORA_ATTENTION_H
#define LORA_ATTENTION_H

#include "lora_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t batch, q_len, k_len;
    int32_t q_heads, k_heads, dim;
    int32_t causal;               /* 0 or 1                                   */
    float scale;                  /* finite, > 0                              */
    float softcap;                /* > 0: the cap; 0: none                    */
    int64_t q[3], k[3], v[3], o[3];         /* strides: batch, token, head    */
    int64_t d_o[3], dq[3], dk[3], dv[3];    /* same, backward only            */
    const float *slopes;          /* device [q_heads], or NULL                */
    const int32_t *q_docs;        /* device, token i of batch b at            */
    const int32_t *k_docs;        /*   [b * stride + i]; both or neither      */
    int64_t q_docs_stride, k_docs_stride;
    const int32_t *prefix;        /* device [batch], or NULL; needs causal    */
} lora_attention_t;

/* Bytes of device workspace of the forward (backward = 0) or the backward
 * pass.  0 for bad arguments. */
size_t lora_attention_workspace_bytes(const lora_attention_t *shape, int backward);

/* o and lse from q, k and v, which o must not overlap.  lse may be NULL where no
 * backward follows. */
lora_status_t lora_attention_fwd(const lora_attention_t *shape, const void *q, const void *k,
                                 const void *v, void *o, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* dq, dk and dv from do and the forward's tensors.  Outputs are overwritten;
 * they must not overlap an input. */
lora_status_t lora_attention_bwd(const lora_attention_t *shape, const void *d_o, const void *q,
                                 const void *k, const void *v, const void *o, const float *lse,
                                 void *dq, void *dk, void *dv, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * One new token per sequence over a static cache: q [batch, q_heads, dim]
 * against the first lengths[b] of k_len positions of k and v, the token being
 * the last of them (p = lengths[b] - 1).  Uses of `shape`: the sizes with
 * q_len = 1, scale, softcap, slopes and the strides of q, k, v and o; causal,
 * documents and prefix must be unset (the new token sees all that is kept).
 *   lengths    in, device int32 [batch]; clamped to [0, k_len].  With 0 the
 *              output is zero.  What lies past a length is not read.
 *   workspace  device scratch of lora_attention_token_workspace_bytes.
 * One launch, or two where the cache's length is split over blocks: the second
 * joins the parts in a fixed order.
 */
size_t lora_attention_token_workspace_bytes(const lora_attention_t *shape);
lora_status_t lora_attention_token(const lora_attention_t *shape, const void *q, const void *k,
                                   const void *v, const int32_t *lengths, void *o,
                                   void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_ATTENTION_H */
