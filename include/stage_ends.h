/*
 * The operators at the two ends of a training pipeline, beside the masked
 * boundary between its stages: the first stage's embedding with its gradient,
 * the residual sum + RMSNorm that keeps its input in 8 bits for the backward
 * pass, and the last stage's softmax cross entropy over a large vocabulary
 * with its gradients ("Communication-Efficient LLM Adaptation over
 * Decentralized GPU Meshes", arXiv 2609.14339, trains a causal language model
 * through them; the page leaves their arithmetic to the model).
 *
 * Conventions: device pointers, row-major tensors without gaps between rows,
 * aligned to their element size (16-byte aligned tensors whose rows are
 * multiples of 16 bytes take the vectorised paths); the head's w is 16-byte
 * aligned.  Calls are asynchronous on
 * `stream` (a cudaStream_t as void*), return the status codes of specoptim.h
 * (message in specoptim_last_error()) and allocate nothing: where a call takes
 * a workspace, the caller provides at least the bytes its *_workspace function
 * returns (16-byte aligned, any content, free for reuse once the call's work
 * on the stream is done).  A *_workspace function returns -1 on sizes that the
 * call refuses.  Types are STAGE_BF16 or STAGE_FP32; token ids and targets are
 * int32 or int64 (id_bytes 4 or 8).  An id or target outside the vocabulary is
 * skipped and reported as SPECOPTIM_ERR_BOUNDS by the next
 * specoptim_check_device.  Results do not depend on timing: no sum is formed
 * by floating-point atomics.
 */
#ifndef STAGE_ENDS_H
#define STAGE_ENDS_H

#include <stdint.h>

#include "specoptim.h"

#ifdef __cplusplus
extern "C" {
#endif

#define STAGE_BF16 0
#define STAGE_FP32 1

/* values of an 8-bit checkpoint that share one scale, along a row */
#define STAGE_CKPT_GROUP 128

/* out[t] = scale * table[ids[t]], rounded once to out_type.
 * table: [vocab][dim], out: [tokens][dim].  The row of an id outside
 * [0, vocab) is +0. */
int embed_lookup(const void *table, int32_t table_type, const void *ids, int32_t id_bytes, int64_t tokens,
                 int64_t vocab, int32_t dim, float scale, void *out, int32_t out_type, void *stream);

int64_t embed_grad_workspace(int64_t tokens, int64_t vocab, int32_t dim);

/* grad[v] = scale * sum over t with ids[t] = v of dy[t], in fp32, rounded once
 * to grad_type; rows of absent ids are +0.  With accumulate != 0 the sum is
 * added to what grad holds and rows of absent ids are left alone.  Tokens are
 * sorted by id (stable), so each row's sum is formed in token order, in pieces
 * of a length that depends on the sizes alone.  Tokens whose id is padding_idx
 * (-1: none) contribute nothing.  dy: [tokens][dim], grad: [vocab][dim]. */
int embed_grad(const void *ids, int32_t id_bytes, const void *dy, int32_t dy_type, int64_t tokens, int64_t vocab,
               int32_t dim, int64_t padding_idx, float scale, void *grad, int32_t grad_type, int32_t accumulate,
               void *workspace, int64_t workspace_bytes, void *stream);

/* Residual sum, RMSNorm and the 8-bit checkpoint of the sum, one pass:
 *   s = x + r (rounded to the type),  rstd = 1 / sqrt(mean_j s_j^2 + eps),
 *   y = s * rstd * gamma,
 *   for each group of STAGE_CKPT_GROUP values of a row:
 *     scale = max(max_j |s_j| / 448, 2^-126),  q_j = e4m3(s_j * (1 / scale)).
 * x, r, s, y: [rows][dim], gamma: [dim], all of `type`; q: [rows][dim] bytes
 * (e4m3, nearest even), scale: [rows][ceil(dim / 128)] fp32, rstd: [rows] fp32.
 * r NULL: s = x, and s is not written (it may be NULL).  s may be x or r.  A
 * group that holds an infinity or a NaN dequantises to NaN.  dim <= 32768. */
int resnorm_forward(const void *x, const void *r, const void *gamma, int32_t type, float eps, void *s, void *y,
                    void *q, float *scale, float *rstd, int64_t rows, int32_t dim, void *stream);

/* y = n * gamma from a checkpoint, n_j = q_j * scale * rstd. */
int resnorm_recompute(const void *q, const float *scale, const float *rstd, const void *gamma, int32_t type,
                      void *y, int64_t rows, int32_t dim, void *stream);

int64_t resnorm_backward_workspace(int64_t rows, int32_t dim);

/* Backward pass of resnorm_forward from its checkpoint, n as above:
 *   dx     = ds + rstd * (gamma dy - n * mean_j(gamma_j dy_j n_j))   (= dr)
 *   dgamma = sum over rows of dy * n                                  (fp32)
 *   y      = n * gamma            (not written when y is NULL)
 * ds is the gradient that reaches s through the residual stream (NULL: none).
 * dx may be dy or ds.  rows = 0 writes dgamma = 0. */
int resnorm_backward(const void *dy, const void *ds, const void *q, const float *scale, const float *rstd,
                     const void *gamma, int32_t type, void *dx, float *dgamma, void *y, int64_t rows, int32_t dim,
                     void *workspace, int64_t workspace_bytes, void *stream);

/* Softmax cross entropy of the vocabulary head, from bf16 hidden states
 * h: [tokens][dim] and bf16 weights w: [vocab][dim]:
 *   l_i = h_i w^T (fp32 sums),  row_loss_i = log sum_v exp(l_iv) - l_i,target_i,
 *   loss = sum_i row_loss_i / (mean ? number of tokens with a target : 1).
 * The sums run on the tensor cores, which cut off what falls below fp32's last place
 * every 16 products; their mean loss, dim 2^-30 of a logit, is given back.  What is left
 * of a logit's error is within some dim 2^-30 of it either way, for exact sums of dense h
 * too; the target's logit is a separate fp32 dot product, and a logit to which only one
 * group of 16 values of h contributes is exact to fp32.
 * Tokens whose target is ignore_index have row_loss 0 and cost nothing; if no
 * token has a target, loss = 0.  row_loss: [tokens] fp32, loss: one fp32. */
int64_t head_loss_workspace(int64_t tokens, int64_t vocab, int32_t dim);
int head_loss(const void *h, const void *w, const void *targets, int32_t id_bytes, int64_t ignore_index,
              int64_t tokens, int64_t vocab, int32_t dim, int32_t mean, float *loss, float *row_loss,
              void *workspace, int64_t workspace_bytes, void *stream);

/* The loss above together with the gradients of grad_scale * loss:
 *   d_i = (softmax(l_i) - onehot(target_i)) * (mean ? 1 / tokens with a target : 1) * grad_scale
 *   dh = d w  (bf16, zero rows for ignored tokens),  dw = d^T h  (dw_type; added to dw if accumulate).
 * The vocabulary is worked through in pieces: a piece's probabilities are
 * formed again from h and w once the rows' sums are known, so no [tokens][vocab]
 * tensor exists.  Probabilities enter the two products as bf16, sums are fp32. */
int64_t head_loss_grad_workspace(int64_t tokens, int64_t vocab, int32_t dim);
int head_loss_grad(const void *h, const void *w, const void *targets, int32_t id_bytes, int64_t ignore_index,
                   int64_t tokens, int64_t vocab, int32_t dim, int32_t mean, float grad_scale, float *loss,
                   float *row_loss, void *dh, void *dw, int32_t dw_type, int32_t accumulate, void *workspace,
                   int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* STAGE_ENDS_H */
