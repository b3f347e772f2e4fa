/*
 * The operators of a fine-tuning step, beside the pipeline's end stages
 * (stage_ends.h): LayerNorm with its gradients for models that use it, the
 * log-probabilities of given tokens under the vocabulary head with a gradient
 * weighted token by token, the losses that work on log-probabilities (paired
 * preferences; the clipped policy ratio with a KL term) and the global norm and
 * clipping of all gradients before the optimizer's step.  The page that
 * specoptim.h cites adapts a language model and leaves these to the trainer.
 *
 * Conventions are those of stage_ends.h: device pointers, rows without gaps,
 * tensors aligned to their elements (16-byte aligned ones take the vectorised
 * paths), asynchronous calls on `stream` that allocate nothing, workspaces of
 * the caller's (16-byte aligned, at least the bytes that the *_workspace
 * function returns, which is -1 for sizes that the call refuses; it may be NULL
 * where that is 0), the status
 * codes of specoptim.h.  No sum is formed by floating-point atomics: results
 * repeat bit for bit.  Outputs do not overlap inputs or one another unless a
 * call says that they may.
 */
#ifndef FINETUNE_H
#define FINETUNE_H

#include <stdint.h>

#include "stage_ends.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Residual sum and LayerNorm, one pass:
 *   s = x + r (rounded to the type),  mean = mean_j s_j,
 *   rstd = 1 / sqrt(mean_j (s_j - mean)^2 + eps),
 *   y = (s - mean) * rstd * gamma + beta.
 * x, r, s, y: [rows][dim], gamma, beta: [dim], all of `type` (STAGE_BF16 or
 * STAGE_FP32); mean, rstd: [rows] fp32.  r NULL: s = x, and s is not written (it
 * may be NULL).  beta NULL: none.  s may be x or r.  dim <= 32768.  Statistics are
 * fp32: where the squares of a row leave its range (differences from the mean of
 * 1e17 in wide rows, 1e19 in narrow ones), rstd is 0. */
int layernorm_forward(const void *x, const void *r, const void *gamma, const void *beta, int32_t type, float eps,
                      void *s, void *y, float *mean, float *rstd, int64_t rows, int32_t dim, void *stream);

int64_t layernorm_backward_workspace(int64_t rows, int32_t dim);

/* Backward pass of layernorm_forward, n = (s - mean) * rstd, g = gamma dy:
 *   dx     = ds + rstd * (g - mean_j g_j - n * mean_j(g_j n_j))   (= dr)
 *   dgamma = sum over rows of dy * n,  dbeta = sum over rows of dy   (fp32)
 * ds is the gradient that reaches s through the residual stream (NULL: none);
 * dbeta NULL: not formed.  dx may be dy or ds.  rows = 0 writes zeros to dgamma
 * and dbeta. */
int layernorm_backward(const void *dy, const void *ds, const void *s, const float *mean, const float *rstd,
                       const void *gamma, int32_t type, void *dx, float *dgamma, float *dbeta, int64_t rows,
                       int32_t dim, void *workspace, int64_t workspace_bytes, void *stream);

/* Log-probabilities of given tokens under the vocabulary head:
 *   logp_i = l_i,target - log sum_v exp(l_iv),  l_i = h_i w^T,
 * with the precision that head_loss describes; 0 where the target is
 * ignore_index.  For the backward pass three values are kept of each token:
 *   kept: [3][tokens] fp32, m (a whole number), 1 / sum_v 2^(log2(e) l_iv - m)
 *   and 1 - exp(logp_i); zeros where the target is ignore_index.
 * h: [tokens][dim] bf16, w: [vocab][dim] bf16 (16-byte aligned). */
int64_t head_logp_workspace(int64_t tokens, int64_t vocab, int32_t dim);
int head_logp(const void *h, const void *w, const void *targets, int32_t id_bytes, int64_t ignore_index,
              int64_t tokens, int64_t vocab, int32_t dim, float *logp, float *kept, void *workspace,
              int64_t workspace_bytes, void *stream);

/* Gradients of any loss over those log-probabilities, dlogp: [tokens] fp32:
 *   d_i = dlogp_i (onehot(target_i) - softmax(l_i)),  dh = d w  (bf16),
 *   dw = d^T h  (dw_type; added to dw if accumulate).
 * Tokens whose target is ignore_index, or whose dlogp is 0 (a clipped ratio, a
 * margin that is met), contribute nothing and cost nothing: their rows of dh
 * are 0 whatever h holds.  d enters the two products as bf16, sums are fp32. */
int64_t head_logp_backward_workspace(int64_t tokens, int64_t vocab, int32_t dim);
int head_logp_backward(const float *dlogp, const float *kept, const void *h, const void *w, const void *targets,
                       int32_t id_bytes, int64_t ignore_index, int64_t tokens, int64_t vocab, int32_t dim, void *dh,
                       void *dw, int32_t dw_type, int32_t accumulate, void *workspace, int64_t workspace_bytes,
                       void *stream);

/* Sequences of the losses below: packed one behind the other in [tokens]
 * arrays, sequence i at offsets[i] .. offsets[i + 1] - 1 (int32 or int64,
 * offset_bytes 4 or 8; not descending, within [0, tokens]).  At most 2^30 tokens
 * and sequences.  A sequence may be empty.  Tokens in front of the first and behind the last one belong to none:
 * their dlogp is 0 and nothing else of them is used.  mask: [tokens] bytes, a
 * token counts where it is not 0 (NULL: all count); what the arrays hold at
 * tokens that do not count, infinities and NaN too, reaches no output.  Offsets
 * that break the rule are moved into it, so that nothing outside the arrays is
 * touched, and reported as SPECOPTIM_ERR_BOUNDS by the next
 * specoptim_check_device; what such a call returns is not defined.  Without
 * sequences the rule is that the only offset lies within [0, tokens]. */

#define PREFERENCE_LOGISTIC 0
#define PREFERENCE_HINGE 1
#define PREFERENCE_SQUARE 2

/* Loss over pairs of sequences, sequence 2p preferred to 2p + 1:
 *   score_s = sum (average: mean) over s's tokens of logp - ref_logp,
 *   reward_s = beta score_s,  delta_p = reward_2p - reward_2p+1,
 *   logistic: -(1 - smoothing) log sigmoid(delta) - smoothing log sigmoid(-delta)
 *   hinge:    max(0, 1 - delta)
 *   square:   (delta / beta - 1 / (2 beta))^2
 *   loss = sum_p loss_p / (mean ? pairs : 1)
 * and the gradient of grad_scale * loss: dlogp [tokens] fp32.  ref_logp NULL: 0.
 * A sequence without a token that counts has score 0.  offsets: 2 pairs + 1
 * values.  pair_loss: [pairs], rewards: [2 pairs], loss: one fp32 (0 without
 * pairs). */
int64_t preference_loss_workspace(int64_t pairs, int64_t tokens);
int preference_loss(const float *logp, const float *ref_logp, const uint8_t *mask, const void *offsets,
                    int32_t offset_bytes, int64_t pairs, int64_t tokens, int32_t kind, float beta, float smoothing,
                    int32_t average, int32_t mean, float grad_scale, float *loss, float *pair_loss, float *rewards,
                    float *dlogp, void *workspace, int64_t workspace_bytes, void *stream);

#define POLICY_TOKEN_MEAN 0
#define POLICY_SEQUENCE_MEAN 1
#define POLICY_SUM 2

/* Clipped policy loss with a KL term, per token with advantage A:
 *   r = exp(logp - old_logp),
 *   gain = A >= 0 ? A min(r, 1 + clip_high) : A max(r, 1 - clip_low),
 *   kl = exp(q) - q - 1,  q = ref_logp - logp   (ref_logp NULL: kl = 0),
 *   loss = aggregate(-gain) + kl_coef aggregate(kl),
 * aggregate: the mean over the tokens that count, the mean over the sequences
 * of their tokens' means (a sequence without one adds 0), or the sum.  The
 * gradient of grad_scale * loss, dlogp [tokens] fp32, is
 *   weight (-A r [not clipped] + kl_coef (1 - exp(q))),
 * a token being clipped where r lies beyond the bound that gain takes; that is
 * decided on logp - old_logp to twice fp32's digits.  A r has fp32's digits however
 * small r is, and is 0 where A is 0 and r overflows.  With kl_coef 0 and ref_logp
 * the divergence is only reported: it reaches neither loss nor dlogp.  advantages: [tokens], or
 * [sequences] with per_sequence.  offsets NULL: all tokens are one sequence
 * (sequences is 1).  parts: aggregate(-gain), aggregate(kl), aggregate(clipped);
 * loss: one fp32.  Without a token that counts all are 0. */
int64_t policy_loss_workspace(int64_t sequences, int64_t tokens);
int policy_loss(const float *logp, const float *old_logp, const float *ref_logp, const uint8_t *mask,
                const float *advantages, int32_t per_sequence, const void *offsets, int32_t offset_bytes,
                int64_t sequences, int64_t tokens, double clip_low, double clip_high, float kl_coef,
                int32_t reduction, float grad_scale, float *loss, float *parts, float *dlogp, void *workspace,
                int64_t workspace_bytes, void *stream);

#define NORM_L2 0
#define NORM_MAX 1

/* Norm over the values of `count` tensors together, scale * grads[i][j]:
 *   NORM_L2: sqrt(sum (scale g)^2),  NORM_MAX: max |scale g|
 * to norm (one fp32); 0 without values.  grads, sizes, types: host arrays of
 * device pointers, numbers of values and STAGE_BF16 / STAGE_FP32, read before
 * the call returns.  The sum runs over the whole range of fp32: squares neither
 * overflow nor vanish. */
int64_t grad_norm_workspace(int32_t count);
int grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *types, int32_t count, float scale,
              int32_t kind, float *norm, void *workspace, int64_t workspace_bytes, void *stream);

/* outs[i] = grads[i] * scale * (norm > max_norm ? max_norm / norm : 1), rounded
 * once to out_types[i], norm as above.  outs[i] may be grads[i] where the types
 * are the same (in place); apart from that outs overlap neither one another nor
 * any of grads, which is checked.  A NaN among the values makes every value NaN,
 * an infinity makes finite values 0 and infinite ones NaN; a norm of finite values
 * that is beyond fp32 is returned as infinity, but scales them by what it is, and
 * max_norm / norm may lie far below fp32's range. */
int clip_grads(const void *const *grads, const int64_t *sizes, const int32_t *types, void *const *outs,
               const int32_t *out_types, int32_t count, float scale, float max_norm, int32_t kind, float *norm,
               void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FINETUNE_H */
