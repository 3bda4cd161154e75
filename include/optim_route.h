/*
 * optim_route.h -- C ABI of what a mixture of experts needs around the weight
 * gradients of optim_grads.h: routing of tokens to experts with its gradient,
 * the step of the balance bias, the rows of every expert, and tokens to those
 * rows and back with their gradients.  The conventions of optim_step.h hold
 * (status codes, ownership, streams, graph capture).
 *
 * A layer's forward pass is optim_route, optim_route_rows, optim_expert_gather,
 * the experts' products, optim_expert_combine; its backward pass
 * optim_expert_combine_grad, the products' gradients with optim_expert_grad
 * (same offsets), optim_expert_combine without weights (the gradient of the
 * gather), optim_route_grad; and before the next step optim_step_route_bias.
 * Nothing of it reads the device back.
 *
 * Sizes everywhere: tokens * topk < 2^31, topk in [1, 32],
 * experts in [1, 1024], dim < 2^24, distances between rows below 2^24
 * elements and at least the row's length.  No written array may overlap
 * another array of the call, each from its first element to its last, but where
 * a call says so.  Results repeat bit for bit.
 */
#ifndef OPTIM_ROUTE_H
#define OPTIM_ROUTE_H

#include "optim_dropout.h"
#include "optim_step.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { OPTIM_ROUTE_SOFTMAX = 0, OPTIM_ROUTE_SIGMOID = 1 };

typedef struct optim_route_hp {
    int32_t topk;        /* experts of a token, at most those of top_groups
                            groups                                          */
    int32_t score;       /* OPTIM_ROUTE_*                                   */
    int32_t renormalise; /* non-zero: weights of a token sum to scale       */
    int32_t groups;      /* experts / groups neighbours are a group (1: none),
                            divides experts, at most 64                     */
    int32_t top_groups;  /* groups of a token, 1 .. groups                  */
    int32_t group_best;  /* a group counts its best one or two: 1 or 2      */
    double scale;        /* of the weights, finite in fp32                  */
} optim_route_hp;

/* ---- routing -------------------------------------------------------------
 * Per token, from its row l of logits [tokens, experts] (rows ldl elements
 * apart, dtype F32, BF16 or F16):
 *   s = softmax(l) over all experts, or sigmoid(l) each
 *   c = s + bias         (bias_dev NULL: s; the bias counts for the choice only)
 *   the choice: of the top_groups groups with the largest sum of their
 *   group_best largest c, the topk experts with the largest c, the largest
 *   first; of equal ones, groups or experts, the lower index.
 *   idx = the chosen experts (int32[tokens, topk])
 *   weights = scale s_idx, or scale s_idx / (sum of the row's s_idx)   (fp32)
 * The choice is that of c in fp64; without a bias and with group_best 1 (or no
 * groups) it goes by l, which orders s without any rounding.
 * An expert whose logit or bias is -inf or NaN is not available: it is never
 * chosen and counts for no group, a group without any is never taken, and
 * where fewer than topk are left the remaining idx are -1 with weight 0 (a
 * token all of whose logits are -inf, as in a padded batch, goes nowhere).  A
 * NaN logit makes its row's weights NaN.  A logit of +inf counts as the largest
 * float; a bias of +inf is above every float.  Weights are fp32 throughout, with
 * the hardware's exponential and reciprocal: off by less than
 *   u = (2.3 r + experts / 16 + 64) 2^-24
 * of themselves, r the distance between the row's largest and smallest finite
 * logit (those below 1e-37 by as much as that).                             */
int optim_route(const void *logits_dev, int64_t ldl, int32_t dtype, int64_t tokens,
                int32_t experts, const float *bias_dev, const optim_route_hp *hp,
                int32_t *idx_dev, float *weights_dev, void *stream);

/* The gradient of the weights by the logits: dlogits [tokens, experts] (rows
 * ldd elements apart, the logits' dtype, written whole) from dweights, the
 * gradient of the weights, and the idx of optim_route (the choice itself has no
 * gradient).  With g = scale dweights where idx is an expert (a dweights beside
 * an idx outside [0, experts) is not looked at), w = s_idx / (sum of s_idx):
 *   softmax:               dl_e = s_e ([e = idx_j] g_j - sum_j g_j s_idx_j)
 *   softmax, renormalised: dl_e = [e = idx_j] w_j (g_j - sum_j g_j w_j)
 *   sigmoid:               dl_e = [e = idx_j] g_j s_e (1 - s_e)
 *   sigmoid, renormalised: dl_e = [e = idx_j] w_j (1 - s_e) (g_j - sum_j g_j w_j)
 * An expert named twice in a row counts twice.  Only the first form reads more
 * of the logits than the chosen ones.  An expert whose logit is -inf or NaN has
 * gradient 0, and a NaN changes no other one's; the bias is not in the scores, so
 * an expert that only its bias shuts has its s_e in the first form.  Each element
 * is fp32, off by less than 2 u (above) of the sum of its terms' magnitudes, where
 * g_e s_e (1 - s_e) counts as one term, and then rounded once to the logits' dtype. */
int optim_route_grad(const void *logits_dev, int64_t ldl, int32_t dtype, int64_t tokens,
                     int32_t experts, const optim_route_hp *hp, const int32_t *idx_dev,
                     const float *dweights_dev, void *dlogits_dev, int64_t ldd, void *stream);

/* The step of the balance bias (L. Wang et al., "Auxiliary-loss-free load
 * balancing strategy for mixture-of-experts", arXiv:2408.15664): with the load
 * n_e = offsets_dev[e + 1] - offsets_dev[e] of every expert,
 *   bias_e <- bias_e + *rate_dev * sign(mean of n - n_e)
 * Nothing changes where found_inf_dev is given and *found_inf_dev is not 0.
 * (Loads of several ranks: pass the running sums of the summed loads.)      */
int optim_step_route_bias(const int32_t *offsets_dev, int32_t experts, float *bias_dev,
                          const float *rate_dev, const float *found_inf_dev, void *stream);

/* ---- rows of the experts ---------------------------------------------------
 * The choices sorted by expert, those of one expert in the order of tokens:
 *   offsets_dev[e]      first row of expert e; [experts]: rows in all
 *                       (int32[experts + 1], as optim_expert_grad takes them)
 *   place_dev[t, j]     row of choice j of token t, -1 where idx is outside
 *                       [0, experts)                  (int32[tokens, topk])
 *   order_dev[row]      t * topk + j of the row's choice, -1 in the rows behind
 *                       the last          (int32[tokens * topk]; may be NULL)
 * `workspace` (device, 256-byte aligned, optim_route_rows_workspace bytes,
 * contents free between calls) may be NULL where that is 0.                 */
int optim_route_rows_workspace(int64_t tokens, int32_t topk, int32_t experts, size_t *bytes);
int optim_route_rows(const int32_t *idx_dev, int64_t tokens, int32_t topk, int32_t experts,
                     int32_t *offsets_dev, int32_t *place_dev, int32_t *order_dev,
                     void *workspace, size_t workspace_bytes, void *stream);

/* ---- tokens to the experts' rows and back ----------------------------------
 * Matrices of `dim` columns, rows ld* elements apart, all of one dtype (F32,
 * BF16, F16; aligned to their element size); weights fp32[tokens, topk], NULL
 * for 1.  A place outside [0, rows) is no row: it is read and written nowhere,
 * whatever its weight.  No row may have two places.  Sums are fp32, over j in
 * order, rounded once.
 *
 * optim_expert_gather:  y[place[t, j]] = weights[t, j] x[t]
 *   Rows of y without a place stay as they are.                             */
int optim_expert_gather(const void *x_dev, int64_t ldx, int32_t dtype, const int32_t *place_dev,
                        const float *weights_dev, int64_t tokens, int32_t topk, int64_t dim,
                        void *y_dev, int64_t ldy, int64_t rows, void *stream);

/* out[t] = drop(sum_j weights[t, j] y[place[t, j]])       (residual_dev NULL)
 * out[t] = residual[t] + drop(...)                        (otherwise)
 * drop: dropout as in optim_dropout.h, element (t, d) at place first + t * dim +
 * d, or nothing where drop is NULL.  out_dev may be residual_dev itself (and ldo
 * ldr).  Without weights, residual and drop it is the gradient of
 * optim_expert_gather without weights.                                      */
int optim_expert_combine(const void *y_dev, int64_t ldy, int64_t rows, int32_t dtype,
                         const int32_t *place_dev, const float *weights_dev, int64_t tokens,
                         int32_t topk, int64_t dim, const void *residual_dev, int64_t ldr,
                         const optim_dropout_hp *drop, const int32_t *step_dev, void *out_dev,
                         int64_t ldo, void *stream);

/* The gradients of optim_expert_combine, from dout, that of out, with
 * d = drop(dout):
 *   dy[place[t, j]]   = weights[t, j] d[t]
 *   dweights[t, j]    = sum over the columns of d[t] y[place[t, j]], 0 without a row
 * (the residual's is dout).  Rows of dy without a place stay as they are.
 * dweights_dev or dy_dev NULL: not wanted (without dweights_dev, y_dev is not
 * read).  dy_dev may be y_dev itself (and lddy ldy).  The gradient of a gather
 * with weights: of x, optim_expert_combine of y's gradient with these weights; of
 * the weights, this call with x for dout, y's gradient for y, dy_dev NULL.  */
int optim_expert_combine_grad(const void *dout_dev, int64_t ldd, int32_t dtype, const void *y_dev,
                              int64_t ldy, int64_t rows, const int32_t *place_dev,
                              const float *weights_dev, int64_t tokens, int32_t topk, int64_t dim,
                              const optim_dropout_hp *drop, const int32_t *step_dev, void *dy_dev,
                              int64_t lddy, float *dweights_dev, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* OPTIM_ROUTE_H */
