/*
 * optim_grads.h -- C ABI of the operators on gradients around the optimizer
 * step of optim_step.h: norms of every tensor of a list and of the whole,
 * clipping where the gradients lie, and the weight gradients of a mixture of
 * experts.  The conventions of optim_step.h hold for every entry point here
 * (status codes, ownership, streams, graph capture); in addition
 * optim_clip_grads and optim_expert_grad write gradients.
 */
#ifndef OPTIM_GRADS_H
#define OPTIM_GRADS_H

#include "optim_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- gradient lists -----------------------------------------------------
 * A plan of algorithm OPTIM_ALGO_GRADS holds the gradients of a list and
 * nothing else: numel, grad and grad_dtype of optim_tensor_list are read
 * (grad_dtype F32, BF16 or F16; arrays aligned to their element size, any
 * tensor may begin anywhere in a bucket), every other pointer is ignored and
 * may be NULL.  It is made, traced and destroyed as every plan
 * (optim_plan_create, optim_plan_create_static, ...); opts may be NULL, and
 * tile, grid, state_dtype and state_layout must be 0 in it.  No two tensors
 * may overlap.  The calls of one plan must not overlap each other (they
 * share its workspace).  A plan holds addresses: gradients that move need a
 * new one (0.4 ms of host time and a copy for 6000 tensors, which a call of
 * 10 us does not earn back), so keep them where they are from step to step.
 * The steps, optim_check_finite and optim_grad_norm refuse such a plan
 * (OPTIM_EINVAL); optim_grad_norms does both of the latter.                */

/* Norms: square root of the sum of squares, sum of magnitudes, largest
 * magnitude.                                                              */
enum { OPTIM_NORM_L2 = 0, OPTIM_NORM_L1 = 1, OPTIM_NORM_INF = 2 };

/* The norm of every tensor of the list and of the whole list, of the
 * unscaled gradients g = G * s, s = *inv_scale_dev (NULL: 1), in one read of
 * the gradients:
 *   norms_dev[i] = ||g_i||   (float[n]; 0 for an empty tensor; may be NULL)
 *   *total_dev   = ||(g_1, ..., g_n)||, from the unrounded sums
 *   *coef_dev    = s * min(1, max_norm / (total + 1e-6))   (may be NULL)
 * max_norm <= 0 or +inf: no clipping (coef = s); NaN is OPTIM_EINVAL.
 * found_inf_dev (may be NULL) is set to 1.0f if any element is NaN or +-Inf
 * and left unchanged otherwise, as by optim_check_finite; the norms of the
 * tensors concerned and the total are then not finite, and coef = s.
 * A 16-byte group of 4 or 8 elements is summed in fp32 and the groups in
 * fp64, so a sum is within 7 * 2^-24 of itself.  Where an item (a run of a
 * tensor's elements, or a small tensor) has a largest magnitude from which
 * fp32 sums could overflow (2^62 for L2, 2^120 for L1) or below 2^-40, its
 * elements are summed again in fp64 alone.  The order of sums is fixed by the
 * list and by where its arrays begin within 16 bytes, so results repeat bit
 * for bit; a finite list has finite norms (up to fp32's range).           */
int optim_grad_norms(optim_plan *plan, int32_t kind, const float *inv_scale_dev,
                     double max_norm, float *found_inf_dev, float *norms_dev,
                     float *total_dev, float *coef_dev, void *stream);

/* One norm over several lists (a model stepped by two algorithms), or over
 * the ranks of a sharded one (their totals gathered into one array): from
 * norms_dev[count], norms of the unscaled gradients of disjoint lists,
 *   *total_dev = their norm of the same kind,
 *   *coef_dev  = s * min(1, max_norm / (total + 1e-6)), s = *inv_scale_dev.
 * Rules for max_norm and a total that is not finite as in optim_grad_norms.
 * total_dev may be an element of norms_dev; count 0 gives total 0.
 * total_dev or coef_dev may be NULL.                                      */
int optim_clip_coef(const float *norms_dev, int64_t count, int32_t kind,
                    const float *inv_scale_dev, double max_norm,
                    float *total_dev, float *coef_dev, void *stream);

/* G <- G * *coef_dev in every gradient of the list, the product in fp32,
 * rounded once to the gradient's type (nearest even).  Nothing is read or
 * written where *coef_dev is 1, or where found_inf_dev is given and
 * *found_inf_dev is not 0 (the step that follows is skipped).  With the coef
 * of optim_grad_norms the gradients are then unscaled and clipped: the step
 * that follows takes inv_scale NULL.                                      */
int optim_clip_grads(optim_plan *plan, const float *coef_dev,
                     const float *found_inf_dev, void *stream);

/* ---- experts' weight gradients -------------------------------------------
 * The weight gradients of a layer of experts, Y_e = X_e W_e, from the rows
 * routed to each, sorted by expert: with X [tokens, m] and dY [tokens, n]
 * (rows ldx and ldy elements apart, in_dtype BF16 or F16) and expert e's rows
 * [offsets_dev[e], offsets_dev[e + 1]),
 *   dW_e = s X_e^T dY_e            (accumulate 0)
 *   dW_e = dW_e + s X_e^T dY_e     (otherwise)
 * for dW [experts, m, n] (dw_dtype F32 or BF16, rows and experts end to end),
 * s = *scale_dev (NULL: 1).  Products on the matrix cores, sums in fp32, one
 * rounding to dw_dtype.  It fills gradients that the plans of a step, of
 * optim_grad_norms and of optim_clip_grads read; accumulating over the
 * micro-batches of a step into fp32 loses nothing to 16 bits in between.
 * An expert without rows gets zeros (or keeps dW_e).  offsets_dev (device
 * int32[experts + 1]) is read by the kernel, so routing needs no host
 * synchronisation; each bound is clamped to [0, tokens], and a run's end to
 * its own beginning.  (Bounds are meant to ascend: where one is below the one
 * before it, that run is empty and the next begins there, so rows may count
 * for two experts.)  Rows outside every run are not read.
 * Runs are summed in one piece, or, where the tiles of dW are too few to fill
 * the GPU, in pieces through `workspace` (device, 256-byte aligned,
 * optim_expert_grad_workspace bytes, contents free between calls); NULL
 * sums in one piece, too few bytes are OPTIM_EWORKSPACE.  Either way the order of
 * sums is fixed by the sizes: results repeat bit for bit.
 * tokens < 2^31; m, n < 2^24; fewer than 2^18 blocks of 512 x 512 over all
 * experts (an expert is at least one); m <= ldx < 2^24, n <= ldy < 2^24.  dW
 * must not overlap X, dY, offsets_dev or the workspace.  16-byte aligned X and
 * dY with m, n, ldx and ldy multiples of 8 take the fastest path.          */
int optim_expert_grad_workspace(int32_t experts, int64_t tokens, int64_t m,
                                int64_t n, size_t *bytes);
int optim_expert_grad(const void *x_dev, int64_t ldx, const void *dy_dev,
                      int64_t ldy, int32_t in_dtype, const int32_t *offsets_dev,
                      int32_t experts, int64_t tokens, int64_t m, int64_t n,
                      void *dw_dev, int32_t dw_dtype, int32_t accumulate,
                      const float *scale_dev, void *workspace,
                      size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* OPTIM_GRADS_H */
