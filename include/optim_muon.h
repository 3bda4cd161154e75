/*
 * optim_muon.h -- C ABI of the Muon step: momentum whose direction is
 * orthogonalised matrix by matrix, for the two-dimensional parameters of a
 * model (the others are stepped by the algorithms of optim_step.h).  The
 * conventions of optim_step.h hold (status codes, ownership, streams, graph
 * capture).
 *
 * After K. Jordan et al., "Muon: An optimizer for hidden layers in neural
 * networks" (2024), and J. Liu et al., "Muon is scalable for LLM training"
 * (arXiv:2502.16982), for decoupled weight decay and the scale that matches
 * an AdamW update's.
 */
#ifndef OPTIM_MUON_H
#define OPTIM_MUON_H

#include "optim_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- plans --------------------------------------------------------------
 * Algorithm OPTIM_ALGO_MUON.  Read from optim_tensor_list: numel, param,
 * grad, m (float[numel], the momentum), weight_decay, rows, cols, and
 * remainder or master as for AdamW (param_dtype F32; BF16 with remainder;
 * BF16 or F16 with master).  Tensor i holds numel / (rows * cols) matrices
 * of rows x cols each, row by row, one after another (the weights of a
 * layer's experts are one tensor); rows, cols in [1, 2^20], and numel must
 * be a multiple of rows * cols (0: skipped).  Fewer than 2^23 matrices in all.
 * opts: segment_bytes bounds the workspace that the matrices of one run of
 * launches take (0 = 4 GiB; a larger matrix has a run alone); results do not
 * depend on it.  grid, state_dtype and state_layout must be 0.
 * The workspace holds, for every matrix of the largest run, about 8 bytes an
 * element and 8 bytes times the square of its shorter side, sides rounded up
 * to 32 (with a side of at most 128: up to 12 bytes an element, that side
 * rounded up to 64 or 128), up to 64 MB beside, and tables of about 150 bytes
 * a matrix of the plan.
 * optim_check_finite, optim_grad_norm, optim_plan_set_schedule and
 * optim_plan_trace take such a plan as any other.                          */

/* Factor of the update of a rows x cols matrix: 1; sqrt(max(1, rows/cols));
 * 0.2 sqrt(max(rows, cols)), which gives the update the root mean square of
 * a typical AdamW update's.                                               */
enum { OPTIM_MUON_SCALE_NONE = 0, OPTIM_MUON_SCALE_ASPECT = 1, OPTIM_MUON_SCALE_RMS = 2 };

typedef struct optim_muon_hp {
    double momentum;      /* mu, in [0, 1)                                  */
    double eps;           /* added to the norm, finite and >= 0 (1e-7)      */
    double a, b, c;       /* the quintic (3.4445, -4.7750, 2.0315)          */
    int32_t steps;        /* its applications, 1 .. 16 (5)                  */
    int32_t nesterov;     /* non-zero: the direction is g + mu m            */
    int32_t scale_kind;   /* OPTIM_MUON_SCALE_*                             */
} optim_muon_hp;

/* With g = grad * inv_scale, per element and then per matrix:
 *   m <- mu m + g;   u = g + mu m (nesterov) or m
 *   X = u / (||u||_F + eps)
 *   steps times:  A = X X^T (on the shorter side), B = b A + c A A,
 *                 X <- a X + B X
 *   p <- p - (lr wd p + lr f X),  f the factor above
 * m in fp32 without contraction; the sum of squares in fp64.  X, A and B are
 * kept as sums of two fp16 numbers and multiplied on the matrix cores as three
 * products of parts with fp32 sums (the product of both low parts, 2^-22 of the
 * whole, is left out).  An element has 22 significant bits down to 2^-15 (of
 * X, whose norm is 1 at first), below that an absolute error of up to 2^-37,
 * which the iteration raises as it raises small singular values (a each step,
 * 485 for five).  So the update agrees with the exact one as an fp32
 * iteration's does, to 1e-6 (64 x 64) to 3e-6 (4096 x 4096) of its norm,
 * where no part of the matrix is far smaller than the rest; beside elements
 * 1e6 to 1e9 times as large to 4e-6 to 1.3e-5 of its norm, where fp32 comes to
 * 1e-7; and rows 1e-6 of the others' size are updated to 2e-4 (64 x 64) to
 * 1.3e-2 (4096 x 4096) of their own small update.
 * Orders of summation are fixed: results repeat bit for bit.
 * A matrix of zeros (an expert without tokens, fresh momentum) has update 0.
 * The polynomial must keep X within what the 16-bit parts hold: the bounds
 * |X|, |B| <= 15 are followed through all steps from |X| <= 1 (the largest
 * singular value), else OPTIM_EINVAL.  A NaN / Inf in a gradient without
 * found_inf makes its matrix NaN, and no other.
 * lr_dev, inv_scale_dev, found_inf_dev, step_dev, schedule: as for the steps
 * of optim_step.h (the step count is advanced, not used).                  */
int optim_step_muon(optim_plan *plan, const optim_muon_hp *hp, float *lr_dev,
                    const float *inv_scale_dev, const float *found_inf_dev,
                    int32_t *step_dev, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* OPTIM_MUON_H */
