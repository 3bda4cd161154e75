/*
 * optim_dropout.h -- C ABI of dropout whose mask is drawn from a counter and
 * never stored: the backward pass draws it again from the same numbers.  The
 * conventions of optim_step.h hold (status codes, ownership, streams, graph
 * capture).
 */
#ifndef OPTIM_DROPOUT_H
#define OPTIM_DROPOUT_H

#include "optim_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What a mask is drawn from.  Element i of a call (0, 1, ... in memory order,
 * rows end to end whatever their distance) has place q = first + i and the 16
 * bits r(q): of the four words that Philox4x32-10 (J. Salmon et al., "Parallel
 * random numbers: as easy as 1, 2, 3", SC 2011) gives for
 *   counter (q/8 mod 2^32, q/8 div 2^32, *step_dev, site)
 *   key     (seed mod 2^32, seed div 2^32)
 * word (q mod 8) div 2, its low half for even q, its high half for odd q.
 * Steps that are counted on the device (the step_dev of a plan's calls) thus
 * draw anew at every replay of a captured graph that moves the count, and a tensor
 * in pieces, or one sharded over ranks, has the mask of the whole where each piece
 * says where it begins.  All calls of one step, site and first have one mask:
 * micro-batches whose gradients one step takes are pieces too, and each says where
 * it begins (micro-batch i of n elements: i * n); so do ranks with batches of their
 * own.  A step that is skipped (found_inf) is not counted, and the next one draws
 * the same again.  An element is dropped where r(q) < bar,
 *   bar = min(65535, floor(65536 p + 1/2)),
 * and is otherwise x * (65536 / (65536 - bar)), the factor rounded to fp32:
 * the mean is x's for every p.  The mask does not depend on type, alignment
 * or GPU.                                                                 */
typedef struct optim_dropout_hp {
    double p;      /* share to drop, in [0, 1)                             */
    uint64_t seed; /* of the run                                           */
    int64_t first; /* place of the first element, 0 .. 2^60                */
    uint32_t site; /* which dropout of the model                           */
} optim_dropout_hp;

/* out = drop(x)  (residual_dev NULL), or  out = residual + drop(x),  n
 * elements, 0 .. 2^48, of dtype F32, BF16 or F16, arrays aligned to their
 * element size; fp32 arithmetic, one rounding.  A dropped element counts as 0
 * whatever x holds there.  step_dev: device int32, or NULL for 0.  out_dev may
 * be x_dev or residual_dev itself, and must not overlap either otherwise.  The
 * gradient of x is the same call on the gradient of out, without residual; that
 * of residual is the gradient of out.                                     */
int optim_dropout(const void *x_dev, int32_t dtype, int64_t n,
                  const void *residual_dev, const optim_dropout_hp *hp,
                  const int32_t *step_dev, void *out_dev, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* OPTIM_DROPOUT_H */
