/*
 * oases_ce.h — softmax cross entropy of a linear head over a large vocabulary,
 * with its gradient (liboases.so).
 *
 * The loss at the end of a stack, where oases_stack_step takes the gradient g
 * of its output y: for the rows x of y and the head's weights w,
 *   l[m, v] = sum_k x[m, k] w[v, k]
 *   lse[m]  = log sum_v exp l[m, v]
 *   loss[m] = lse[m] - l[m, target[m]]
 * and, for the gradient dloss of the losses,
 *   g[m, v] = (exp(l[m, v] - lse[m]) - [v == target[m]]) dloss[m]
 *   dx = g w,  dw = g^T x.
 * The pages (Oases, arXiv 2305.16121) name no loss; this is the textbook one.
 * The logits l are never kept: the forward reduces them, tile by tile of the
 * vocabulary, to lse and the target's logit; the backward computes them again
 * from lse, a piece of the vocabulary at a time, with g of one piece in the
 * workspace.
 *
 * Layout: row-major, contiguous: x, dx [rows, hidden]; w, dw [vocab, hidden];
 * target int64 [rows]; loss, lse, dloss fp32.  Conventions of memory, threads,
 * errors and determinism as in oases.h: the caller owns every buffer, the
 * device pointers of x, w, dx, dw and the workspace are 16-byte aligned (those
 * of target and of loss, lse, dloss need only their elements' alignment, so
 * shifted targets can be a slice), argument errors are returned before anything
 * is enqueued, calls are asynchronous on `stream` (one stream), identical
 * inputs give identical bits.
 *
 * Targets.  A row whose target is ignore_index has loss 0 and no gradient, also
 * where a dloss given for every row is infinite or NaN (its lse is written all
 * the same); its x counts in dw times 0, so an infinite or
 * NaN one makes dw NaN, as in any product.  A target outside [0, vocab) that is
 * not ignore_index is an error that only the device can see: that row's loss is
 * NaN, and so are its row of dx and all of dw.
 *
 * Precision.  Products accumulate in fp32.  loss and lse are fp32: lse = max + log
 * sum e^(l - max) is no less than any logit, so no loss is negative.  With bf16 the
 * logits are sums in the tensor cores' accumulator, which drops what is below its
 * last bit: loss and lse are 1e-7 of their size off at hidden 1024 and 8e-7 at hidden
 * 4096 in the root mean square.  g is rounded to dtype, the type of the operands of dx and dw,
 * after its rows' common factor has been taken out (the dloss of all rows, or the
 * largest finite |dloss|), which is multiplied to the fp32 sums.
 */
#ifndef OASES_CE_H
#define OASES_CE_H

#include <stddef.h>
#include <stdint.h>

#include "oases.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t ignore_index;
  int32_t dtype;         /* OASES_F32 or OASES_BF16: x, w and dx */
  int32_t rows;          /* tokens, >= 0 */
  int32_t hidden;        /* > 0; a multiple of 8 for bf16 */
  int32_t vocab;         /* > 0 */
  int32_t dloss_per_row; /* backward: 1: dloss is [rows]; 0: one value for every row */
  int32_t grad_dtype;    /* backward: dw as OASES_F32 or as dtype */
  int32_t accumulate;    /* backward: 1: dw += (grad_dtype OASES_F32 only), the
                            convention of oases.h; 0: dw is written */
} oases_ce_desc;

/* Bytes of workspace of the forward (backward = 0) or backward (1) call, 0 for
 * an invalid desc.  Its contents need not survive between calls. */
size_t oases_ce_workspace_bytes(const oases_ce_desc *desc, int backward);

/* loss, lse: fp32 [rows], written.
 * Errors: INVALID_ARG for a bad descriptor, a NULL or misaligned pointer;
 * UNSUPPORTED for a bf16 hidden that is no multiple of 8 and for rows, hidden or
 * vocab beyond 2^29 (fp32: 2097120); WORKSPACE for a
 * workspace that is NULL or too small. */
oases_status oases_ce_fwd(const oases_ce_desc *desc, const void *x, const void *w,
                          const int64_t *target, float *loss, float *lse, void *workspace,
                          size_t ws_bytes, void *stream);

/* dx and dw from the forward's lse.  Either may be NULL (left out); they
 * overlap no input.  Errors as oases_ce_fwd. */
oases_status oases_ce_bwd(const oases_ce_desc *desc, const void *x, const void *w,
                          const int64_t *target, const float *lse, const float *dloss, void *dx,
                          void *dw, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* OASES_CE_H */
