/*
 * oases_glu.h — gated feed-forward block, forward and backward (liboases.so).
 *
 * The feed-forward segment of a transformer layer in its gated form, beside
 * the W1 -> GeLU -> W2 form of oases.h:
 *   a = x Wg^T + bg,  b = x Wu^T + bu      [rows, ffn]
 *   h = act(a) * b
 *   y = h W2^T + b2 (+ resid)              [rows, hidden]
 * act is SiLU, a / (1 + e^-a), or the exact GeLU, a Phi(a).  The pages (Oases,
 * arXiv 2305.16121, §IV-A) give the column-parallel / row-parallel pair only
 * as F_i, F_j; the gated form is such a pair: shard k of w owns rows
 * [k ffn/w, (k+1) ffn/w) of Wg and of Wu and the same columns of W2, and the
 * sum over the shards is the contraction over ffn, so one weight buffer and
 * one call serve every w.
 *
 * Layout: row-major, contiguous.  x, y, resid, dy, dx [rows, hidden];
 * w1 [2 ffn, hidden] with rows [Wg | Wu]; b1 [2 ffn] = [bg | bu];
 * w2 [hidden, ffn]; b2 [hidden].  b1 and b2 may each be NULL (no bias).
 * Conventions of memory, threads, errors and determinism as in oases.h: the
 * caller owns every buffer, device pointers are 16-byte aligned, argument
 * errors are returned before anything is enqueued, calls are asynchronous on
 * `stream` (one stream), identical inputs give identical bits.
 */
#ifndef OASES_GLU_H
#define OASES_GLU_H

#include <stddef.h>
#include <stdint.h>

#include "oases.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { OASES_ACT_SILU = 0, OASES_ACT_GELU = 1 } oases_act;

/* What the forward keeps for the backward, beside x.
 * NONE:  nothing; the backward computes a and b again (the recomputation of
 *        Oases §IV, Fig. 4d: the column-parallel part only, never y).
 * PRE:   [a | b] in the storage type: [rows, 2 ffn], contiguous.  In bf16 the
 *        backward is then at other a and b than the forward's h was: dx, dw1 and dw2
 *        are 0.0035 of their size off, where NONE gives 0.0024 and the outputs' own
 *        rounding 0.0017.
 * MXFP8: a and b in 8 bits, half the bytes of PRE in bf16 (plus 1/32): two MX
 *        operands (oases_mx.h: E4M3 codes, one UE8M0 scale per 32 consecutive
 *        columns), gate first:
 *          codes  [2][rows][ldq] bytes, ldq = ffn rounded up to 16,
 *          scales at the next multiple of 256 bytes,
 *                 [2][oases_mx_scale_bytes(rows, ffn)] bytes.
 *        They are quantised from the fp32 accumulators; the forward's own h and
 *        y use the unquantised values, the backward uses the kept values
 *        throughout.  dtype BF16 only. */
typedef enum {
  OASES_GLU_KEEP_NONE = 0,
  OASES_GLU_KEEP_PRE = 1,
  OASES_GLU_KEEP_MXFP8 = 2
} oases_glu_keep;

typedef struct {
  int32_t dtype;       /* OASES_F32 or OASES_BF16: x, y, resid, dy and the weights */
  int32_t rows;        /* tokens, >= 0 */
  int32_t hidden;      /* > 0; a multiple of 8 for bf16 */
  int32_t ffn;         /* > 0; a multiple of 8 for bf16 */
  int32_t act;         /* oases_act */
  int32_t keep;        /* oases_glu_keep */
  int32_t dx_dtype;    /* backward: dx as dtype, or OASES_F32 (the du that
                          oases_debug_layer_norm_bwd takes) */
  int32_t grad_dtype;  /* backward: weight gradients as OASES_F32 or as dtype */
  int32_t accumulate;  /* backward: 1: gradients += (grad_dtype OASES_F32 only),
                          the convention of oases.h; 0: gradients are written */
} oases_glu_desc;

typedef struct {
  const void *w1, *b1, *w2, *b2;
} oases_glu_weights;

/* Gradients, shapes as the weights, type grad_dtype.  A NULL pointer leaves
 * that gradient out. */
typedef struct {
  void *w1, *b1, *w2, *b2;
} oases_glu_grads;

/* Bytes of the kept activations (0 for KEEP_NONE and for an invalid desc). */
size_t oases_glu_saved_bytes(const oases_glu_desc *desc);
/* Bytes of workspace of the forward (backward = 0) or backward (1) call; 0 for
 * an invalid desc (and where none is needed).  Its contents need not survive
 * between calls. */
size_t oases_glu_workspace_bytes(const oases_glu_desc *desc, int backward);

/* y = the block of x.  resid: [rows, hidden] added to y, or NULL; y may be
 * resid itself, and overlaps no other input.  saved: oases_glu_saved_bytes()
 * bytes, written (NULL for KEEP_NONE).
 * Errors: INVALID_ARG for a bad descriptor, a NULL or misaligned pointer;
 * UNSUPPORTED for a bf16 hidden or ffn that is no multiple of 8 and for
 * KEEP_MXFP8 with dtype F32, and for rows, hidden or ffn beyond 2^29 (fp32:
 * 2097120); WORKSPACE for a workspace that is NULL or too small. */
oases_status oases_glu_fwd(const oases_glu_desc *desc, const oases_glu_weights *wts, const void *x,
                           const void *resid, void *y, void *saved, void *workspace,
                           size_t ws_bytes, void *stream);

/* Backward of oases_glu_fwd for the output gradient dy: with dh = dy W2,
 *   da = dh b act'(a), db = dh act(a), dx = da Wg + db Wu,
 *   dw1 = [da | db]^T x, db1 = colsum [da | db], dw2 = dy^T h, db2 = colsum dy.
 * (resid's gradient is dy.)  x and saved as given to and written by the
 * forward; a and b are the kept values, or with KEEP_NONE fp32 sums formed again.
 * da, db and h are rounded to the storage type between the products, which
 * accumulate in fp32; db1 sums the rounded da and db.  dx may be NULL (left out); it overlaps no input.
 * Errors as oases_glu_fwd, and INVALID_ARG for grads->b1 / b2 set where the
 * bias is NULL. */
oases_status oases_glu_bwd(const oases_glu_desc *desc, const oases_glu_weights *wts, const void *x,
                           const void *dy, const void *saved, void *dx,
                           const oases_glu_grads *grads, void *workspace, size_t ws_bytes,
                           void *stream);

#ifdef __cplusplus
}
#endif
#endif /* OASES_GLU_H */
