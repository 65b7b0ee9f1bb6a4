/*
 * oases_qknorm.h — norms of queries and keys per head with the position rotation
 * in the same pass, forward and backward (liboases.so).
 *
 * What stands between the column-parallel QKV projection F_i and its attention
 * (Oases, arXiv 2305.16121, §IV-A) where heads are normalised and positions enter
 * by rotation; the pages name neither, the formulas are the textbook ones.  For
 * every token and head, with x its D = head_dim values and w a weight of D values:
 *   y = R_p (w * x * r),  r = 1 / sqrt(mean(x^2) + eps)
 * where R_p turns the pairs (a, b) among the first `rot` values by the angles of
 * the token's position p, a' = a cos - b sin, b' = a sin + b cos; pair c is the
 * values (c, c + rot / 2), or (2c, 2c + 1) where interleaved, with cos and sin at
 * [p, c] of the caller's tables.  Backward, g = R_p^T dy:
 *   dw = sum over tokens and heads of g * x * r
 *   dx = r (g * w - x r mean(g * w * x r)).
 * Queries and keys have a weight each; the keys may be left out (kv_heads = 0), as
 * for two sequences of different lengths, and the rotation (rot = 0).
 *
 * Layout: q, q_out, dq_out, dq [batch, seq, heads, head_dim], k ... with kv_heads,
 * strides as in oases_attn.h; cos, sin fp32 [positions_len, rot / 2], contiguous;
 * positions int64, [batch, seq] or one [seq] for every sequence, or NULL: token t is
 * at position t.  A position outside [0, positions_len) is an error that only the
 * device can see: the rotated values of its token are NaN, and what follows from them.
 * Conventions of memory, threads, errors and determinism as in oases.h; pointers of
 * the four-dimensional tensors, the weights, the gradients of the weights and the workspace are 16-byte
 * aligned, those of the tables and positions their elements'.
 * Statistics and sums are fp32; y, dx and the weights' gradients are rounded once.
 */
#ifndef OASES_QKNORM_H
#define OASES_QKNORM_H

#include <stddef.h>
#include <stdint.h>

#include "oases_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t dtype;            /* OASES_F32 or OASES_BF16 */
  int32_t batch, seq;       /* >= 0 */
  int32_t heads;            /* >= 0 */
  int32_t kv_heads;         /* >= 0 */
  int32_t head_dim;         /* a multiple of 8, 8 .. 256 */
  int32_t rot;              /* even, 0 .. head_dim */
  int32_t interleaved;      /* 1: pairs (2c, 2c + 1) */
  int32_t positions_len;    /* rows of cos and sin */
  int32_t positions_shared; /* 1: positions is [seq] for every sequence */
  int32_t grad_dtype;       /* backward: the weights' gradients as OASES_F32 or as dtype */
  int32_t accumulate;       /* backward: 1: they are added to (OASES_F32 only) */
  float eps;                /* > 0 */
  oases_strides q, k, q_out, k_out; /* x and y; backward: q_out, k_out those of dy */
  oases_strides dq, dk;             /* backward only: dx */
} oases_qknorm_desc;

/* Bytes of workspace of the backward call on the current device (the forward needs
 * none); 0 for an invalid desc. */
size_t oases_qknorm_workspace_bytes(const oases_qknorm_desc *desc);

/* q_out and k_out, written (q_out may be q and k_out k, with the same strides).
 * q_weight, k_weight: [head_dim], or NULL (1).
 * Errors: INVALID_ARG for a bad descriptor, a NULL or misaligned pointer or stride;
 * UNSUPPORTED for a head_dim beyond the rule above and for more than 2^29 tokens
 * or heads. */
oases_status oases_qknorm_fwd(const oases_qknorm_desc *desc, const void *q, const void *k,
                              const float *cos, const float *sin, const int64_t *positions,
                              const void *q_weight, const void *k_weight, void *q_out, void *k_out,
                              void *stream);

/* dq, dk (gradients of q and k as given to the forward) and the weights' gradients,
 * any of which may be NULL (left out); dq may be dq_out and dk dk_out, with the same
 * strides.  Errors as oases_qknorm_fwd, and WORKSPACE. */
oases_status oases_qknorm_bwd(const oases_qknorm_desc *desc, const void *q, const void *k,
                              const void *dq_out, const void *dk_out, const float *cos,
                              const float *sin, const int64_t *positions, const void *q_weight,
                              const void *k_weight, void *dq, void *dk, void *dq_weight,
                              void *dk_weight, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* OASES_QKNORM_H */
