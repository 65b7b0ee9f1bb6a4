/*
 * oases_attn.h — softmax attention over keys of another length, with a learned
 * relative position bias, forward and backward (liboases.so).
 *
 * Beside the block's attention (oases.h: one packed sequence, as many key heads
 * as query heads, keys of the queries' own length), for every sequence b and
 * query head h, with key head g = h / (heads / kv_heads):
 *   s[i, j] = scale q[b, i, h] . k[b, j, g] + bias[bucket(j - p_i), h],  p_i = q_start[b] + i
 *   key j is visible where j < kv_lens[b] and, if causal, j <= p_i
 *   lse[b, h, i] = log sum_visible e^s,  o[b, i, h] = sum_visible e^(s - lse) v[b, j, g]
 * and, for the gradient d_o of o,
 *   delta = rowsum(d_o * o),  dP = d_o v^T,  dS = e^(s - lse) (dP - delta)
 *   dq = scale dS k,  dk = scale dS^T q,  dv = P^T d_o  (dk, dv summed over the query
 *   heads of a key head),  dbias[u, h] = sum of dS[i, j] with bucket(j - p_i) = u.
 * The pages (Oases, arXiv 2305.16121, §IV-A) name the attention layer only as a
 * column-parallel operator F_i whose shards own heads; heads are independent
 * here too, so a shard is a slice of the heads.  The scores are never stored.
 *
 * A query that sees no key (kv_lens[b] = 0, or a bias of -infinity on all of
 * them) has o = 0 and lse = -infinity, and gives no gradient.  Nor does one whose
 * lse lies below -2^20 (a finite bias that hides all of its keys) or above 2^24: there
 * an fp32 lse no longer tells their weights.  One that sees a single key has dS = 0.
 * What stands in k and v at and behind kv_lens[b], and causal at and behind p_q_len (keys
 * that no query of the sequence sees), is not used, whatever it holds; dk and dv are 0
 * there.  Nearer ones are to be finite, also where a query does not see them: its weight 0
 * times an infinity is a NaN; and so is d_o of the queries without keys.  kv_lens values
 * outside [0, k_len] are taken as the nearest in it, q_start values within 2^28 of 0.
 *
 * Buckets.  n = j - p_i, the key's position relative to the query's.  With
 * bidirectional set, N = buckets / 2 buckets serve each sign (those of n > 0 are
 * the table's upper half); else N = buckets serve n <= 0, and n > 0 is taken as 0.
 * For a = |n| and E = N / 2 (rounded down):
 *   bucket = a                                                            a < E
 *   bucket = min(N - 1, E + floor((N - E) log(a / E) / log(max_distance / E)))  else
 * The floor is that of the real number, also where it is whole (not of a rounded logarithm).
 *
 * Layout.  q, o, d_o, dq [batch, q_len, heads, head_dim] and k, v, dk, dv
 * [batch, k_len, kv_heads, head_dim], a head's values side by side and the other
 * strides free, so that packed projections can be read and written in place; lse
 * fp32 [batch, heads, q_len]; bias and dbias [buckets, heads].  Conventions of
 * memory, threads, errors and determinism as in oases.h: the caller owns every
 * buffer, the pointers of q, k, v, o, d_o, dq, dk, dv and the workspace are
 * 16-byte aligned (the others' their elements'), argument errors are returned
 * before anything is enqueued, calls are asynchronous on `stream` (one stream),
 * identical inputs give identical bits.
 *
 * Precision.  Scores, softmax statistics and all sums are fp32.  In bf16 the
 * weights e^(s - m) and dS are rounded to bf16 as operands of the products with
 * v, d_o, k and q; delta is formed from the rounded o, but as sum P dP where a query
 * sees 128 keys or less, and for dk, dv and dbias wherever there is a bias.  fp32 rounds nothing but
 * fp32 sums.
 */
#ifndef OASES_ATTN_H
#define OASES_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "oases.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Elements between neighbours in each dimension (of one element or less: not
 * read).  Multiples of 16 bytes, positive, at most 2^36. */
typedef struct {
  int64_t batch, token, head;
} oases_strides;

typedef struct {
  int32_t dtype;          /* OASES_F32 or OASES_BF16: all tensors but lse and dbias */
  int32_t batch;          /* sequences, >= 0 */
  int32_t q_len, k_len;   /* >= 0 */
  int32_t heads;          /* > 0, a multiple of kv_heads */
  int32_t kv_heads;       /* > 0 */
  int32_t head_dim;       /* a multiple of 8, 8 .. 128 */
  int32_t causal;         /* 1: key j is visible where j <= p_i */
  int32_t q_start;        /* p_0 of every sequence where no q_start array is given, >= 0 */
  int32_t buckets;        /* 0: no bias; else 2 .. 128, at least 4 and even where bidirectional */
  int32_t max_distance;   /* > E, at most 65536 (read with a bias only) */
  int32_t bidirectional;  /* (read with a bias only) */
  int32_t grad_dtype;     /* backward: dbias as OASES_F32 or as dtype */
  int32_t accumulate;     /* backward: 1: dbias += (grad_dtype OASES_F32 only), the
                             convention of oases.h; 0: dbias is written */
  float scale;            /* > 0, finite */
  oases_strides q, k, v, o;
  oases_strides d_o, dq, dk, dv; /* backward only */
} oases_attn_desc;

/* Bytes of workspace of the forward (backward = 0) or backward (1) call on the
 * current device, 0 for an invalid desc (and where none is needed).  Its contents
 * need not survive between calls. */
size_t oases_attn_workspace_bytes(const oases_attn_desc *desc, int backward);

/* o and lse, written.  kv_lens, q_start: device int32 [batch], or NULL (k_len, and
 * desc->q_start).  bias: NULL iff desc->buckets == 0.
 * Errors: INVALID_ARG for a bad descriptor, a NULL or misaligned pointer or stride;
 * UNSUPPORTED for a head_dim beyond the rule above, more than 128 buckets,
 * a max_distance beyond 65536, lengths beyond 2^24, and more than 2^24 heads or
 * heads times sequences; WORKSPACE for a workspace that is NULL or too small. */
oases_status oases_attn_fwd(const oases_attn_desc *desc, const void *q, const void *k,
                            const void *v, const int32_t *kv_lens, const int32_t *q_start,
                            const void *bias, void *o, float *lse, void *workspace,
                            size_t ws_bytes, void *stream);

/* dq, dk, dv and dbias from the forward's o and lse.  dq, dk, dv are written whole;
 * dbias may be NULL (left out).  They overlap no input.  Errors as oases_attn_fwd,
 * and INVALID_ARG for a dbias where there is no bias. */
oases_status oases_attn_bwd(const oases_attn_desc *desc, const void *q, const void *k,
                            const void *v, const int32_t *kv_lens, const int32_t *q_start,
                            const void *bias, const void *o, const float *lse, const void *d_o,
                            void *dq, void *dk, void *dv, void *dbias, void *workspace,
                            size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* OASES_ATTN_H */
