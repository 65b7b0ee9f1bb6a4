// Cross entropy of the linear head: shapes and row factors shared by the host
// path (ce.cu) and the tensor-core kernels (ce_tc.cu).
#pragma once
#include <math_constants.h>

#include "common.cuh"
#include "oases_ce.h"

namespace oases {

struct CeShape {
  int M, H, V;
  DType t, grad_t;
  bool per_row, accumulate;
  int64_t ignore;
  int piece;   // fp32: columns of the vocabulary per piece of the backward
  int64_t ld;  // leading dimension of a piece's buffer
};

// g = s r (softmax - onehot): s one factor for all rows, r one per row.  s is
// the dloss given for all rows, or the largest finite |dloss| of the rows that
// have a loss, so r is at most 1 in magnitude, and exactly 1 where the rows share one
// dloss: the products then see entries of g / s such as the target's, close to
// -1, that do not depend on how dloss itself rounds to the storage type.  A dloss
// given for all rows that is infinite or NaN (the mean over no rows: 1 / 0) is r of
// the rows with a loss instead, and s counts as 1 (product_factor): rows without a
// loss keep their 0.
struct CeRows {
  const int64_t* target;
  const float* dloss;
  const float* scale;  // s
  int per_row, V;
  int64_t ignore;
};
__device__ __forceinline__ float row_factor(const CeRows& c, int64_t t, int m) {
  if (t == c.ignore) return 0.f;
  if (t < 0 || t >= c.V) return CUDART_NAN_F;
  if (!c.per_row) {
    const float d = *c.dloss;
    return fabsf(d) < INFINITY ? 1.f : d;
  }
  const float d = c.dloss[m], s = *c.scale;
  return s == 0.f ? d : d / s;  // s == 0: d is 0, infinite or NaN
}
__device__ __forceinline__ float row_loss(int64_t t, int64_t ignore, int V, float lse, float at) {
  return t == ignore ? 0.f : t < 0 || t >= V ? CUDART_NAN_F : lse - at;
}

// bf16, tensor cores.
// Forward: loss and lse of every row; ws as ce_tc_fwd_bytes.
size_t ce_tc_fwd_bytes(const CeShape& s);
cudaError_t ce_tc_fwd(const CeShape& s, const void* x, const void* w, const int64_t* target,
                      float* loss, float* lse, char* ws, cudaStream_t st);
// Backward without the row scale (rows.scale is given): dx, dw of all pieces.
size_t ce_tc_bwd_bytes(const CeShape& s);
cudaError_t ce_tc_bwd(const CeShape& s, const void* x, const void* w, const CeRows& rows,
                      const float* lse, void* dx, void* dw, char* ws, cudaStream_t st);
// Joins `slots` partial results (r, s) per row, part [slots][M], to lse and loss.
cudaError_t ce_join(const float2* part, int slots, const float* at, const int64_t* target,
                    const CeShape& s, int M, float* loss, float* lse, cudaStream_t st);
int ce_read_and_clear_error();

}  // namespace oases
