// Gated feed-forward block: shapes shared by the host path (glu.cu) and the
// tensor-core kernels (glu_tc.cu).
#pragma once
#include "common.cuh"
#include "oases_glu.h"

namespace oases {

inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct GluShape {
  int M, H, F;
  DType t, dx_t, grad_t;
  int act, keep;
  bool accumulate;
  int64_t ldq;  // leading dimension of the 8-bit codes
};

// Kept activations (oases_glu_keep): where the scales of the 8-bit form start.
inline size_t saved_scale_offset(const GluShape& s) { return align256(2 * (size_t)s.M * s.ldq); }

// bf16, tensor cores.
// [a | b] = x w1^T + b1 of every row, and from the fp32 accumulators
//   h = act(a) b      (h given)
//   pre = [a | b]     (pre given), bf16 [M, 2F]
//   the 8-bit form    (kept8 given, laid out as oases_glu_keep MXFP8)
cudaError_t glu_project_tc(const GluShape& s, const void* x, const void* w1, const void* b1,
                           void* h, void* pre, void* kept8, cudaStream_t st);
// dh = dy w2, and from it dpre = [da | db] [M, 2F] and h [M, F] at the a, b of
// pre (bf16 [M, 2F]) or kept8.
cudaError_t glu_grad_tc(const GluShape& s, const void* dy, const void* w2, const void* pre,
                        const void* kept8, void* dpre, void* h, cudaStream_t st);
// y = h w2^T + b2 (+ resid)
cudaError_t glu_down_tc(const GluShape& s, const void* h, const void* w2, const void* b2,
                        const void* resid, void* y, cudaStream_t st);
int glu_read_and_clear_error();

}  // namespace oases
