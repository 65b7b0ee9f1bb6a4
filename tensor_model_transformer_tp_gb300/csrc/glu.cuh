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
  // Leading dimensions in the workspace of h, and of [a | b] and [da | db]: bf16
  // rows start on 128-byte lines.  (A row that does not makes every 128-byte
  // operand row of a TMA box two lines: 1531 x 2048 x 5464 took 37 us against 29
  // with the rows of both operands on lines.)
  int64_t ldh, ldp;
};

// Kept activations (oases_glu_keep): where the scales of the 8-bit form start.
inline size_t saved_scale_offset(const GluShape& s) { return align256(2 * (size_t)s.M * s.ldq); }

// SiLU and its derivative: s = 1 / (1 + e^-a), act = a s,
// act' = s (1 + a (1 - s)) = s + act (1 - s).  Hardware base-2 exponential and
// reciprocal (relative error ~2^-22); an exponential that overflows gives
// s = 0, one that underflows s = 1.
__device__ __forceinline__ void silu(float a, float& f, float& s) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * a));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  f = a * s;
}
__device__ __forceinline__ void act_both_fast(int act, float a, float& f, float& df) {
  if (act == OASES_ACT_SILU) {
    float s;
    silu(a, f, s);
    df = fmaf(f, 1.0f - s, s);
  } else {
    float cdf, pdf;
    gelu_cdf_pdf(a, cdf, pdf);
    f = a * cdf;
    df = fmaf(a, pdf, cdf);
  }
}
__device__ __forceinline__ float act_fast(int act, float a) {
  if (act != OASES_ACT_SILU) return gelu_f(a);
  float f, s;
  silu(a, f, s);
  return f;
}

// bf16, tensor cores.
// [a | b] = x w1^T + b1 of every row, and from the fp32 accumulators
//   h = act(a) b      (h given)
//   pre = [a | b]     (pre given), bf16 [M, 2F], leading dimension ld_pre
//   the 8-bit form    (kept8 given, laid out as oases_glu_keep MXFP8)
cudaError_t glu_project_tc(const GluShape& s, const void* x, const void* w1, const void* b1,
                           void* h, void* pre, int64_t ld_pre, void* kept8, cudaStream_t st);
// dh = dy w2, and from it dpre = [da | db] [M, 2F] and h [M, F] at the a, b of
// pre (bf16 [M, 2F], leading dimension ld_pre) or kept8.
cudaError_t glu_grad_tc(const GluShape& s, const void* dy, const void* w2, const void* pre,
                        int64_t ld_pre, const void* kept8, void* dpre, void* h, cudaStream_t st);
// dw2 (+)= dy^T h, dw1 (+)= dpre^T x, dx = dpre w1, each where it is given; ws
// as glu_grads_tc_bytes.
size_t glu_grads_tc_bytes(const GluShape& s);
cudaError_t glu_grads_tc(const GluShape& s, const void* x, const void* dy, const void* w1,
                         const void* dpre, const void* h, void* dx, void* dw1, void* dw2, char* ws,
                         cudaStream_t st);
// y = h w2^T + b2 (+ resid); ws as glu_down_tc_bytes
size_t glu_down_tc_bytes(const GluShape& s);
cudaError_t glu_down_tc(const GluShape& s, const void* h, const void* w2, const void* b2,
                        const void* resid, void* y, char* ws, cudaStream_t st);
int glu_read_and_clear_error();
// The forward's two products for at most GLU_FEW_ROWS rows (glu_few.cu).
constexpr int GLU_FEW_ROWS = 128;
cudaError_t glu_project_few(const GluShape& s, const void* x, const void* w1, const void* b1,
                            void* h, void* pre, int64_t ld_pre, void* kept8, cudaStream_t st);
cudaError_t glu_down_few(const GluShape& s, const void* h, const void* w2, const void* b2,
                         const void* resid, void* y, cudaStream_t st);
int glu_few_read_and_clear_error();

}  // namespace oases
