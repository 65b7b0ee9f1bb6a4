// Gated feed-forward block: shapes shared by the host path (glu.cu) and the
// tensor-core kernels (glu_tc.cu).
#pragma once
#include "gemm_core.cuh"
#include "oases_glu.h"

namespace oases {

struct GluShape {
  int M, H, F;
  DType t, dx_t, grad_t;
  int act, keep;
  bool accumulate;
  int64_t ldq;  // leading dimension of the 8-bit codes
  // Leading dimensions in the workspace of h and of [da | db]: bf16 rows start on 128-byte lines.  (A row that does not makes every 128-byte
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

// Of 32 columns of one row: wa = da = d b act'(a), wb = db = d act(a), wh = h =
// act(a) b, rounded to bf16 pairs.
template <int ACT>
__device__ __forceinline__ void gradients(const float (&a)[32], const float (&b)[32],
                                          const float (&d)[32], uint32_t (&wa)[16], uint32_t (&wb)[16],
                                          uint32_t (&wh)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float f0, f1, g0, g1;
    act_both_fast(ACT, a[2 * i], f0, g0);
    act_both_fast(ACT, a[2 * i + 1], f1, g1);
    const float d0 = d[2 * i], d1 = d[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
    wa[i] = core::pack2(d0 * b0 * g0, d1 * b1 * g1);
    wb[i] = core::pack2(d0 * f0, d1 * f1);
    wh[i] = core::pack2(f0 * b0, f1 * b1);
  }
}
// 16-byte unit u of a lane's 64-byte row in a 2 KB staging buffer (64-byte swizzle).
__device__ __forceinline__ uint4* row_unit(uint8_t* buf, int lane, int u) {
  return reinterpret_cast<uint4*>(buf + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4));
}
__device__ __forceinline__ void put_row(uint8_t* buf, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    *row_unit(buf, lane, u) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
}
// v[i] += src[i] for i < left, left a multiple of 8
__device__ __forceinline__ void add_bias(const __nv_bfloat16* src, int left, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    if (i < left) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + i));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = core::unpack2(w[k]);
        add2_inplace(v[i + 2 * k], v[i + 2 * k + 1], f.x, f.y);
      }
    }
}
// Maps of pre's (or dpre's) two halves, boxes of 32 rows x `box` columns.
inline bool halves(CUtensorMap* a, CUtensorMap* b, const void* pre, int64_t ld, const GluShape& s,
                   int box) {
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(pre);
  return core::tensor_map(a, q, false, s.F, s.M, ld, box, 32) &&
         core::tensor_map(b, q + s.F, false, s.F, s.M, ld, box, 32);
}

// bf16, tensor cores.
// [a | b] = x w1^T + b1 of every row, and from the fp32 accumulators
//   h = act(a) b
//   pre = [a | b]     (pre given), bf16 [M, 2F]
//   the 8-bit form    (kept8 given, laid out as oases_glu_keep MXFP8)
cudaError_t glu_project_tc(const GluShape& s, const void* x, const void* w1, const void* b1,
                           void* h, void* pre, void* kept8, cudaStream_t st);
// dh = dy w2, and from it dpre = [da | db] [M, 2F] and h [M, F] at the a, b of
// pre (bf16 [M, 2F]) or kept8.
cudaError_t glu_grad_tc(const GluShape& s, const void* dy, const void* w2, const void* pre,
                        const void* kept8, void* dpre, void* h, cudaStream_t st);
// The same at a, b = x w1^T + b1, computed again (glu_again.cu).
cudaError_t glu_grad_again_tc(const GluShape& s, const void* x, const void* dy, const void* w1,
                              const void* b1, const void* w2, void* dpre, void* h, cudaStream_t st);
int glu_again_read_and_clear_error();
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
                            void* h, void* pre, void* kept8, cudaStream_t st);
cudaError_t glu_down_few(const GluShape& s, const void* h, const void* w2, const void* b2,
                         const void* resid, void* y, cudaStream_t st);
int glu_few_read_and_clear_error();

}  // namespace oases
