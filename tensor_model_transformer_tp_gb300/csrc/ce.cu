// Softmax cross entropy of a linear head (oases_ce.h).  bf16 runs on the
// tensor-core kernels of ce_tc.cu, fp32 on the CUDA-core GEMM with the same
// epilogues.
#include <cuda_runtime.h>

#include <algorithm>

#include "ce.cuh"
#include "gemm_f32.cuh"

namespace oases {
void api_begin();
oases_status api_end(cudaError_t e);

namespace {

constexpr int64_t PART_BYTES = 256ll << 20;   // fp32: partial maxima and sums of the forward
constexpr int64_t PIECE_BYTES = 256ll << 20;  // fp32: g of one piece of the backward

oases_status ce_shape(const oases_ce_desc* d, CeShape* s) {
  if (!d) return OASES_ERR_INVALID_ARG;
  if (d->dtype != OASES_F32 && d->dtype != OASES_BF16) return OASES_ERR_INVALID_ARG;
  if (d->rows < 0 || d->hidden <= 0 || d->vocab <= 0) return OASES_ERR_INVALID_ARG;
  if (d->dloss_per_row != 0 && d->dloss_per_row != 1) return OASES_ERR_INVALID_ARG;
  if (d->grad_dtype != OASES_F32 && d->grad_dtype != d->dtype) return OASES_ERR_INVALID_ARG;
  if (d->accumulate != 0 && d->accumulate != 1) return OASES_ERR_INVALID_ARG;
  if (d->accumulate && d->grad_dtype != OASES_F32) return OASES_ERR_INVALID_ARG;
  if (d->dtype == OASES_BF16 && d->hidden % 8 != 0) return OASES_ERR_UNSUPPORTED;
  if (std::max({d->rows, d->hidden, d->vocab}) > (d->dtype == OASES_F32 ? f32::MAX_DIM : 1 << 29))
    return OASES_ERR_UNSUPPORTED;  // 32-bit tile and TMA coordinates
  s->M = d->rows;
  s->H = d->hidden;
  s->V = d->vocab;
  s->t = static_cast<DType>(d->dtype);
  s->grad_t = static_cast<DType>(d->grad_dtype);
  s->per_row = d->dloss_per_row != 0;
  s->accumulate = d->accumulate != 0;
  s->ignore = d->ignore_index;
  const int64_t fit = PIECE_BYTES / (4 * std::max<int64_t>(1, s->M)) / 256 * 256;
  s->piece = (int)std::min<int64_t>(s->V, std::max<int64_t>(256, fit));
  s->ld = (s->piece + 7) / 8 * 8;
  return OASES_OK;
}

// fp32: one partial result per row and 64 columns; rows per pass of the forward.
int f32_slots(const CeShape& s) { return (s.V + f32::BN - 1) / f32::BN; }
int fwd_rows(const CeShape& s) {
  const int64_t fit = PART_BYTES / (8ll * f32_slots(s)) / 64 * 64;
  return (int)std::min<int64_t>(s.M, std::max<int64_t>(fit, 64));
}

struct Layout {
  size_t tc = 0, part = 0, at = 0, g = 0, scale = 0, total = 0;
};
Layout layout(const CeShape& s, bool backward) {
  Layout l;
  auto take = [&](size_t* at, size_t bytes) {
    *at = l.total;
    l.total += align256(bytes);
  };
  if (s.M == 0) return l;
  if (backward && s.per_row) take(&l.scale, 256);
  if (s.t == DType::BF16) {
    l.tc = l.total;  // the tensor-core path's own region
    l.total += backward ? ce_tc_bwd_bytes(s) : ce_tc_fwd_bytes(s);
    return l;
  }
  if (backward) {
    take(&l.g, (size_t)s.M * s.ld * 4);
  } else {
    take(&l.part, (size_t)fwd_rows(s) * f32_slots(s) * 8);
    take(&l.at, (size_t)fwd_rows(s) * 4);
  }
  return l;
}

__device__ __forceinline__ float block_max(float v, float* red) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < (int)blockDim.x / 32 ? red[lane] : -INFINITY;
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  __syncthreads();
  return v;
}

// fp32 forward: a row's 64 columns, four per thread of sixteen, to (r, s) as in
// ce_tc.cu: the maximum and the sum of e^(l - r).
struct StatF32 {
  static constexpr bool DUAL = false;
  float2* part;
  float* at;
  const int64_t* target;
  __device__ __forceinline__ void tile(int m, int n0, const float (&v)[4], int col, int M, int N) const {
    float r = -INFINITY, s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + col + i < N) r = fmaxf(r, v[i]);
#pragma unroll
    for (int o = 8; o; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
    const float ref = r == -INFINITY ? 0.f : r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + col + i < N) s += expf(v[i] - ref);
#pragma unroll
    for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (m >= M) return;
    if (col == 0) part[(int64_t)(n0 / f32::BN) * M + m] = make_float2(r, s);
    const int64_t d = target[m] - n0 - col;
    if (d >= 0 && d < 4 && target[m] < N) at[m] = d == 0 ? v[0] : d == 1 ? v[1] : d == 2 ? v[2] : v[3];
  }
};

// fp32 backward: g / s of a piece, (exp(l - lse) - [v == target]) r; rows
// without a loss are 0 whatever their logits are.
struct GradF32 {
  static constexpr bool DUAL = false;
  float* g;
  int64_t ld;
  CeRows rows;
  const float* lse;
  int v0;
  __device__ __forceinline__ void tile(int m, int n0, const float (&v)[4], int col, int M, int N) const {
    if (m >= M) return;
    const int64_t t = rows.target[m];
    const float r = row_factor(rows, t, m), l = lse[m];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + col + i;
      if (n >= N) {  // the row's padding
        if (n < ld) g[(int64_t)m * ld + n] = 0.f;
        continue;
      }
      const float p = expf(v[i] - l) - (t == v0 + n ? 1.f : 0.f);
      g[(int64_t)m * ld + n] = t == rows.ignore ? 0.f : p * r;
    }
  }
};

// The largest finite |dloss| of the rows that have a loss (CeRows::scale).
__global__ void __launch_bounds__(1024)
ce_scale_kernel(const float* dloss, const int64_t* target, int64_t ignore, int M, float* scale) {
  __shared__ float red[32];
  pdl_wait();
  pdl_trigger();
  float mx = 0.f;
  for (int m = threadIdx.x; m < M; m += blockDim.x)
    if (const float a = fabsf(dloss[m]); target[m] != ignore && a < INFINITY) mx = fmaxf(mx, a);
  mx = block_max(mx, red);
  if (threadIdx.x == 0) scale[0] = mx;
}

cudaError_t fwd(const CeShape& s, const void* x, const void* w, const int64_t* target, float* loss,
                float* lse, char* ws, cudaStream_t st) {
  const Layout l = layout(s, false);
  if (s.t == DType::BF16) return ce_tc_fwd(s, x, w, target, loss, lse, ws + l.tc, st);
  const int step = fwd_rows(s);
  for (int m0 = 0; m0 < s.M; m0 += step) {
    const int M = std::min(step, s.M - m0);
    const StatF32 e{reinterpret_cast<float2*>(ws + l.part), reinterpret_cast<float*>(ws + l.at),
                    target + m0};
    const f32::Args g{M, s.V, s.H, static_cast<const float*>(x) + (int64_t)m0 * s.H, s.H,
                      static_cast<const float*>(w), s.H};
    OASES_TRY((f32::launch<StatF32, true, true>(g, e, st)));
    OASES_TRY(ce_join(e.part, f32_slots(s), e.at, e.target, s, M, loss + m0, lse + m0, st));
  }
  return cudaSuccess;
}

cudaError_t bwd(const CeShape& s, const void* x, const void* w, const int64_t* target,
                const float* lse, const float* dloss, void* dx, void* dw, char* ws,
                cudaStream_t st) {
  const Layout l = layout(s, true);
  CeRows rows{target, dloss, dloss, s.per_row ? 1 : 0, s.V, s.ignore};
  if (s.per_row) {
    float* scale = reinterpret_cast<float*>(ws + l.scale);
    OASES_TRY(launch_pdl(ce_scale_kernel, dim3(1), dim3(1024), 0, st, dloss, target, s.ignore, s.M,
                         scale));
    rows.scale = scale;
  }
  if (s.t == DType::BF16) return ce_tc_bwd(s, x, w, rows, lse, dx, dw, ws + l.tc, st);
  float* g = reinterpret_cast<float*>(ws + l.g);
  for (int v0 = 0; v0 < s.V; v0 += s.piece) {
    const int n = std::min(s.piece, s.V - v0);
    const float* wp = static_cast<const float*>(w) + (int64_t)v0 * s.H;
    OASES_TRY((f32::launch<GradF32, true, true>(
        f32::Args{s.M, n, s.H, (const float*)x, s.H, wp, s.H},
        GradF32{g, s.ld, rows, lse, v0}, st)));
    const f32::Args args[3] = {{s.M, s.H, n, g, s.ld, wp, s.H, 0, 1},
                               {n, s.H, s.M, g, s.ld, (const float*)x, s.H, 0, 1},
                               {}};
    float* out_w = dw ? static_cast<float*>(dw) + (int64_t)v0 * s.H : nullptr;
    const f32::Out out[3] = {{(float*)dx, s.H, rows.scale, nullptr, nullptr, v0 > 0},
                             {out_w, s.H, rows.scale, nullptr, nullptr, s.accumulate},
                             {}};
    OASES_TRY(f32::launch_group(args, out, {true, false, false}, st));
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace oases

extern "C" size_t oases_ce_workspace_bytes(const oases_ce_desc* desc, int backward) {
  oases::CeShape s;
  if (oases::ce_shape(desc, &s) != OASES_OK) return 0;
  return oases::layout(s, backward != 0).total;
}

extern "C" oases_status oases_ce_fwd(const oases_ce_desc* desc, const void* x, const void* w,
                                     const int64_t* target, float* loss, float* lse,
                                     void* workspace, size_t ws_bytes, void* stream) {
  using namespace oases;
  api_begin();
  CeShape s;
  const oases_status v = ce_shape(desc, &s);
  if (v != OASES_OK) return v;
  if (s.M == 0) return OASES_OK;
  if (!x || !w || !target || !loss || !lse) return OASES_ERR_INVALID_ARG;
  if (misaligned({x, w, workspace}, 16) || misaligned({target}, 8) || misaligned({loss, lse}, 4))
    return OASES_ERR_INVALID_ARG;
  const size_t need = layout(s, false).total;
  if (need > 0 && (!workspace || ws_bytes < need)) return OASES_ERR_WORKSPACE;
  return api_end(fwd(s, x, w, target, loss, lse, static_cast<char*>(workspace),
                     static_cast<cudaStream_t>(stream)));
}

extern "C" oases_status oases_ce_bwd(const oases_ce_desc* desc, const void* x, const void* w,
                                     const int64_t* target, const float* lse, const float* dloss,
                                     void* dx, void* dw, void* workspace, size_t ws_bytes,
                                     void* stream) {
  using namespace oases;
  api_begin();
  CeShape s;
  const oases_status v = ce_shape(desc, &s);
  if (v != OASES_OK) return v;
  if (misaligned({x, w, dx, dw, workspace}, 16) || misaligned({target}, 8) ||
      misaligned({lse, dloss}, 4))
    return OASES_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.M == 0) {  // sums over no rows
    if (!dw || s.accumulate) return OASES_OK;
    return api_end(cudaMemsetAsync(dw, 0, (size_t)s.V * s.H * dtype_size(s.grad_t), st));
  }
  if (!x || !w || !target || !lse || !dloss) return OASES_ERR_INVALID_ARG;
  const size_t need = layout(s, true).total;
  if (need > 0 && (!workspace || ws_bytes < need)) return OASES_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  return api_end(bwd(s, x, w, target, lse, dloss, dx, dw, ws, st));
}
