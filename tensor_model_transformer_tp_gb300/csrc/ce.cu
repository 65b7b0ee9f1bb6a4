// Softmax cross entropy of a linear head (oases_ce.h).  bf16 runs on the
// tensor-core kernels of ce_tc.cu.  fp32, on the CUDA-core GEMM, goes through
// the vocabulary in pieces: logits of a piece l = x W_piece^T, reduced to a
// running maximum and sum of every row, and, in the backward, turned into g of
// the piece, from which dx += g W_piece and dW_piece = g^T x.
#include <cuda_runtime.h>

#include <algorithm>

#include "ce.cuh"

namespace oases {
void api_begin();
void api_set_error(const char* what);
oases_status api_end(cudaError_t e);

namespace {

constexpr int64_t PIECE_BYTES = 256ll << 20;  // logits of one piece in the workspace

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

oases_status ce_shape(const oases_ce_desc* d, CeShape* s) {
  if (!d) return OASES_ERR_INVALID_ARG;
  if (d->dtype != OASES_F32 && d->dtype != OASES_BF16) return OASES_ERR_INVALID_ARG;
  if (d->rows < 0 || d->hidden <= 0 || d->vocab <= 0) return OASES_ERR_INVALID_ARG;
  if (d->dloss_per_row != 0 && d->dloss_per_row != 1) return OASES_ERR_INVALID_ARG;
  if (d->grad_dtype != OASES_F32 && d->grad_dtype != d->dtype) return OASES_ERR_INVALID_ARG;
  if (d->accumulate != 0 && d->accumulate != 1) return OASES_ERR_INVALID_ARG;
  if (d->accumulate && d->grad_dtype != OASES_F32) return OASES_ERR_INVALID_ARG;
  if (d->dtype == OASES_BF16 && d->hidden % 8 != 0) return OASES_ERR_UNSUPPORTED;
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

struct Layout {
  size_t logits = 0, run = 0, scale = 0, total = 0;
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
    l.logits = l.total;  // the tensor-core path's own region
    l.total += backward ? ce_tc_bwd_bytes(s) : ce_tc_fwd_bytes(s);
    return l;
  }
  take(&l.logits, (size_t)s.M * s.ld * 4);
  take(&l.run, backward ? (size_t)s.piece * s.H * 4 : (size_t)s.M * 12);
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
__device__ __forceinline__ float block_sum(float v, float* red) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < (int)blockDim.x / 32 ? red[lane] : 0.f;
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();
  return v;
}

// The reference point of exponentials of values with maximum m: m, or 0 where
// every value is -inf (exp(-inf - 0) = 0).
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

// One row of a piece [v0, v0 + n): joins its maximum and sum with the row's
// running ones (run[0], run[1] of [3][M]) and notes the target's logit
// (run[2]); the last piece writes lse and loss.
__global__ void __launch_bounds__(256)
ce_stat_kernel(const float* logits, int64_t ld, int n, int v0, bool first, bool last, float* run,
               const int64_t* target, int64_t ignore, int V, float* loss, float* lse, int M) {
  __shared__ float red[8];
  pdl_wait();
  pdl_trigger();
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    const float* row = logits + (int64_t)m * ld;
    float mx = -INFINITY;
    for (int i = threadIdx.x; i < n; i += blockDim.x) mx = fmaxf(mx, row[i]);
    mx = block_max(mx, red);
    const float old = first ? -INFINITY : run[m], top = fmaxf(old, mx), ref = ref_of(top);
    float s = 0.f;
    for (int i = threadIdx.x; i < n; i += blockDim.x) s += expf(row[i] - ref);
    s = block_sum(s, red);
    if (threadIdx.x == 0) {
      if (!first) s += run[M + m] * expf(old - ref);
      const int64_t t = target[m];
      float at = first ? 0.f : run[2 * M + m];
      if (t >= v0 && t < v0 + n) at = row[t - v0];
      if (last) {
        const float l = ref + logf(s);
        lse[m] = l;
        loss[m] = row_loss(t, ignore, V, l, at);
      } else {
        run[m] = top;
        run[M + m] = s;
        run[2 * M + m] = at;
      }
    }
  }
}

// The largest |dloss| of the rows that have a loss (CeRows::scale).
__global__ void __launch_bounds__(1024)
ce_scale_kernel(const float* dloss, const int64_t* target, int64_t ignore, int M, float* scale) {
  __shared__ float red[32];
  pdl_wait();
  pdl_trigger();
  float mx = 0.f;
  for (int m = threadIdx.x; m < M; m += blockDim.x)
    if (target[m] != ignore) mx = fmaxf(mx, fabsf(dloss[m]));
  mx = block_max(mx, red);
  if (threadIdx.x == 0) scale[0] = mx;
}

// g / s of a piece over its logits: (exp(l - lse) - [v == target]) r; rows
// without a loss are 0 whatever their logits are.
__global__ void __launch_bounds__(256)
ce_grad_kernel(float* logits, int64_t ld, int n, int v0, const float* lse, const CeRows rows, int M) {
  pdl_wait();
  pdl_trigger();
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    const int64_t t = rows.target[m];
    const float r = row_factor(rows, t, m), l = lse[m];
    float* row = logits + (int64_t)m * ld;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const float p = expf(row[i] - l) - (t == v0 + i ? 1.f : 0.f);
      row[i] = t == rows.ignore ? 0.f : p * r;
    }
  }
}

// out (+)= s in
__global__ void __launch_bounds__(256)
ce_finish_kernel(const float* in, const float* scale, float* out, int64_t n, int accumulate) {
  pdl_wait();
  pdl_trigger();
  const float s = scale[0];
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x)
    out[i] = accumulate ? out[i] + s * in[i] : s * in[i];
}

int grid_for(int64_t n) { return (int)std::min<int64_t>((n + 255) / 256, 152 * 16); }

#define OASES_TRY(expr)                       \
  do {                                        \
    const cudaError_t e_ = (expr);            \
    if (e_ != cudaSuccess) return e_;         \
  } while (0)

const char* row_of(const void* p, int64_t row, int H, DType t) {
  return static_cast<const char*>(p) + (size_t)row * H * dtype_size(t);
}

// Logits of the piece [v0, v0 + n), fp32.
cudaError_t piece_logits(const CeShape& s, const void* x, const void* w, int v0, int n, float* out,
                         cudaStream_t st) {
  GemmArgs g;
  g.M = s.M;
  g.N = n;
  g.K = s.H;
  g.in_t = s.t;
  g.A = x;
  g.lda = s.H;
  g.B = row_of(w, v0, s.H, s.t);
  g.ldb = s.H;
  g.C = out;
  g.ldc = s.ld;
  g.c_t = DType::F32;
  return gemm(g, st);
}

cudaError_t fwd(const CeShape& s, const void* x, const void* w, const int64_t* target, float* loss,
                float* lse, char* ws, cudaStream_t st) {
  const Layout l = layout(s, false);
  if (s.t == DType::BF16) return ce_tc_fwd(s, x, w, target, loss, lse, ws + l.logits, st);
  float* logits = reinterpret_cast<float*>(ws + l.logits);
  for (int v0 = 0; v0 < s.V; v0 += s.piece) {
    const int n = std::min(s.piece, s.V - v0);
    OASES_TRY(piece_logits(s, x, w, v0, n, logits, st));
    OASES_TRY(launch_pdl(ce_stat_kernel, dim3(std::min(s.M, 152 * 8)), dim3(256), 0, st,
                         (const float*)logits, s.ld, n, v0, v0 == 0, v0 + n == s.V,
                         reinterpret_cast<float*>(ws + l.run), target, s.ignore, s.V, loss, lse,
                         s.M));
  }
  return cudaSuccess;
}

cudaError_t finish(const float* in, const float* scale, void* out, int64_t n, bool accumulate,
                   cudaStream_t st) {
  return launch_pdl(ce_finish_kernel, dim3(grid_for(n)), dim3(256), 0, st, in, scale,
                    static_cast<float*>(out), n, accumulate ? 1 : 0);
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
  if (s.t == DType::BF16) return ce_tc_bwd(s, x, w, rows, lse, dx, dw, ws + l.logits, st);
  float* g = reinterpret_cast<float*>(ws + l.logits);
  float* tmp = reinterpret_cast<float*>(ws + l.run);
  for (int v0 = 0; v0 < s.V; v0 += s.piece) {
    const int n = std::min(s.piece, s.V - v0);
    OASES_TRY(piece_logits(s, x, w, v0, n, g, st));
    OASES_TRY(launch_pdl(ce_grad_kernel, dim3(std::min(s.M, 152 * 8)), dim3(256), 0, st, g, s.ld, n,
                         v0, lse, rows, s.M));
    if (dw) {
      GemmArgs q;
      q.M = n;
      q.N = s.H;
      q.K = s.M;
      q.in_t = s.t;
      q.A = g;
      q.lda = s.ld;
      q.a_kmajor = false;
      q.B = x;
      q.ldb = s.H;
      q.b_kmajor = false;
      q.C = tmp;
      q.ldc = s.H;
      q.c_t = DType::F32;
      OASES_TRY(gemm(q, st));
      OASES_TRY(finish(tmp, rows.scale, static_cast<float*>(dw) + (size_t)v0 * s.H, (int64_t)n * s.H,
                       s.accumulate, st));
    }
    if (dx) {
      GemmArgs q;
      q.M = s.M;
      q.N = s.H;
      q.K = n;
      q.in_t = s.t;
      q.A = g;
      q.lda = s.ld;
      q.B = row_of(w, v0, s.H, s.t);
      q.ldb = s.H;
      q.b_kmajor = false;
      q.epi = v0 == 0 ? Epi::Store : Epi::Accum;
      q.C = dx;
      q.ldc = s.H;
      q.c_t = DType::F32;
      OASES_TRY(gemm(q, st));
    }
  }
  if (dx) OASES_TRY(finish((const float*)dx, rows.scale, dx, (int64_t)s.M * s.H, false, st));
  return cudaSuccess;
}

bool misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p & 15) return true;
  return false;
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
  if (misaligned({x, w, target, loss, lse, workspace})) return OASES_ERR_INVALID_ARG;
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
  if (misaligned({x, w, target, lse, dloss, dx, dw, workspace})) return OASES_ERR_INVALID_ARG;
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
