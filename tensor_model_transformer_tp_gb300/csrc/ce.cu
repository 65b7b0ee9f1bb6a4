// Softmax cross entropy of a linear head (oases_ce.h), in pieces of the
// vocabulary: logits of a piece l = x W_piece^T, reduced to a running maximum
// and sum of every row, and, in the backward, turned into g of the piece, from
// which dx += g W_piece and dW_piece = g^T x.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "oases_ce.h"

namespace oases {
void api_begin();
void api_set_error(const char* what);
oases_status api_end(cudaError_t e);

namespace {

constexpr int64_t PIECE_BYTES = 256ll << 20;  // logits of one piece in the workspace

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct CeShape {
  int M, H, V;
  DType t, grad_t;
  bool per_row, accumulate;
  int64_t ignore;
  int piece;     // columns of the vocabulary per piece
  int64_t ld;    // leading dimension of the piece buffers
};

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
  size_t logits = 0, g = 0, run = 0, dx = 0, dw = 0, scale = 0, total = 0;
};
Layout layout(const CeShape& s, bool backward) {
  Layout l;
  auto take = [&](size_t* at, size_t bytes) {
    *at = l.total;
    l.total += align256(bytes);
  };
  if (s.M == 0) return l;
  take(&l.logits, (size_t)s.M * s.ld * 4);
  if (!backward) {
    take(&l.run, (size_t)s.M * 12);
  } else {
    take(&l.g, (size_t)s.M * s.ld * dtype_size(s.t));
    take(&l.dx, (size_t)s.M * s.H * 4);
    take(&l.dw, (size_t)s.piece * s.H * 4);
    take(&l.scale, 256);
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
        loss[m] = t == ignore ? 0.f : t < 0 || t >= V ? NAN : l - at;
      } else {
        run[m] = top;
        run[M + m] = s;
        run[2 * M + m] = at;
      }
    }
  }
}

// The largest |dloss| of the rows that have a loss, as the common factor s of
// g: g / s has entries up to 1 in magnitude, and with one dloss for every row
// the entry of the target, about -1, does not depend on what dloss rounds to.
__global__ void __launch_bounds__(1024)
ce_scale_kernel(const float* dloss, int per_row, const int64_t* target, int64_t ignore, int M,
                float* scale) {
  __shared__ float red[32];
  pdl_wait();
  pdl_trigger();
  float mx = 0.f;
  for (int m = threadIdx.x; m < M; m += blockDim.x)
    if (target[m] != ignore) mx = fmaxf(mx, fabsf(dloss[per_row ? m : 0]));
  mx = block_max(mx, red);
  if (threadIdx.x == 0) scale[0] = mx;
}

__device__ __forceinline__ float row_factor(const float* dloss, int per_row, const float* scale,
                                            int64_t t, int64_t ignore, int V, int m) {
  if (t == ignore) return 0.f;
  if (t < 0 || t >= V) return NAN;
  const float d = dloss[per_row ? m : 0], s = scale[0];
  return s == 0.f ? d : d / s;  // s == 0: d is 0 or NaN
}

// g / s of a piece: (exp(l - lse) - [v == target]) dloss / s; rows without a
// loss are 0 whatever their logits are.
template <typename T>
__global__ void __launch_bounds__(256)
ce_grad_kernel(const float* logits, int64_t ld, int n, int v0, const float* lse,
               const int64_t* target, int64_t ignore, int V, const float* dloss, int per_row,
               const float* scale, T* g, int M) {
  pdl_wait();
  pdl_trigger();
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    const int64_t t = target[m];
    const float r = row_factor(dloss, per_row, scale, t, ignore, V, m), l = lse[m];
    const float* row = logits + (int64_t)m * ld;
    T* out = g + (int64_t)m * ld;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const float p = expf(row[i] - l) - (t == v0 + i ? 1.f : 0.f);
      st_elem(out, i, t == ignore ? 0.f : p * r);
    }
  }
}

// out (+)= s in
template <typename T>
__global__ void __launch_bounds__(256)
ce_finish_kernel(const float* in, const float* scale, T* out, int64_t n, int accumulate) {
  pdl_wait();
  pdl_trigger();
  const float s = scale[0];
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    float v = s * in[i];
    if (accumulate) v += ld_elem(out, i);
    st_elem(out, i, v);
  }
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

template <typename T>
cudaError_t finish(const float* in, const float* scale, void* out, int64_t n, bool accumulate,
                   cudaStream_t st) {
  return launch_pdl(ce_finish_kernel<T>, dim3(grid_for(n)), dim3(256), 0, st, in, scale,
                    static_cast<T*>(out), n, accumulate ? 1 : 0);
}

template <typename T>
cudaError_t bwd(const CeShape& s, const void* x, const void* w, const int64_t* target,
                const float* lse, const float* dloss, void* dx, void* dw, char* ws,
                cudaStream_t st) {
  const Layout l = layout(s, true);
  float* logits = reinterpret_cast<float*>(ws + l.logits);
  T* gp = reinterpret_cast<T*>(ws + l.g);
  float* dx32 = reinterpret_cast<float*>(ws + l.dx);
  float* dw32 = reinterpret_cast<float*>(ws + l.dw);
  float* scale = reinterpret_cast<float*>(ws + l.scale);
  OASES_TRY(launch_pdl(ce_scale_kernel, dim3(1), dim3(1024), 0, st, dloss, (int)s.per_row, target,
                       s.ignore, s.M, scale));
  for (int v0 = 0; v0 < s.V; v0 += s.piece) {
    const int n = std::min(s.piece, s.V - v0);
    OASES_TRY(piece_logits(s, x, w, v0, n, logits, st));
    OASES_TRY(launch_pdl(ce_grad_kernel<T>, dim3(std::min(s.M, 152 * 8)), dim3(256), 0, st,
                         (const float*)logits, s.ld, n, v0, lse, target, s.ignore, s.V, dloss,
                         (int)s.per_row, (const float*)scale, gp, s.M));
    if (dx) {
      GemmArgs g;
      g.M = s.M;
      g.N = s.H;
      g.K = n;
      g.in_t = s.t;
      g.A = gp;
      g.lda = s.ld;
      g.B = row_of(w, v0, s.H, s.t);
      g.ldb = s.H;
      g.b_kmajor = false;
      g.epi = v0 == 0 ? Epi::Store : Epi::Accum;
      g.C = dx32;
      g.ldc = s.H;
      g.c_t = DType::F32;
      OASES_TRY(gemm(g, st));
    }
    if (dw) {
      GemmArgs g;
      g.M = n;
      g.N = s.H;
      g.K = s.M;
      g.in_t = s.t;
      g.A = gp;
      g.lda = s.ld;
      g.a_kmajor = false;
      g.B = x;
      g.ldb = s.H;
      g.b_kmajor = false;
      g.C = dw32;
      g.ldc = s.H;
      g.c_t = DType::F32;
      OASES_TRY(gemm(g, st));
      const int64_t n_out = (int64_t)n * s.H;
      char* out = static_cast<char*>(dw) + (size_t)v0 * s.H * dtype_size(s.grad_t);
      OASES_TRY(s.grad_t == DType::F32
                    ? finish<float>(dw32, scale, out, n_out, s.accumulate, st)
                    : finish<__nv_bfloat16>(dw32, scale, out, n_out, false, st));
    }
  }
  if (dx) OASES_TRY(finish<T>(dx32, scale, dx, (int64_t)s.M * s.H, false, st));
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
  return api_end(s.t == DType::F32 ? bwd<float>(s, x, w, target, lse, dloss, dx, dw, ws, st)
                                   : bwd<__nv_bfloat16>(s, x, w, target, lse, dloss, dx, dw, ws, st));
}
