// Gated feed-forward block (oases_glu.h):
//   a = x Wg^T + bg, b = x Wu^T + bu, h = act(a) b, y = h W2^T + b2 (+ resid)
// and its backward.  The products are GEMMs; what lies between them is
// element-wise over [rows, ffn].
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "oases_glu.h"
#include "oases_mx.h"

namespace oases {
void api_begin();
void api_set_error(const char* what);
oases_status api_end(cudaError_t e);

namespace {

constexpr int MXB = 32;  // elements per scale of the 8-bit form

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct GluShape {
  int M, H, F;
  DType t, dx_t, grad_t;
  int act, keep;
  bool accumulate;
  int64_t ldq;  // leading dimension of the 8-bit codes
};

oases_status glu_shape(const oases_glu_desc* d, GluShape* s) {
  if (!d) return OASES_ERR_INVALID_ARG;
  if (d->dtype != OASES_F32 && d->dtype != OASES_BF16) return OASES_ERR_INVALID_ARG;
  if (d->rows < 0 || d->hidden <= 0 || d->ffn <= 0 || d->ffn > (1 << 29)) return OASES_ERR_INVALID_ARG;
  if (d->act != OASES_ACT_SILU && d->act != OASES_ACT_GELU) return OASES_ERR_INVALID_ARG;
  if (d->keep < OASES_GLU_KEEP_NONE || d->keep > OASES_GLU_KEEP_MXFP8) return OASES_ERR_INVALID_ARG;
  if (d->dx_dtype != OASES_F32 && d->dx_dtype != d->dtype) return OASES_ERR_INVALID_ARG;
  if (d->grad_dtype != OASES_F32 && d->grad_dtype != d->dtype) return OASES_ERR_INVALID_ARG;
  if (d->accumulate != 0 && d->accumulate != 1) return OASES_ERR_INVALID_ARG;
  if (d->accumulate && d->grad_dtype != OASES_F32) return OASES_ERR_INVALID_ARG;
  if (d->dtype == OASES_BF16 && (d->hidden % 8 != 0 || d->ffn % 8 != 0)) return OASES_ERR_UNSUPPORTED;
  if (d->dtype == OASES_F32 && d->keep == OASES_GLU_KEEP_MXFP8) return OASES_ERR_UNSUPPORTED;
  s->M = d->rows;
  s->H = d->hidden;
  s->F = d->ffn;
  s->t = static_cast<DType>(d->dtype);
  s->dx_t = static_cast<DType>(d->dx_dtype);
  s->grad_t = static_cast<DType>(d->grad_dtype);
  s->act = d->act;
  s->keep = d->keep;
  s->accumulate = d->accumulate != 0;
  s->ldq = (s->F + 15) / 16 * 16;
  return OASES_OK;
}

// Kept activations (oases_glu_keep): where the scales of the 8-bit form start.
size_t saved_scale_offset(const GluShape& s) { return align256(2 * (size_t)s.M * s.ldq); }
size_t saved_bytes(const GluShape& s) {
  if (s.keep == OASES_GLU_KEEP_PRE) return 2 * (size_t)s.M * s.F * dtype_size(s.t);
  if (s.keep == OASES_GLU_KEEP_MXFP8)
    return saved_scale_offset(s) + 2 * (size_t)mx_sf_bytes(s.M, s.F);
  return 0;
}

// Workspace regions, each a multiple of 256 bytes.
struct Layout {
  size_t pre = 0, h = 0, dh = 0, dpre = 0, bias = 0, part = 0, total = 0;
};
Layout layout(const GluShape& s, bool backward) {
  Layout l;
  const size_t MF = (size_t)s.M * s.F, e = dtype_size(s.t);
  auto take = [&](size_t* at, size_t bytes) {
    *at = l.total;
    l.total += align256(bytes);
  };
  if (s.M == 0) return l;
  const int wide = std::max(2 * s.F, s.H);
  if (!backward || s.keep == OASES_GLU_KEEP_NONE) take(&l.pre, 2 * MF * 4);
  take(&l.h, MF * e);
  if (backward) {
    take(&l.dh, MF * 4);
    take(&l.dpre, 2 * MF * e);
    take(&l.part, (size_t)colsum_blocks(s.M) * wide * 4);
  }
  take(&l.bias, (size_t)wide * 4);
  return l;
}

// ---- element-wise kernels ----------------------------------------------------
// act(a) and its derivative in fp32.  SiLU: s = 1 / (1 + e^-a), act = a s,
// act' = s (1 + a (1 - s)).
__device__ __forceinline__ void act_both(int act, float a, float& f, float& df) {
  if (act == OASES_ACT_SILU) {
    const float s = 1.0f / (1.0f + expf(-a));
    f = a * s;
    df = s * fmaf(a, 1.0f - s, 1.0f);
  } else {
    float cdf, pdf;
    gelu_cdf_pdf(a, cdf, pdf);
    f = a * cdf;
    df = fmaf(a, pdf, cdf);
  }
}

// h = act(a + bg) (b + bu) from the fp32 projections p [M, 2F]; keeps [a | b]
// with the biases in `kept` if given, and leaves them in p (what the 8-bit
// form is quantised from).
template <typename T>
__global__ void __launch_bounds__(256)
glu_act_kernel(float* p, const T* bias, T* h, T* kept, int64_t MF, int F, int act) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < MF;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t m = i / F;
    const int f = (int)(i - m * F);
    const int64_t ia = m * 2 * F + f, ib = ia + F;
    float a = p[ia], b = p[ib];
    if (bias) {
      a += ld_elem(bias, f);
      b += ld_elem(bias, F + f);
      p[ia] = a;
      p[ib] = b;
    }
    if (kept) {
      st_elem(kept, ia, a);
      st_elem(kept, ib, b);
    }
    float g, dg;
    act_both(act, a, g, dg);
    if (h) st_elem(h, i, g * b);
  }
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  // sign, 4 exponent bits (bias 7), 3 mantissa bits
  const int e = (c >> 3) & 15, m = c & 7;
  const float v = e ? ldexpf((float)(8 + m), e - 10) : ldexpf((float)m, -9);
  return c & 0x80 ? -v : v;
}

// Where the backward takes a and b from.
struct KeptIn {
  const void* pre;        // [M, 2F] in the storage type
  const float* pre32;     // [M, 2F] fp32 (recomputed)
  const uint8_t* codes;   // MX operands, gate then up
  const uint8_t* scales;
  int64_t code_stride, scale_stride, ldq;
  int kgroups;
};

// dh fp32 [M, F] -> dpre = [da | db] [M, 2F] and h [M, F].
template <typename T>
__global__ void __launch_bounds__(256)
glu_grad_kernel(const KeptIn k, const float* dh, T* dpre, T* h, int64_t MF, int F, int act) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < MF;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t m = i / F;
    const int f = (int)(i - m * F);
    const int64_t ia = m * 2 * F + f, ib = ia + F;
    float a, b;
    if (k.codes) {
      const int64_t at = ((m / 128) * k.kgroups + f / 128) * 512 + (m % 32) * 16 + ((m % 128) / 32) * 4 +
                         (f / MXB) % 4;
      const int64_t c = m * k.ldq + f;
      a = e4m3_value(k.codes[c]) * ldexpf(1.0f, (int)k.scales[at] - 127);
      b = e4m3_value(k.codes[k.code_stride + c]) *
          ldexpf(1.0f, (int)k.scales[k.scale_stride + at] - 127);
    } else if (k.pre32) {
      a = k.pre32[ia];
      b = k.pre32[ib];
    } else {
      a = ld_elem(static_cast<const T*>(k.pre), ia);
      b = ld_elem(static_cast<const T*>(k.pre), ib);
    }
    float g, dg;
    act_both(act, a, g, dg);
    const float d = dh[i];
    st_elem(dpre, ia, d * b * dg);
    st_elem(dpre, ib, d * g);
    st_elem(h, i, g * b);
  }
}

// out (type T) = in (fp32)
template <typename T>
__global__ void __launch_bounds__(256) cast_kernel(const float* in, T* out, int n) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) st_elem(out, i, in[i]);
}

int grid_for(int64_t n) { return (int)std::min<int64_t>((n + 255) / 256, 152 * 16); }

struct Gemm : GemmArgs {
  Gemm(int m, int n, int k, DType t) {
    M = m;
    N = n;
    K = k;
    in_t = aux_t = t;
  }
};

// Column sums of in [M, N] (type t) to a bias gradient.
cudaError_t bias_grad(const void* in, int M, int N, DType t, void* out, DType out_t, bool accumulate,
                      float* part, float* tmp, cudaStream_t st) {
  if (accumulate) return colsum_accum(in, N, M, N, t, part, static_cast<float*>(out), st);
  float* sum = out_t == DType::F32 ? static_cast<float*>(out) : tmp;
  cudaError_t e = cudaMemsetAsync(sum, 0, (size_t)N * 4, st);
  if (e == cudaSuccess) e = colsum_accum(in, N, M, N, t, part, sum, st);
  if (e == cudaSuccess && out_t == DType::BF16)
    e = launch_pdl(cast_kernel<__nv_bfloat16>, dim3((N + 255) / 256), dim3(256), 0, st,
                   (const float*)tmp, (__nv_bfloat16*)out, N);
  return e;
}

#define OASES_TRY(expr)                       \
  do {                                        \
    const cudaError_t e_ = (expr);            \
    if (e_ != cudaSuccess) return e_;         \
  } while (0)

// [a | b] without biases, fp32, and what follows from it.
template <typename T>
cudaError_t project(const GluShape& s, const oases_glu_weights& w, const void* x, float* pre, T* h,
                    void* saved, cudaStream_t st) {
  const int64_t MF = (int64_t)s.M * s.F;
  Gemm g(s.M, 2 * s.F, s.H, s.t);
  g.A = x;
  g.lda = s.H;
  g.B = w.w1;
  g.ldb = s.H;
  g.C = pre;
  g.ldc = 2 * s.F;
  g.c_t = DType::F32;
  OASES_TRY(gemm(g, st));
  OASES_TRY(launch_pdl(glu_act_kernel<T>, dim3(grid_for(MF)), dim3(256), 0, st, pre, (const T*)w.b1,
                       h, s.keep == OASES_GLU_KEEP_PRE ? (T*)saved : (T*)nullptr, MF, s.F, s.act));
  if (s.keep == OASES_GLU_KEEP_MXFP8 && saved) {
    uint8_t* q = static_cast<uint8_t*>(saved);
    uint8_t* sf = q + saved_scale_offset(s);
    for (int half = 0; half < 2; ++half)
      OASES_TRY(mx_quantize_rows(pre + half * s.F, 2 * s.F, s.M, s.F, DType::F32,
                                 q + (size_t)half * s.M * s.ldq, s.ldq,
                                 sf + (size_t)half * mx_sf_bytes(s.M, s.F), st));
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t fwd(const GluShape& s, const oases_glu_weights& w, const void* x, const void* resid,
                void* y, void* saved, char* ws, cudaStream_t st) {
  const Layout l = layout(s, false);
  T* h = reinterpret_cast<T*>(ws + l.h);
  OASES_TRY(project<T>(s, w, x, reinterpret_cast<float*>(ws + l.pre), h, saved, st));
  Gemm g(s.M, s.H, s.F, s.t);
  g.A = h;
  g.lda = s.F;
  g.B = w.w2;
  g.ldb = s.F;
  g.C = y;
  g.ldc = s.H;
  g.c_t = s.t;
  g.bias = w.b2;
  if (resid) {
    if (!w.b2) {  // BiasResid with a zero bias
      OASES_TRY(cudaMemsetAsync(ws + l.bias, 0, (size_t)s.H * 4, st));
      g.bias = ws + l.bias;
    }
    g.epi = Epi::BiasResid;
    g.aux = resid;
    g.ld_aux = s.H;
  } else {
    g.epi = w.b2 ? Epi::Bias : Epi::Store;
  }
  return gemm(g, st);
}

// dW [N, K] (+)= A^T B over the rows, A [M, N], B [M, K].
cudaError_t weight_grad(const GluShape& s, const void* A, int N, const void* B, int K, void* out,
                        cudaStream_t st) {
  Gemm g(N, K, s.M, s.t);
  g.A = A;
  g.lda = N;
  g.a_kmajor = false;
  g.B = B;
  g.ldb = K;
  g.b_kmajor = false;
  g.epi = s.accumulate ? Epi::Accum : Epi::Store;
  g.C = out;
  g.ldc = K;
  g.c_t = s.grad_t;
  return gemm(g, st);
}

template <typename T>
cudaError_t bwd(const GluShape& s, const oases_glu_weights& w, const void* x, const void* dy,
                const void* saved, void* dx, const oases_glu_grads& gr, char* ws, cudaStream_t st) {
  const Layout l = layout(s, true);
  const int64_t MF = (int64_t)s.M * s.F;
  T* h = reinterpret_cast<T*>(ws + l.h);
  T* dpre = reinterpret_cast<T*>(ws + l.dpre);
  float* dh = reinterpret_cast<float*>(ws + l.dh);
  float* part = reinterpret_cast<float*>(ws + l.part);
  float* tmp = reinterpret_cast<float*>(ws + l.bias);
  KeptIn k = {};
  if (s.keep == OASES_GLU_KEEP_NONE) {
    float* pre = reinterpret_cast<float*>(ws + l.pre);
    OASES_TRY(project<T>(s, w, x, pre, (T*)nullptr, nullptr, st));
    k.pre32 = pre;
  } else if (s.keep == OASES_GLU_KEEP_PRE) {
    k.pre = saved;
  } else {
    k.codes = static_cast<const uint8_t*>(saved);
    k.scales = k.codes + saved_scale_offset(s);
    k.code_stride = (int64_t)s.M * s.ldq;
    k.scale_stride = mx_sf_bytes(s.M, s.F);
    k.ldq = s.ldq;
    k.kgroups = (s.F + 127) / 128;
  }
  Gemm g(s.M, s.F, s.H, s.t);
  g.A = dy;
  g.lda = s.H;
  g.B = w.w2;
  g.ldb = s.F;
  g.b_kmajor = false;
  g.C = dh;
  g.ldc = s.F;
  g.c_t = DType::F32;
  OASES_TRY(gemm(g, st));
  OASES_TRY(launch_pdl(glu_grad_kernel<T>, dim3(grid_for(MF)), dim3(256), 0, st, k, (const float*)dh,
                       dpre, h, MF, s.F, s.act));
  if (gr.w2) OASES_TRY(weight_grad(s, dy, s.H, h, s.F, gr.w2, st));
  if (gr.w1) OASES_TRY(weight_grad(s, dpre, 2 * s.F, x, s.H, gr.w1, st));
  if (gr.b2) OASES_TRY(bias_grad(dy, s.M, s.H, s.t, gr.b2, s.grad_t, s.accumulate, part, tmp, st));
  if (gr.b1)
    OASES_TRY(bias_grad(dpre, s.M, 2 * s.F, s.t, gr.b1, s.grad_t, s.accumulate, part, tmp, st));
  if (dx) {
    Gemm q(s.M, s.H, 2 * s.F, s.t);
    q.A = dpre;
    q.lda = 2 * s.F;
    q.B = w.w1;
    q.ldb = s.H;
    q.b_kmajor = false;
    q.C = dx;
    q.ldc = s.H;
    q.c_t = s.dx_t;
    OASES_TRY(gemm(q, st));
  }
  return cudaSuccess;
}

bool misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p & 15) return true;
  return false;
}

}  // namespace
}  // namespace oases

extern "C" size_t oases_glu_saved_bytes(const oases_glu_desc* desc) {
  oases::GluShape s;
  if (oases::glu_shape(desc, &s) != OASES_OK) return 0;
  return oases::saved_bytes(s);
}

extern "C" size_t oases_glu_workspace_bytes(const oases_glu_desc* desc, int backward) {
  oases::GluShape s;
  if (oases::glu_shape(desc, &s) != OASES_OK) return 0;
  return oases::layout(s, backward != 0).total;
}

extern "C" oases_status oases_glu_fwd(const oases_glu_desc* desc, const oases_glu_weights* wts,
                                      const void* x, const void* resid, void* y, void* saved,
                                      void* workspace, size_t ws_bytes, void* stream) {
  using namespace oases;
  api_begin();
  GluShape s;
  const oases_status v = glu_shape(desc, &s);
  if (v != OASES_OK) return v;
  if (s.M == 0) return OASES_OK;
  if (!wts || !wts->w1 || !wts->w2 || !x || !y) return OASES_ERR_INVALID_ARG;
  if (s.keep != OASES_GLU_KEEP_NONE && !saved) return OASES_ERR_INVALID_ARG;
  if (misaligned({wts->w1, wts->b1, wts->w2, wts->b2, x, resid, y, saved, workspace}))
    return OASES_ERR_INVALID_ARG;
  const size_t need = layout(s, false).total;
  if (need > 0 && (!workspace || ws_bytes < need)) return OASES_ERR_WORKSPACE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  return api_end(s.t == DType::F32 ? fwd<float>(s, *wts, x, resid, y, saved, ws, st)
                                   : fwd<__nv_bfloat16>(s, *wts, x, resid, y, saved, ws, st));
}

extern "C" oases_status oases_glu_bwd(const oases_glu_desc* desc, const oases_glu_weights* wts,
                                      const void* x, const void* dy, const void* saved, void* dx,
                                      const oases_glu_grads* grads, void* workspace,
                                      size_t ws_bytes, void* stream) {
  using namespace oases;
  api_begin();
  GluShape s;
  const oases_status v = glu_shape(desc, &s);
  if (v != OASES_OK) return v;
  if (!wts || !grads) return OASES_ERR_INVALID_ARG;
  if ((grads->b1 && !wts->b1) || (grads->b2 && !wts->b2)) return OASES_ERR_INVALID_ARG;
  if (misaligned({wts->w1, wts->b1, wts->w2, wts->b2, x, dy, saved, dx, grads->w1, grads->b1,
                  grads->w2, grads->b2, workspace}))
    return OASES_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s.M == 0) {  // sums over no rows
    if (s.accumulate) return OASES_OK;
    const size_t e = dtype_size(s.grad_t), F = s.F, H = s.H;
    cudaError_t err = cudaSuccess;
    auto zero = [&](void* p, size_t n) {
      if (p && err == cudaSuccess) err = cudaMemsetAsync(p, 0, n * e, st);
    };
    zero(grads->w1, 2 * F * H);
    zero(grads->b1, 2 * F);
    zero(grads->w2, F * H);
    zero(grads->b2, H);
    return api_end(err);
  }
  if (!wts->w1 || !wts->w2 || !x || !dy) return OASES_ERR_INVALID_ARG;
  if (s.keep != OASES_GLU_KEEP_NONE && !saved) return OASES_ERR_INVALID_ARG;
  const size_t need = layout(s, true).total;
  if (need > 0 && (!workspace || ws_bytes < need)) return OASES_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  return api_end(s.t == DType::F32
                     ? bwd<float>(s, *wts, x, dy, saved, dx, *grads, ws, st)
                     : bwd<__nv_bfloat16>(s, *wts, x, dy, saved, dx, *grads, ws, st));
}
