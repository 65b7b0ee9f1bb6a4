// Gated feed-forward block (oases_glu.h):
//   a = x Wg^T + bg, b = x Wu^T + bu, h = act(a) b, y = h W2^T + b2 (+ resid)
// and its backward.  bf16 runs on the fused tensor-core kernels of glu_tc.cu,
// glu_few.cu and glu_again.cu, fp32 on the CUDA-core GEMM with the same epilogues.
#include <cuda_runtime.h>

#include <algorithm>

#include "gemm_f32.cuh"
#include "glu.cuh"

namespace oases {
void api_begin();
oases_status api_end(cudaError_t e);

namespace {

constexpr int MAX_DIM = 1 << 29;  // rows, hidden, ffn: 32-bit tile and TMA coordinates

oases_status glu_shape(const oases_glu_desc* d, GluShape* s) {
  if (!d) return OASES_ERR_INVALID_ARG;
  if (d->dtype != OASES_F32 && d->dtype != OASES_BF16) return OASES_ERR_INVALID_ARG;
  if (d->rows < 0 || d->hidden <= 0 || d->ffn <= 0) return OASES_ERR_INVALID_ARG;
  if (d->act != OASES_ACT_SILU && d->act != OASES_ACT_GELU) return OASES_ERR_INVALID_ARG;
  if (d->keep < OASES_GLU_KEEP_NONE || d->keep > OASES_GLU_KEEP_MXFP8) return OASES_ERR_INVALID_ARG;
  if (d->dx_dtype != OASES_F32 && d->dx_dtype != d->dtype) return OASES_ERR_INVALID_ARG;
  if (d->grad_dtype != OASES_F32 && d->grad_dtype != d->dtype) return OASES_ERR_INVALID_ARG;
  if (d->accumulate != 0 && d->accumulate != 1) return OASES_ERR_INVALID_ARG;
  if (d->accumulate && d->grad_dtype != OASES_F32) return OASES_ERR_INVALID_ARG;
  if (d->dtype == OASES_BF16 && (d->hidden % 8 != 0 || d->ffn % 8 != 0)) return OASES_ERR_UNSUPPORTED;
  if (std::max({d->rows, d->hidden, d->ffn}) > (d->dtype == OASES_F32 ? f32::MAX_DIM : MAX_DIM))
    return OASES_ERR_UNSUPPORTED;
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
  const bool bf = s->t == DType::BF16;
  s->ldh = bf ? ((int64_t)s->F + 63) / 64 * 64 : s->F;
  s->ldp = bf ? (2 * (int64_t)s->F + 63) / 64 * 64 : 2 * (int64_t)s->F;
  return OASES_OK;
}

size_t saved_bytes(const GluShape& s) {
  if (s.keep == OASES_GLU_KEEP_PRE) return 2 * (size_t)s.M * s.F * dtype_size(s.t);
  if (s.keep == OASES_GLU_KEEP_MXFP8)
    return saved_scale_offset(s) + 2 * (size_t)mx_sf_bytes(s.M, s.F);
  return 0;
}

// Workspace regions, each a multiple of 256 bytes.
struct Layout {
  size_t pre = 0, h = 0, dpre = 0, dx = 0 /* partial sums of dx, or of y */, total = 0;
};
Layout layout(const GluShape& s, bool backward) {
  Layout l;
  const size_t e = dtype_size(s.t), h = (size_t)s.M * s.ldh * e, pre = (size_t)s.M * s.ldp * e;
  auto take = [&](size_t* at, size_t bytes) {
    *at = l.total;
    l.total += align256(bytes);
  };
  if (s.M == 0) return l;
  take(&l.h, h);
  if (!backward && s.t == DType::BF16) take(&l.dx, glu_down_tc_bytes(s));
  if (backward) {
    if (s.keep == OASES_GLU_KEEP_NONE && s.t == DType::F32) take(&l.pre, pre);
    take(&l.dpre, pre);
    if (s.t == DType::BF16) take(&l.dx, glu_grads_tc_bytes(s));
  }
  return l;
}

// ---- fp32 epilogues ------------------------------------------------------------
// act(a) and its derivative, to fp32's own accuracy: SiLU with s = 1 / (1 + e^-a),
// act = a s, act' = s (1 + a (1 - s)); GeLU a Phi(a), Phi(a) + a phi(a).  (The
// rational form of Phi that serves bf16 is off by up to 7.5e-8, which at a = -5 is a
// quarter of Phi; it saves 8 of 530 us in a forward of 4096 x 512 x 2048.)
__device__ __forceinline__ void act_both(int act, float a, float& f, float& df) {
  if (act == OASES_ACT_SILU) {
    const float s = 1.0f / (1.0f + expf(-a));
    f = a * s;
    df = s * fmaf(a, 1.0f - s, 1.0f);
  } else {
    const float cdf = normcdff(a);
    f = a * cdf;
    df = fmaf(a, 0.39894228040143268f * expf(-0.5f * a * a), cdf);
  }
}

// Both projections of an output: h = act(a + bg) (b + bu), and [a | b] to `pre`.
struct UpF32 {
  static constexpr bool DUAL = true;
  const float* bias;
  float *h, *pre;
  int act;
  __device__ __forceinline__ void tile(int m, int n0, const float (&va)[4], const float (&vb)[4],
                                       int col, int M, int N) const {
    if (m >= M) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + col + i;
      if (n >= N) break;
      float a = va[i], b = vb[i], f, df;
      if (bias) {
        a += bias[n];
        b += bias[N + n];
      }
      if (pre) {
        pre[(int64_t)m * 2 * N + n] = a;
        pre[(int64_t)m * 2 * N + N + n] = b;
      }
      if (h) {
        act_both(act, a, f, df);
        h[(int64_t)m * N + n] = f * b;
      }
    }
  }
};

// dh of an output: [da | db] to `dpre` and h, at pre = [a | b].
struct GradF32 {
  static constexpr bool DUAL = false;
  const float* pre;
  float *dpre, *h;
  int act;
  __device__ __forceinline__ void tile(int m, int n0, const float (&d)[4], int col, int M, int N) const {
    if (m >= M) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + col + i;
      if (n >= N) break;
      const int64_t ia = (int64_t)m * 2 * N + n, ib = ia + N;
      const float a = pre[ia], b = pre[ib];
      float f, df;
      act_both(act, a, f, df);
      dpre[ia] = d[i] * b * df;
      dpre[ib] = d[i] * f;
      h[(int64_t)m * N + n] = f * b;
    }
  }
};

// Column sums of in[0] [M, N0] and in[1] [M, N1] (leading dimensions ld) in one
// launch, out (+)= sums.  (At 8192 rows and ffn 4096, 10 us less than blocks of
// rows summed to partial rows and those in a second launch.)  Few columns and many
// rows: a cluster of `split` CTAs shares the rows, and its first CTA joins the sums
// in order.
struct Sums {
  const void* in[2];
  void* out[2];
  int N[2];
  int64_t ld[2];
};
// V neighbouring columns per thread (16 bytes of bf16 rows, which start on such;
// one column of fp32 rows), 8 V columns and 64 row groups per block.
template <typename T, int V>
struct RowLoad;
template <>
struct RowLoad<__nv_bfloat16, 8> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void add(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
      v[2 * k] += f.x;
      v[2 * k + 1] += f.y;
    }
  }
};
template <>
struct RowLoad<float, 1> {
  float u;
  __device__ __forceinline__ void load(const float* p) { u = __ldg(p); }
  __device__ __forceinline__ void add(float (&v)[1]) const { v[0] += u; }
};
template <typename T, typename O, int V>
__global__ void __launch_bounds__(512) column_sums_kernel(const Sums s, int rows, int split, int accumulate) {
  __shared__ float red[16][8 * V + 1];
  __shared__ float part[8 * V];
  pdl_wait();
  pdl_trigger();
  const int x = threadIdx.x % 8, y = threadIdx.x / 8, first = (s.N[0] + 8 * V - 1) / (8 * V);
  const int block = (int)blockIdx.x / split, rank = (int)blockIdx.x % split;
  const int which = block < first ? 0 : 1;
  const int n0 = (block - (which ? first : 0)) * 8 * V, n = n0 + V * x, N = s.N[which];
  const int span = (rows + split - 1) / split, m0 = min(rows, rank * span), M = min(rows - m0, span);
  const int64_t ld = s.ld[which];
  const T* in = static_cast<const T*>(s.in[which]) + m0 * ld + n;
  float v[V] = {};
  if (n < N) {  // bf16: N is a multiple of V
    RowLoad<T, V> r[8];
    int m = y;
    for (; m + 7 * 64 < M; m += 8 * 64) {  // eight rows in flight
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i].load(in + (m + 64 * i) * ld);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i].add(v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (m + 64 * i < M) r[i].load(in + (m + 64 * i) * ld);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (m + 64 * i < M) r[i].add(v);
  }
  // the four row groups of a warp, then the sixteen warps, in a fixed order
#pragma unroll
  for (int k = 0; k < V; ++k) {
    v[k] += __shfl_down_sync(0xffffffffu, v[k], 16);
    v[k] += __shfl_down_sync(0xffffffffu, v[k], 8);
    if (threadIdx.x % 32 < 8) red[threadIdx.x / 32][V * x + k] = v[k];
  }
  __syncthreads();
  float t = 0.f;
  if ((int)threadIdx.x < 8 * V) {
    for (int i = 0; i < 16; ++i) t += red[i][threadIdx.x];
    part[threadIdx.x] = t;
  }
  if (split > 1) {
    ptx::cluster_sync();
    if (rank == 0 && (int)threadIdx.x < 8 * V)
      for (int i = 1; i < split; ++i) t += ptx::ld_cluster(ptx::mapa(ptx::smem_u32(&part[threadIdx.x]), i));
    ptx::cluster_sync();  // the others' shared memory is there while it is read
  }
  if (rank == 0 && (int)threadIdx.x < 8 * V && n0 + (int)threadIdx.x < N) {
    O* out = static_cast<O*>(s.out[which]) + n0 + threadIdx.x;
    st_elem(out, 0, accumulate ? ld_elem(out, 0) + t : t);
  }
}

// The rows are split, 512 at least to a CTA, where the blocks of columns leave SMs
// idle: 16384 rows of 1536 x 2 + 1024 columns 58 -> 35 us, 65536 of 64 x 2 + 64 in
// fp32 116 -> 18; with 102 and 144 blocks a split only costs (13 -> 20 us).
template <typename T, typename O, int V>
cudaError_t launch_sums(const Sums& q, int M, int accumulate, cudaStream_t st) {
  const int blocks = (q.N[0] + 8 * V - 1) / (8 * V) + (q.N[1] + 8 * V - 1) / (8 * V);
  int split = 1;
  while (split < 8 && 2 * split * blocks <= 192 && M >= 1024 * split) split *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attrs[2];
  f32::configure(&cfg, attrs, dim3((unsigned)split), st);
  cfg.gridDim = dim3((unsigned)split * blocks);
  cfg.blockDim = dim3(512);
  return cudaLaunchKernelEx(&cfg, column_sums_kernel<T, O, V>, q, M, split, accumulate);
}

// db1 = colsum(dpre), db2 = colsum(dy), each where it is wanted.  dpre holds da and db
// as they are rounded for dw1 and dx: the rounding errors of M rows mostly cancel in
// the fp32 sum (2^-9 / sqrt(M) of its terms' size), and the epilogues that form da and
// db need no second set of column sums.
cudaError_t bias_grads(const GluShape& s, const void* dpre, const void* dy, const oases_glu_grads& gr,
                       cudaStream_t st) {
  if (!gr.b1 && !gr.b2) return cudaSuccess;
  const Sums q{{dpre, dy}, {gr.b1, gr.b2}, {gr.b1 ? 2 * s.F : 0, gr.b2 ? s.H : 0},
               {s.ldp, s.H}};
  const int acc = s.accumulate ? 1 : 0;
  if (s.t == DType::F32) return launch_sums<float, float, 1>(q, s.M, acc, st);
  if (s.grad_t == DType::F32) return launch_sums<__nv_bfloat16, float, 8>(q, s.M, acc, st);
  return launch_sums<__nv_bfloat16, __nv_bfloat16, 8>(q, s.M, acc, st);
}

// [a | b] and h = act(a) b; pre and kept8 (and, fp32, h) are left out when null.
cudaError_t project(const GluShape& s, const oases_glu_weights& w, const void* x, void* h, void* pre,
                    void* kept8, cudaStream_t st) {
  if (s.t == DType::BF16) return glu_project_tc(s, x, w.w1, w.b1, h, pre, kept8, st);
  const f32::Args g{s.M, s.F, s.H, (const float*)x, s.H, (const float*)w.w1, s.H, s.F};
  return f32::launch<UpF32, true, true>(
      g, UpF32{(const float*)w.b1, (float*)h, (float*)pre, s.act}, st);
}

cudaError_t fwd(const GluShape& s, const oases_glu_weights& w, const void* x, const void* resid,
                void* y, void* saved, char* ws, cudaStream_t st) {
  void* h = ws + layout(s, false).h;
  OASES_TRY(project(s, w, x, h, s.keep == OASES_GLU_KEEP_PRE ? saved : nullptr,
                    s.keep == OASES_GLU_KEEP_MXFP8 ? saved : nullptr, st));
  if (s.t == DType::BF16)
    return glu_down_tc(s, h, w.w2, w.b2, resid, y, ws + layout(s, false).dx, st);
  const f32::Args g{s.M, s.H, s.F, (const float*)h, s.F, (const float*)w.w2, s.F};
  return f32::launch<f32::Out, true, true>(
      g, f32::Out{(float*)y, s.H, nullptr, (const float*)w.b2, (const float*)resid, 0}, st);
}

cudaError_t bwd(const GluShape& s, const oases_glu_weights& w, const void* x, const void* dy,
                const void* saved, void* dx, const oases_glu_grads& gr, char* ws, cudaStream_t st) {
  const Layout l = layout(s, true);
  void *h = ws + l.h, *dpre = ws + l.dpre;
  if (s.t == DType::BF16) {
    if (s.keep == OASES_GLU_KEEP_NONE)
      OASES_TRY(glu_grad_again_tc(s, x, dy, w.w1, w.b1, w.w2, dpre, h, st));
    else if (s.keep == OASES_GLU_KEEP_PRE)
      OASES_TRY(glu_grad_tc(s, dy, w.w2, saved, nullptr, dpre, h, st));
    else
      OASES_TRY(glu_grad_tc(s, dy, w.w2, nullptr, saved, dpre, h, st));
    OASES_TRY(glu_grads_tc(s, x, dy, w.w1, dpre, h, dx, gr.w1, gr.w2, ws + l.dx, st));
  } else {
    const void* pre = saved;
    if (s.keep == OASES_GLU_KEEP_NONE) {
      OASES_TRY(project(s, w, x, nullptr, ws + l.pre, nullptr, st));
      pre = ws + l.pre;
    }
    const f32::Args g{s.M, s.F, s.H, (const float*)dy, s.H, (const float*)w.w2, s.F};
    OASES_TRY((f32::launch<GradF32, true, false>(
        g, GradF32{(const float*)pre, (float*)dpre, (float*)h, s.act}, st)));
    // dx, dw1 = dpre^T x, dw2 = dy^T h
    const float *px = (const float*)x, *pdy = (const float*)dy, *pw1 = (const float*)w.w1;
    const float *pd = (const float*)dpre, *ph = (const float*)h;
    const f32::Args args[3] = {{s.M, s.H, 2 * s.F, pd, 2 * s.F, pw1, s.H},
                               {2 * s.F, s.H, s.M, pd, 2 * s.F, px, s.H},
                               {s.H, s.F, s.M, pdy, s.H, ph, s.F}};
    const int acc = s.accumulate;
    const f32::Out out[3] = {{(float*)dx, s.H, nullptr, nullptr, nullptr, 0},
                             {(float*)gr.w1, s.H, nullptr, nullptr, nullptr, acc},
                             {(float*)gr.w2, s.F, nullptr, nullptr, nullptr, acc}};
    OASES_TRY(f32::launch_group(args, out, {true, false, false}, st));
  }
  return bias_grads(s, dpre, dy, gr, st);
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
  if (misaligned({wts->w1, wts->b1, wts->w2, wts->b2, x, resid, y, saved, workspace}, 16))
    return OASES_ERR_INVALID_ARG;
  const size_t need = layout(s, false).total;
  if (need > 0 && (!workspace || ws_bytes < need)) return OASES_ERR_WORKSPACE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  return api_end(fwd(s, *wts, x, resid, y, saved, ws, st));
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
                  grads->w2, grads->b2, workspace}, 16))
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
  return api_end(bwd(s, *wts, x, dy, saved, dx, *grads, ws, st));
}
