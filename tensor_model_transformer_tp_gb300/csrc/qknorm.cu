// Norms of queries and keys per head with the position rotation in the same
// pass (oases_qknorm.h), forward and backward.
//
// Each value is read once and written once (plus dy read in the backward), so
// the kernels are bound by HBM.  A head's D values lie in D / 8 lanes of a warp,
// 8 each (16 bytes of bf16), so a warp holds 32 / L heads at once, L the power of
// two not below D / 8; the sum of squares is a shuffle reduction over L lanes.  A
// warp's unit is up to HB heads of one token, all queries or all keys: the
// token's angles and the weight are loaded once per unit, folded into two factors
// per value, y_i = r (x_i A_i + x_partner B_i), and the unit's rows are in flight
// together.  The partner of value i in the rotation sits
//   PAIRS   beside it in the lane (interleaved),
//   LANES   rot / 2 values on, in another lane: the raw words are shuffled,
//   LOADS   at an offset that is no multiple of 8: loaded again, one by one.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "oases_qknorm.h"

namespace oases {
void api_begin();
oases_status api_end(cudaError_t e);

namespace {

enum class Partner { NONE, PAIRS, LANES, LOADS };
constexpr int WARPS = 8;
constexpr int BWD_CTAS_PER_SM = 4;

struct Tensor {
  const void* x;      // forward: input; backward: the same
  const void* dy;     // backward only
  void* out;          // forward: y; backward: dx (may be null)
  const void* w;      // weight or null
  int heads;
  int64_t xb, xs, xh;  // strides in elements
  int64_t yb, ys, yh;  // of out (forward), of dy (backward)
  int64_t ob, os, oh;  // of dx (backward)
};

struct QkArgs {
  Tensor t[2];  // queries, keys
  const float *cos, *sin;
  const int64_t* positions;
  int64_t pos_batch;  // elements between sequences in positions (0: shared)
  int positions_len;
  int seq, D, rot, L;
  int units[2];       // units per token
  int64_t tokens, total;
  float eps;
  float* part;        // backward: [blocks][2][D]
};

// Eight values of a row as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ Raw shuffled(int src, int width) const {
    Raw r;
    r.v = make_uint4(__shfl_sync(~0u, v.x, src, width), __shfl_sync(~0u, v.y, src, width),
                     __shfl_sync(~0u, v.z, src, width), __shfl_sync(~0u, v.w, src, width));
    return r;
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ Raw shuffled(int src, int width) const {
    Raw r;
    r.a = make_float4(__shfl_sync(~0u, a.x, src, width), __shfl_sync(~0u, a.y, src, width),
                      __shfl_sync(~0u, a.z, src, width), __shfl_sync(~0u, a.w, src, width));
    r.b = make_float4(__shfl_sync(~0u, b.x, src, width), __shfl_sync(~0u, b.y, src, width),
                      __shfl_sync(~0u, b.z, src, width), __shfl_sync(~0u, b.w, src, width));
    return r;
  }
};
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// A lane's place: its 8 values of a head, and where their partners are.
template <Partner P>
struct Place {
  int i0;        // first value
  bool active;
  int lane;      // LANES: the partner's lane within the head's
  __device__ __forceinline__ Place(const QkArgs& a) {
    const int c = threadIdx.x % a.L;
    i0 = 8 * c;
    active = i0 < a.D;
    const int half = a.rot / 2;
    lane = P != Partner::LANES || i0 >= a.rot ? c : i0 < half ? c + half / 8 : c - half / 8;
  }
  // partner of value i0 + e
  __device__ __forceinline__ int partner(const QkArgs& a, int e) const {
    const int i = i0 + e;
    if (i >= a.rot) return i;
    if (P == Partner::PAIRS) return i ^ 1;
    return i < a.rot / 2 ? i + a.rot / 2 : i - a.rot / 2;
  }
  // cos and signed sin of the lane's values: y_i = x_i c_i + x_partner s_i
  __device__ __forceinline__ void angles(const QkArgs& a, int64_t token, float (&c)[8], float (&s)[8]) const {
    if (P == Partner::NONE) {
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
      return;
    }
    const int64_t b = token / a.seq;
    const int t = (int)(token - b * a.seq);
    const int64_t p = a.positions ? a.positions[b * a.pos_batch + t] : t;
    const bool good = p >= 0 && p < a.positions_len;
    const int half = a.rot / 2;
    const float* ct = a.cos + (good ? p : 0) * half;
    const float* st = a.sin + (good ? p : 0) * half;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = i0 + e;
      c[e] = 1.f, s[e] = 0.f;
      if (i < a.rot) {
        const int at = P == Partner::PAIRS ? i / 2 : i < half ? i : i - half;
        const bool first = P == Partner::PAIRS ? (i & 1) == 0 : i < half;
        c[e] = good ? ct[at] : NAN;
        const float v = good ? st[at] : NAN;
        s[e] = first ? -v : v;
      }
    }
  }
  // the partners' values of a row whose own values are `raw`
  template <typename T>
  __device__ __forceinline__ void partners(const QkArgs& a, const Raw<T>& raw, const float (&x)[8],
                                           const T* row, bool valid, float (&o)[8]) const {
    if (P == Partner::PAIRS) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = x[e ^ 1];
    } else if (P == Partner::LANES) {
      raw.shuffled(lane, a.L).get(o);
    } else if (P == Partner::LOADS) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = valid && i0 + e < a.rot ? ld_elem(row, partner(a, e)) : 0.f;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 0.f;
    }
  }
};

__device__ __forceinline__ float lanes_sum(float v, int L) {
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Unit u: which token, tensor and first head.
struct Unit {
  int64_t token;
  int which, h0;
};
__device__ __forceinline__ Unit unit_of(const QkArgs& a, int64_t u, int heads_per_unit) {
  const int per = a.units[0] + a.units[1];
  Unit r;
  r.token = u / per;
  int k = (int)(u - r.token * per);
  r.which = k >= a.units[0];
  if (r.which) k -= a.units[0];
  r.h0 = k * heads_per_unit;
  return r;
}

constexpr int FWD_ROWS = 4, BWD_ROWS = 2;  // rows of one lane in flight

template <typename T, Partner P>
__global__ void __launch_bounds__(32 * WARPS)
qknorm_fwd_kernel(const __grid_constant__ QkArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t u = (int64_t)blockIdx.x * WARPS + threadIdx.x / 32;
  if (u >= a.total) return;
  const int groups = 32 / a.L, sub = threadIdx.x % 32 / a.L;
  const Unit un = unit_of(a, u, FWD_ROWS * groups);
  const Tensor& t = a.t[un.which];
  const Place<P> pl(a);
  const int64_t b = un.token / a.seq, tk = un.token - b * a.seq;
  const T* x = static_cast<const T*>(t.x) + b * t.xb + tk * t.xs;
  Raw<T> raw[FWD_ROWS];
  bool valid[FWD_ROWS];
#pragma unroll
  for (int k = 0; k < FWD_ROWS; ++k) {
    const int h = un.h0 + k * groups + sub;
    valid[k] = pl.active && h < t.heads;
    raw[k].zero();
    if (valid[k]) raw[k].load(x + h * t.xh + pl.i0);
  }
  float A[8], B[8];  // the factors of a value and of its partner
  pl.angles(a, un.token, A, B);
  if (t.w != nullptr && pl.active) {
    const T* w = static_cast<const T*>(t.w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      A[e] *= ld_elem(w, pl.i0 + e);
      if (P != Partner::NONE) B[e] *= ld_elem(w, pl.partner(a, e));
    }
  }
  T* y = static_cast<T*>(t.out) + b * t.yb + tk * t.ys;
#pragma unroll
  for (int k = 0; k < FWD_ROWS; ++k) {
    const int h = un.h0 + k * groups + sub;
    float v[8], o[8];
    raw[k].get(v);
    pl.partners(a, raw[k], v, x + h * t.xh, valid[k], o);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
    const float r = 1.f / sqrtf(lanes_sum(ss, a.L) / (float)a.D + a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = r * (P == Partner::NONE ? v[e] * A[e] : fmaf(o[e], B[e], v[e] * A[e]));
    __syncwarp();  // y may be x: a row's partners have been read
    if (valid[k]) put8(y + h * t.yh + pl.i0, v);
  }
}

template <typename T, Partner P>
__global__ void __launch_bounds__(32 * WARPS)
qknorm_bwd_kernel(const __grid_constant__ QkArgs a) {
  __shared__ float red[2][WARPS][256];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int groups = 32 / a.L, sub = lane / a.L;
  const Place<P> pl(a);
  float dw[2][8] = {};
  for (int64_t u = (int64_t)blockIdx.x * WARPS + warp; u < a.total; u += (int64_t)gridDim.x * WARPS) {
    const Unit un = unit_of(a, u, BWD_ROWS * groups);
    const Tensor& t = a.t[un.which];
    const int64_t b = un.token / a.seq, tk = un.token - b * a.seq;
    const T* x = static_cast<const T*>(t.x) + b * t.xb + tk * t.xs;
    const T* dy = static_cast<const T*>(t.dy) + b * t.yb + tk * t.ys;
    Raw<T> rx[BWD_ROWS], rg[BWD_ROWS];
    bool valid[BWD_ROWS];
#pragma unroll
    for (int k = 0; k < BWD_ROWS; ++k) {
      const int h = un.h0 + k * groups + sub;
      valid[k] = pl.active && h < t.heads;
      rx[k].zero();
      rg[k].zero();
      if (valid[k]) {
        rx[k].load(x + h * t.xh + pl.i0);
        rg[k].load(dy + h * t.yh + pl.i0);
      }
    }
    float c[8], s[8], w[8];
    pl.angles(a, un.token, c, s);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[e] = t.w != nullptr && pl.active ? ld_elem(static_cast<const T*>(t.w), pl.i0 + e) : 1.f;
    T* dx = t.out ? static_cast<T*>(t.out) + b * t.ob + tk * t.os : nullptr;
    float add[8] = {};
#pragma unroll
    for (int k = 0; k < BWD_ROWS; ++k) {
      const int h = un.h0 + k * groups + sub;
      float xv[8], gv[8], o[8];
      rx[k].get(xv);
      rg[k].get(gv);
      pl.partners(a, rg[k], gv, dy + h * t.yh, valid[k], o);
      float ss = 0.f, sg = 0.f, gw[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (P != Partner::NONE) gv[e] = fmaf(-s[e], o[e], gv[e] * c[e]);  // R^T dy
        gw[e] = gv[e] * w[e];
        ss = fmaf(xv[e], xv[e], ss);
        sg = fmaf(gw[e], xv[e], sg);
      }
      const float r = 1.f / sqrtf(lanes_sum(ss, a.L) / (float)a.D + a.eps);
      const float m = lanes_sum(sg, a.L) / (float)a.D * r * r;
      if (valid[k]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) add[e] = fmaf(gv[e], xv[e] * r, add[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) gw[e] = r * fmaf(-xv[e], m, gw[e]);
      __syncwarp();  // dx may be dy: a row's partners have been read
      if (valid[k] && dx != nullptr) put8(dx + h * t.oh + pl.i0, gw);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // (uniform per warp)
      if (un.which) dw[1][e] += add[e];
      else dw[0][e] += add[e];
    }
  }
  if (a.part == nullptr) return;
  // over the warp's head groups, then over the warps, in a fixed order
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      for (int o = a.L; o < 32; o <<= 1) dw[q][e] += __shfl_xor_sync(~0u, dw[q][e], o);
      if (lane < a.L && pl.active) red[q][warp][pl.i0 + e] = dw[q][e];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
    const int q = i / a.D, d = i - q * a.D;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += red[q][k][d];
    a.part[(int64_t)blockIdx.x * 2 * a.D + i] = v;
  }
}

// Weights' gradients: the blocks' partial rows in a fixed order, 32 columns of a
// block and 32 rows at a time.
__global__ void __launch_bounds__(1024)
qknorm_dw_kernel(const float* part, int blocks, int D, void* dwq, void* dwk, DType t, int accumulate) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * 32 + threadIdx.x % 32, r0 = threadIdx.x / 32;
  float v = 0.f;
  if (c < 2 * D)
    for (int r = r0; r < blocks; r += 32) v += part[(int64_t)r * 2 * D + c];
  red[r0][threadIdx.x % 32] = v;
  __syncthreads();
  if (r0 != 0 || c >= 2 * D) return;
  v = 0.f;
#pragma unroll
  for (int r = 0; r < 32; ++r) v += red[r][threadIdx.x];
  void* out = c < D ? dwq : dwk;
  const int64_t i = c < D ? c : c - D;
  if (out == nullptr) return;
  if (accumulate) v += static_cast<const float*>(out)[i];
  store_any(out, t, i, v);
}

bool strides_ok(const oases_strides& s, int64_t esize, int batch, int seq, int heads) {
  const int64_t v[3] = {s.batch, s.token, s.head};
  const int n[3] = {batch, seq, heads};
  if (batch == 0 || seq == 0 || heads == 0) return true;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (v[i] <= 0 || v[i] > (1ll << 36) || v[i] * esize % 16 != 0)) return false;
  return true;
}

oases_status qk_check(const oases_qknorm_desc* d, bool backward) {
  if (!d) return OASES_ERR_INVALID_ARG;
  if (d->dtype != OASES_F32 && d->dtype != OASES_BF16) return OASES_ERR_INVALID_ARG;
  if (d->batch < 0 || d->seq < 0 || d->heads < 0 || d->kv_heads < 0 || d->head_dim <= 0)
    return OASES_ERR_INVALID_ARG;
  if (d->rot < 0 || d->rot > d->head_dim || d->rot % 2 || d->positions_len < 0)
    return OASES_ERR_INVALID_ARG;
  if ((d->interleaved | d->positions_shared | d->accumulate) & ~1) return OASES_ERR_INVALID_ARG;
  if (d->grad_dtype != OASES_F32 && d->grad_dtype != d->dtype) return OASES_ERR_INVALID_ARG;
  if (d->accumulate && d->grad_dtype != OASES_F32) return OASES_ERR_INVALID_ARG;
  if (!(d->eps > 0.f) || !(d->eps < INFINITY)) return OASES_ERR_INVALID_ARG;
  if (d->head_dim % 8 != 0 || d->head_dim > 256) return OASES_ERR_UNSUPPORTED;
  if ((int64_t)d->batch * d->seq > 1 << 29 || std::max(d->heads, d->kv_heads) > 1 << 29)
    return OASES_ERR_UNSUPPORTED;
  const int64_t e = d->dtype == OASES_F32 ? 4 : 2;
  auto ok = [&](const oases_strides& s, int heads) { return strides_ok(s, e, d->batch, d->seq, heads); };
  if (!ok(d->q, d->heads) || !ok(d->k, d->kv_heads) || !ok(d->q_out, d->heads) ||
      !ok(d->k_out, d->kv_heads))
    return OASES_ERR_INVALID_ARG;
  if (backward && (!ok(d->dq, d->heads) || !ok(d->dk, d->kv_heads))) return OASES_ERR_INVALID_ARG;
  return OASES_OK;
}

// The parts of the launch that follow from the descriptor.
QkArgs qk_args(const oases_qknorm_desc* d, int rows) {
  QkArgs a = {};
  a.seq = std::max(d->seq, 1);
  a.D = d->head_dim;
  a.rot = d->rot;
  a.L = 1;
  while (8 * a.L < a.D) a.L *= 2;
  a.positions_len = d->positions_len;
  a.pos_batch = d->positions_shared ? 0 : d->seq;
  a.eps = d->eps;
  a.tokens = (int64_t)d->batch * d->seq;
  const int heads[2] = {d->heads, d->kv_heads}, per = rows * 32 / a.L;
  const oases_strides* x[2] = {&d->q, &d->k};
  const oases_strides* y[2] = {&d->q_out, &d->k_out};
  const oases_strides* o[2] = {&d->dq, &d->dk};
  for (int i = 0; i < 2; ++i) {
    Tensor& t = a.t[i];
    t.heads = heads[i];
    t.xb = x[i]->batch, t.xs = x[i]->token, t.xh = x[i]->head;
    t.yb = y[i]->batch, t.ys = y[i]->token, t.yh = y[i]->head;
    t.ob = o[i]->batch, t.os = o[i]->token, t.oh = o[i]->head;
    a.units[i] = (heads[i] + per - 1) / per;
  }
  a.total = a.tokens * (a.units[0] + a.units[1]);
  return a;
}

Partner partner_of(const oases_qknorm_desc* d) {
  if (d->rot == 0) return Partner::NONE;
  if (d->interleaved) return Partner::PAIRS;
  return d->rot % 16 == 0 ? Partner::LANES : Partner::LOADS;
}

int bwd_blocks(const QkArgs& a) {
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, current_device()) != cudaSuccess) sms = 0;
  return (int)std::min<int64_t>((a.total + WARPS - 1) / WARPS, BWD_CTAS_PER_SM * (sms > 0 ? sms : 152));
}

template <typename T, bool BWD>
cudaError_t launch(Partner p, const QkArgs& a, int blocks, cudaStream_t st) {
  void (*kern)(QkArgs) = nullptr;
  if (BWD)
    kern = p == Partner::NONE    ? qknorm_bwd_kernel<T, Partner::NONE>
           : p == Partner::PAIRS ? qknorm_bwd_kernel<T, Partner::PAIRS>
           : p == Partner::LANES ? qknorm_bwd_kernel<T, Partner::LANES>
                                 : qknorm_bwd_kernel<T, Partner::LOADS>;
  else
    kern = p == Partner::NONE    ? qknorm_fwd_kernel<T, Partner::NONE>
           : p == Partner::PAIRS ? qknorm_fwd_kernel<T, Partner::PAIRS>
           : p == Partner::LANES ? qknorm_fwd_kernel<T, Partner::LANES>
                                 : qknorm_fwd_kernel<T, Partner::LOADS>;
  return launch_pdl(kern, dim3(blocks), dim3(32 * WARPS), 0, st, a);
}

}  // namespace
}  // namespace oases

extern "C" size_t oases_qknorm_workspace_bytes(const oases_qknorm_desc* desc) {
  using namespace oases;
  if (qk_check(desc, false) != OASES_OK) return 0;
  const QkArgs a = qk_args(desc, BWD_ROWS);
  return a.total == 0 ? 0 : align256((size_t)bwd_blocks(a) * 2 * a.D * 4);
}

extern "C" oases_status oases_qknorm_fwd(const oases_qknorm_desc* desc, const void* q, const void* k,
                                         const float* cos, const float* sin,
                                         const int64_t* positions, const void* q_weight,
                                         const void* k_weight, void* q_out, void* k_out,
                                         void* stream) {
  using namespace oases;
  api_begin();
  const oases_status v = qk_check(desc, false);
  if (v != OASES_OK) return v;
  if (misaligned({q, k, q_weight, k_weight, q_out, k_out}, 16) || misaligned({cos, sin}, 4) ||
      misaligned({positions}, 8))
    return OASES_ERR_INVALID_ARG;
  QkArgs a = qk_args(desc, FWD_ROWS);
  if (a.total == 0) return OASES_OK;
  if ((desc->heads && (!q || !q_out)) || (desc->kv_heads && (!k || !k_out)) ||
      (desc->rot && (!cos || !sin)))
    return OASES_ERR_INVALID_ARG;
  if ((a.total + WARPS - 1) / WARPS > INT32_MAX) return OASES_ERR_UNSUPPORTED;
  a.t[0].x = q, a.t[0].out = q_out, a.t[0].w = q_weight;
  a.t[1].x = k, a.t[1].out = k_out, a.t[1].w = k_weight;
  a.cos = cos, a.sin = sin, a.positions = positions;
  const int blocks = (int)((a.total + WARPS - 1) / WARPS);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return api_end(desc->dtype == OASES_F32
                     ? launch<float, false>(partner_of(desc), a, blocks, st)
                     : launch<__nv_bfloat16, false>(partner_of(desc), a, blocks, st));
}

extern "C" oases_status oases_qknorm_bwd(const oases_qknorm_desc* desc, const void* q, const void* k,
                                         const void* dq_out, const void* dk_out, const float* cos,
                                         const float* sin, const int64_t* positions,
                                         const void* q_weight, const void* k_weight, void* dq,
                                         void* dk, void* dq_weight, void* dk_weight,
                                         void* workspace, size_t ws_bytes, void* stream) {
  using namespace oases;
  api_begin();
  const oases_status v = qk_check(desc, true);
  if (v != OASES_OK) return v;
  if (misaligned({q, k, dq_out, dk_out, q_weight, k_weight, dq, dk, dq_weight, dk_weight, workspace}, 16) ||
      misaligned({cos, sin}, 4) || misaligned({positions}, 8))
    return OASES_ERR_INVALID_ARG;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return OASES_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  QkArgs a = qk_args(desc, BWD_ROWS);
  if (a.total == 0) {  // sums over no rows
    if (desc->accumulate) return OASES_OK;
    const size_t n = (size_t)a.D * dtype_size(static_cast<DType>(desc->grad_dtype));
    cudaError_t e = cudaSuccess;
    if (dq_weight) e = cudaMemsetAsync(dq_weight, 0, n, st);
    if (dk_weight && e == cudaSuccess) e = cudaMemsetAsync(dk_weight, 0, n, st);
    return api_end(e);
  }
  if ((desc->heads && (!q || !dq_out)) || (desc->kv_heads && (!k || !dk_out)) ||
      (desc->rot && (!cos || !sin)))
    return OASES_ERR_INVALID_ARG;
  const int blocks = bwd_blocks(a);
  const bool weights = dq_weight || dk_weight;
  if (weights && (!workspace || ws_bytes < align256((size_t)blocks * 2 * a.D * 4)))
    return OASES_ERR_WORKSPACE;
  a.t[0].x = q, a.t[0].dy = dq_out, a.t[0].out = dq, a.t[0].w = q_weight;
  a.t[1].x = k, a.t[1].dy = dk_out, a.t[1].out = dk, a.t[1].w = k_weight;
  a.cos = cos, a.sin = sin, a.positions = positions;
  a.part = weights ? static_cast<float*>(workspace) : nullptr;
  cudaError_t e = desc->dtype == OASES_F32
                      ? launch<float, true>(partner_of(desc), a, blocks, st)
                      : launch<__nv_bfloat16, true>(partner_of(desc), a, blocks, st);
  if (e == cudaSuccess && weights)
    e = launch_pdl(qknorm_dw_kernel, dim3((2 * a.D + 31) / 32), dim3(1024), 0, st,
                   (const float*)a.part, blocks, a.D, dq_weight, dk_weight,
                   static_cast<DType>(desc->grad_dtype), desc->accumulate);
  return api_end(e);
}
