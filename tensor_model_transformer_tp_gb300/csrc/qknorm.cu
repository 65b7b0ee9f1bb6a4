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
//   HALVES  rot / 2 values on (rot a multiple of 8): a lane of the rotated part holds four
//           values of its first half and their four partners,
//   LOADS   rot / 2 values on, otherwise: loaded again, one by one.
// Arithmetic goes two values at a time.  8192 tokens of 20 + 20 heads of 128, forward and
// backward (420 MB): 88 us; with the partners' words shuffled from other lanes, values one
// by one and IEEE roots and quotients, which issuing bound, 121.  (Persistent warps with
// the loads ahead in shared memory read as much at once with fewer warps, and took 98.)
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "oases_qknorm.h"

namespace oases {
void api_begin();
oases_status api_end(cudaError_t e);

namespace {

enum class Partner { NONE, PAIRS, HALVES, LOADS };
constexpr int WARPS = 8;
constexpr int BWD_CTAS_PER_SM = 2;

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
  int tables16;       // cos and sin are 16-byte aligned
  int batches;        // of rows in flight that a unit goes through
  int seq, D, rot, L;
  int units[2];       // units per token
  int64_t tokens, total;
  float eps;
  int q_blocks;       // backward: blocks that go through the queries, the others the keys
  float* part;        // backward: [blocks][D]
};

// Eight values of a row as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  // four values each
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
    const uint2 x = *reinterpret_cast<const uint2*>(p), y = *reinterpret_cast<const uint2*>(q);
    v = make_uint4(x.x, x.y, y.x, y.y);
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void load(const float* p, const float* q) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(q);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};
__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}
__device__ __forceinline__ void put8(__nv_bfloat16* p, __nv_bfloat16* q, const float (&f)[8]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]));
  *reinterpret_cast<uint2*>(q) = make_uint2(bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}
__device__ __forceinline__ void put8(float* p, float* q, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(q) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void put8(float* p, const float (&f)[8]) { put8(p, p + 4, f); }

// 1 / sqrt(x) of x > 0: the hardware's, and one step of Newton's on it (e = (1 - x r^2) / 2).
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x), e = fmaf(-0.5f * x * r, r, 0.5f);
  return r == 0.f ? r : fmaf(r, e, r);  // (x infinite: 0)
}
__device__ __forceinline__ uint64_t pair(const float (&f)[8], int e) { return f2_pack(f[e], f[e + 1]); }
__device__ __forceinline__ void set_pair(float (&f)[8], int e, uint64_t v) { f[e] = f2_lo(v), f[e + 1] = f2_hi(v); }
__device__ __forceinline__ float dot8(const float (&f)[8], const float (&g)[8]) {
  uint64_t s = f2_mul(pair(f, 0), pair(g, 0));
#pragma unroll
  for (int e = 2; e < 8; e += 2) s = f2_fma(pair(f, e), pair(g, e), s);
  return f2_lo(s) + f2_hi(s);
}

// A lane's place: its 8 values of a head, from i0 and from i1 on.
template <Partner P>
struct Place {
  int i0, i1;
  bool active, turned;  // turned: in two halves (HALVES: of the rotated part; NONE: of the head)
  __device__ __forceinline__ Place(const QkArgs& a) {
    const int c = threadIdx.x % a.L;
    active = 8 * c < a.D;
    const int part = P == Partner::HALVES ? a.rot : P == Partner::NONE ? a.D : 0;
    turned = 8 * c < part;
    i0 = turned ? 4 * c : 8 * c;
    i1 = i0 + (turned ? part / 2 : 4);
  }
  __device__ __forceinline__ int index(int e) const { return e < 4 ? i0 + e : i1 + e - 4; }
  template <typename T>
  __device__ __forceinline__ void load(const T* row, Raw<T>& r) const {
    if (P == Partner::HALVES || P == Partner::NONE) r.load(row + i0, row + i1);
    else r.load(row + i0);
  }
  template <typename T>
  __device__ __forceinline__ void get(const T* row, float (&f)[8]) const {
    Raw<T> r;
    load(row, r);
    r.get(f);
  }
  template <typename T>
  __device__ __forceinline__ void put(T* row, const float (&f)[8]) const {
    if (P == Partner::HALVES || P == Partner::NONE) put8(row + i0, row + i1, f);
    else put8(row + i0, f);
  }
  // LOADS: the partner of value e
  __device__ __forceinline__ int partner(const QkArgs& a, int e) const {
    const int i = i0 + e;
    if (i >= a.rot) return i;
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
    if constexpr (P == Partner::HALVES) {
      float u[4] = {1.f, 1.f, 1.f, 1.f}, v[4] = {};
      if (turned) {
        if (a.tables16) {
          *reinterpret_cast<float4*>(u) = *reinterpret_cast<const float4*>(ct + i0);
          *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(st + i0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) u[e] = ct[i0 + e], v[e] = st[i0 + e];
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (turned && !good) u[e] = v[e] = NAN;
        c[e] = c[e + 4] = u[e];
        s[e] = -v[e], s[e + 4] = v[e];
      }
    } else {
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
  }
  template <typename T>
  __device__ __forceinline__ void partner_weights(const QkArgs& a, const T* w, const float (&own)[8],
                                                  float (&o)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      o[e] = P == Partner::PAIRS    ? own[e ^ 1]
             : P == Partner::HALVES ? own[e ^ 4]
             : P == Partner::LOADS  ? ld_elem(w, partner(a, e))
                                    : 0.f;
  }
  // the partners' values of a row whose own values are x
  template <typename T>
  __device__ __forceinline__ void partners(const QkArgs& a, const float (&x)[8], const T* row, bool valid,
                                           float (&o)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      o[e] = P == Partner::PAIRS    ? x[e ^ 1]
             : P == Partner::HALVES ? x[e ^ 4]
             : P == Partner::LOADS  ? (valid && i0 + e < a.rot ? ld_elem(row, partner(a, e)) : 0.f)
                                    : 0.f;
  }
};

// Sums over the L lanes of a head (a power of two): every step a predicate, no loop.
template <int N>
__device__ __forceinline__ void lanes_sum(int L, float (&v)[N]) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    if (L > o) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(~0u, v[i], o);
    }
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

// rows of one lane in flight: what the registers hold
// (20 heads of 128 are two batches of 5 rows; three of 4 took 104 us, forward and backward,
// against 90.  Of other counts some rows are empty: from a cold L2, 8192 tokens, the forward and
// the backward of 20 + 20 heads read and write at 4.2 and 4.0 TB/s, of 16 + 16 at 3.7 and 3.6,
// of 32 + 32 at 4.6 and 4.4, of 32 + 8 at 3.3 and 3.0)
constexpr int rows_in_flight(bool bwd, bool f32, Partner p) {
  return p == Partner::LOADS || (bwd && f32) ? 2 : f32 ? 4 : 5;
}

template <typename T, Partner P>
__global__ void __launch_bounds__(32 * WARPS, 3)
qknorm_fwd_kernel(const __grid_constant__ QkArgs a) {
  constexpr int ROWS = rows_in_flight(false, sizeof(T) == 4, P);
  pdl_wait();
  pdl_trigger();
  const int64_t u = (int64_t)blockIdx.x * WARPS + threadIdx.x / 32;
  if (u >= a.total) return;
  const int groups = 32 / a.L, sub = threadIdx.x % 32 / a.L;
  const Unit un = unit_of(a, u, ROWS * groups * a.batches);
  const Tensor& t = a.t[un.which];
  const Place<P> pl(a);
  const int64_t b = un.token / a.seq, tk = un.token - b * a.seq;
  // the lane's first row, and from one to the next
  const T* x = static_cast<const T*>(t.x) + b * t.xb + tk * t.xs + (un.h0 + sub) * t.xh;
  T* y = static_cast<T*>(t.out) + b * t.yb + tk * t.ys + (un.h0 + sub) * t.yh;
  const int64_t x_step = groups * t.xh, y_step = groups * t.yh;
  const float over_d = 1.f / (float)a.D;
  float A[8], B[8];  // the factors of a value and of its partner
  Raw<T> raw[ROWS];
  const T* next = x;  // the next row to load
  auto load = [&](int batch) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int h = un.h0 + (batch * ROWS + k) * groups + sub;
      raw[k].zero();
      if (pl.active && h < t.heads) pl.load(next, raw[k]);
      next += x_step;
    }
  };
  load(0);
  pl.angles(a, un.token, A, B);
  if (t.w != nullptr && pl.active) {
    const T* w = static_cast<const T*>(t.w);
    float own[8], other[8];
    pl.get(w, own);
    pl.template partner_weights<T>(a, w, own, other);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      A[e] *= own[e];
      if (P != Partner::NONE) B[e] *= other[e];
    }
  }
  for (int batch = 0; batch < a.batches && un.h0 + batch * ROWS * groups < t.heads; ++batch) {
    if (batch) load(batch);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int h = un.h0 + (batch * ROWS + k) * groups + sub;
      if (h - sub >= t.heads) break;  // (uniform: none of the warp's)
      const bool valid = pl.active && h < t.heads;
      float v[8], o[8];
      raw[k].get(v);
      pl.partners(a, v, x, valid, o);
      float ss[1] = {dot8(v, v)};
      lanes_sum(a.L, ss);
      const uint64_t r2 = f2_splat(inverse_root(fmaf(ss[0], over_d, a.eps)));
      float y8[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        uint64_t z = f2_mul(pair(v, e), pair(A, e));
        if (P != Partner::NONE) z = f2_fma(pair(o, e), pair(B, e), z);
        set_pair(y8, e, f2_mul(z, r2));
      }
      __syncwarp();  // y may be x: a row's partners have been read
      if (valid) pl.put(y, y8);
      x += x_step;
      y += y_step;
    }
  }
}

template <typename T, Partner P>
__global__ void __launch_bounds__(32 * WARPS, 2)
qknorm_bwd_kernel(const __grid_constant__ QkArgs a) {
  constexpr int ROWS = rows_in_flight(true, sizeof(T) == 4, P);
  __shared__ float red[WARPS][256];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int groups = 32 / a.L, sub = lane / a.L;
  const Place<P> pl(a);
  const float over_d = 1.f / (float)a.D;
  const int which = (int)blockIdx.x >= a.q_blocks;
  const int first = which ? a.q_blocks : 0, blocks = which ? gridDim.x - a.q_blocks : a.q_blocks;
  const Tensor& t = a.t[which];
  float dw[8] = {};
  for (int64_t u = (int64_t)(blockIdx.x - first) * WARPS + warp; u < a.tokens * a.units[which];
       u += (int64_t)blocks * WARPS) {
    const int64_t token = u / a.units[which];
    const int h0 = (int)(u - token * a.units[which]) * ROWS * groups * a.batches;
    const int64_t b = token / a.seq, tk = token - b * a.seq;
    const T* x = static_cast<const T*>(t.x) + b * t.xb + tk * t.xs + (h0 + sub) * t.xh;  // next to load
    const T* dy = static_cast<const T*>(t.dy) + b * t.yb + tk * t.ys + (h0 + sub) * t.yh;
    const T* dy_row = dy;  // in work
    float c[8], s[8], w[8];
    Raw<T> rx[ROWS], rg[ROWS];
    auto load = [&](int batch) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const int h = h0 + (batch * ROWS + k) * groups + sub;
        rx[k].zero();
        rg[k].zero();
        if (pl.active && h < t.heads) {
          pl.load(x, rx[k]);
          pl.load(dy, rg[k]);
        }
        x += groups * t.xh;
        dy += groups * t.yh;
      }
    };
    load(0);
    pl.angles(a, token, c, s);
    if (t.w != nullptr && pl.active) {
      pl.get(static_cast<const T*>(t.w), w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.f;
    }
    T* dx = static_cast<T*>(t.out);
    if (dx != nullptr) dx += b * t.ob + tk * t.os + (h0 + sub) * t.oh;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = -s[e];  // of R^T
    for (int batch = 0; batch < a.batches && h0 + batch * ROWS * groups < t.heads; ++batch) {
      if (batch) load(batch);
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const int h = h0 + (batch * ROWS + k) * groups + sub;
        if (h - sub >= t.heads) break;  // (uniform: none of the warp's)
        const bool valid = pl.active && h < t.heads;
        float xv[8], gv[8], o[8], gw[8];
        rx[k].get(xv);
        rg[k].get(gv);
        pl.partners(a, gv, dy_row, valid, o);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          if (P != Partner::NONE)  // R^T dy
            set_pair(gv, e, f2_fma(pair(o, e), pair(s, e), f2_mul(pair(gv, e), pair(c, e))));
          set_pair(gw, e, f2_mul(pair(gv, e), pair(w, e)));
        }
        float sums[2] = {dot8(xv, xv), dot8(gw, xv)};
        lanes_sum(a.L, sums);
        const float r = inverse_root(fmaf(sums[0], over_d, a.eps));
        const uint64_t r2 = f2_splat(r), m2 = f2_splat(-(sums[1] * over_d * r * r));
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const uint64_t d = f2_fma(pair(gv, e), f2_mul(pair(xv, e), r2), pair(dw, e));
          set_pair(dw, e, d);  // (0 of a lane without a row, but in a token that is NaN anyway)
          set_pair(gw, e, f2_mul(f2_fma(pair(xv, e), m2, pair(gw, e)), r2));
        }
        __syncwarp();  // dx may be dy: a row's partners have been read
        if (t.out != nullptr) {
          if (valid) pl.put(dx, gw);
          dx += groups * t.oh;
        }
        if (P == Partner::LOADS) dy_row += groups * t.yh;
      }
    }
  }
  if (a.part == nullptr) return;
  // over the warp's head groups, then over the warps, in a fixed order
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    for (int o = a.L; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(~0u, dw[e], o);
    if (lane < a.L && pl.active) red[warp][pl.index(e)] = dw[e];
  }
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += red[k][d];
    a.part[(int64_t)blockIdx.x * a.D + d] = v;
  }
}

// Weights' gradients: the blocks' partial rows in a fixed order, 32 columns of a
// block and 32 rows at a time.
__global__ void __launch_bounds__(1024)
qknorm_dw_kernel(const float* part, int q_blocks, int blocks, int D, void* dwq, void* dwk, DType t,
                 int accumulate) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * 32 + threadIdx.x % 32, r0 = threadIdx.x / 32;
  const int last = blockIdx.y ? blocks : q_blocks;
  float v = 0.f;
  if (c < D)
    for (int r = (blockIdx.y ? q_blocks : 0) + r0; r < last; r += 32) v += part[(int64_t)r * D + c];
  red[r0][threadIdx.x % 32] = v;
  __syncthreads();
  void* out = blockIdx.y ? dwk : dwq;
  if (r0 != 0 || c >= D || out == nullptr) return;
  v = 0.f;
#pragma unroll
  for (int r = 0; r < 32; ++r) v += red[r][threadIdx.x];
  if (accumulate) v += static_cast<const float*>(out)[c];
  store_any(out, t, c, v);
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

Partner partner_of(const oases_qknorm_desc* d) {
  if (d->rot == 0) return Partner::NONE;
  if (d->interleaved) return Partner::PAIRS;
  return d->rot % 8 == 0 ? Partner::HALVES : Partner::LOADS;
}

// The parts of the launch that follow from the descriptor.
QkArgs qk_args(const oases_qknorm_desc* d, bool bwd) {
  QkArgs a = {};
  const int rows = rows_in_flight(bwd, d->dtype == OASES_F32, partner_of(d));
  a.seq = std::max(d->seq, 1);
  a.D = d->head_dim;
  a.rot = d->rot;
  a.L = 1;
  while (8 * a.L < a.D) a.L *= 2;
  a.positions_len = d->positions_len;
  a.pos_batch = d->positions_shared ? 0 : d->seq;
  a.eps = d->eps;
  a.tokens = (int64_t)d->batch * d->seq;
  // a unit goes through all of its token's heads where the tokens alone fill the GPU (64
  // warps an SM), so that the angles and weights are loaded once; through one batch of
  // rows in flight where they do not
  const int heads[2] = {d->heads, d->kv_heads}, batch = rows * 32 / a.L;
  const int most = std::max(1, (std::max(heads[0], heads[1]) + batch - 1) / batch);
  a.batches = 1;
  while (a.batches < most && a.tokens * 2 * (most / (a.batches + 1)) >= 64ll * sm_count()) ++a.batches;
  const int per = batch * a.batches;
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

// Blocks of the backward, and how many of them go through the queries: in proportion.
int bwd_blocks(const QkArgs& a, int* q_blocks) {
  const int64_t u[2] = {a.tokens * a.units[0], a.tokens * a.units[1]};
  const int64_t need[2] = {(u[0] + WARPS - 1) / WARPS, (u[1] + WARPS - 1) / WARPS};
  const int64_t most = BWD_CTAS_PER_SM * sm_count();
  if (need[0] + need[1] <= most) {
    *q_blocks = (int)need[0];
    return (int)(need[0] + need[1]);
  }
  const int64_t q = most * u[0] / (u[0] + u[1]);
  *q_blocks = (int)std::max<int64_t>(need[0] > 0, std::min<int64_t>(q, most - (need[1] > 0)));
  return (int)most;
}

template <typename T, bool BWD>
cudaError_t launch(Partner p, const QkArgs& a, int blocks, cudaStream_t st) {
  void (*kern)(QkArgs) = nullptr;
  if (BWD)
    kern = p == Partner::NONE    ? qknorm_bwd_kernel<T, Partner::NONE>
           : p == Partner::PAIRS ? qknorm_bwd_kernel<T, Partner::PAIRS>
           : p == Partner::HALVES ? qknorm_bwd_kernel<T, Partner::HALVES>
                                 : qknorm_bwd_kernel<T, Partner::LOADS>;
  else
    kern = p == Partner::NONE    ? qknorm_fwd_kernel<T, Partner::NONE>
           : p == Partner::PAIRS ? qknorm_fwd_kernel<T, Partner::PAIRS>
           : p == Partner::HALVES ? qknorm_fwd_kernel<T, Partner::HALVES>
                                 : qknorm_fwd_kernel<T, Partner::LOADS>;
  return launch_pdl(kern, dim3(blocks), dim3(32 * WARPS), 0, st, a);
}

}  // namespace
}  // namespace oases

extern "C" size_t oases_qknorm_workspace_bytes(const oases_qknorm_desc* desc) {
  using namespace oases;
  if (qk_check(desc, false) != OASES_OK) return 0;
  const QkArgs a = qk_args(desc, true);
  int q_blocks;
  return a.total == 0 ? 0 : align256((size_t)bwd_blocks(a, &q_blocks) * a.D * 4);
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
  QkArgs a = qk_args(desc, false);
  if (a.total == 0) return OASES_OK;
  if ((desc->heads && (!q || !q_out)) || (desc->kv_heads && (!k || !k_out)) ||
      (desc->rot && (!cos || !sin)))
    return OASES_ERR_INVALID_ARG;
  if ((a.total + WARPS - 1) / WARPS > INT32_MAX) return OASES_ERR_UNSUPPORTED;
  a.t[0].x = q, a.t[0].out = q_out, a.t[0].w = q_weight;
  a.t[1].x = k, a.t[1].out = k_out, a.t[1].w = k_weight;
  a.cos = cos, a.sin = sin, a.positions = positions, a.tables16 = !misaligned({cos, sin}, 16);
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
  QkArgs a = qk_args(desc, true);
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
  const int blocks = bwd_blocks(a, &a.q_blocks);
  const bool weights = dq_weight || dk_weight;
  if (weights && (!workspace || ws_bytes < align256((size_t)blocks * a.D * 4)))
    return OASES_ERR_WORKSPACE;
  a.t[0].x = q, a.t[0].dy = dq_out, a.t[0].out = dq, a.t[0].w = q_weight;
  a.t[1].x = k, a.t[1].dy = dk_out, a.t[1].out = dk, a.t[1].w = k_weight;
  a.cos = cos, a.sin = sin, a.positions = positions, a.tables16 = !misaligned({cos, sin}, 16);
  a.part = weights ? static_cast<float*>(workspace) : nullptr;
  cudaError_t e = desc->dtype == OASES_F32
                      ? launch<float, true>(partner_of(desc), a, blocks, st)
                      : launch<__nv_bfloat16, true>(partner_of(desc), a, blocks, st);
  if (e == cudaSuccess && weights)
    e = launch_pdl(qknorm_dw_kernel, dim3((a.D + 31) / 32, 2), dim3(1024), 0, st,
                   (const float*)a.part, a.q_blocks, blocks, a.D, dq_weight, dk_weight,
                   static_cast<DType>(desc->grad_dtype), desc->accumulate);
  return api_end(e);
}
