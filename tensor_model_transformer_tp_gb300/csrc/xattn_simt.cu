// Attention over keys of another length, CUDA cores: fp32, where the tensor cores'
// operand types would round the inputs.
//
// Tiles of 64 queries x 64 keys, 256 threads.  Thread (ty, tx) of 16 x 16 holds the
// scores of rows 4 ty .. + 3 and columns tx, tx + 16, tx + 32, tx + 48, and of an
// output tile the same rows and DP / 16 columns.  Tiles stand row by row in shared
// memory with 4 floats of padding, so that eight rows read at once (16 bytes each)
// fall into different banks; both kinds of product read 16 bytes per operand and
// 4 x 4 (scores) or 4 x 8 (outputs) FMAs from them.
#include <math.h>

#include <algorithm>

#include "xattn.cuh"

namespace oases {
namespace {
using namespace xattn;

constexpr int TQ = 64, NT = 256, PITCH_P = TQ + 4;

template <int DP>
constexpr int pitch() { return DP + 4; }

// rows [r0, r0 + 64) of a head into dst, zero from row `rows` and column D on
template <int DP>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int64_t stride, int r0, int rows, int D) {
  constexpr int C = DP / 4;
#pragma unroll 4
  for (int i = threadIdx.x; i < TQ * C; i += NT) {
    const int r = i / C, c = i % C * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < rows && c < D) v = *reinterpret_cast<const float4*>(src + (int64_t)(r0 + r) * stride + c);
    *reinterpret_cast<float4*>(dst + r * pitch<DP>() + c) = v;
  }
}

// s[i][j] = A row (4 ty + i) . B row (tx + 16 j)
template <int DP>
__device__ __forceinline__ void rows_product(float (&s)[4][4], const float* A, const float* B) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < DP; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * pitch<DP>() + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * pitch<DP>() + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
  }
}

// The columns of an output tile that thread tx holds: n of DP / 16.
template <int DP>
__device__ __forceinline__ int out_col(int tx, int n) {
  return DP == 32 ? 2 * tx + n : 4 * tx + (n & 3) + 64 * (n >> 2);
}
// acc[i][n] += sum over 64 of P[4 ty + i][k] V[k][column n]
template <int DP>
__device__ __forceinline__ void add_product(float (&acc)[4][DP / 16], const float* P, const float* V) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  constexpr int N = DP / 16;
#pragma unroll 2
  for (int k = 0; k < TQ; k += 4) {
    float p[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(P + (4 * ty + i) * PITCH_P + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      float v[N];
      const float* row = V + (k + kk) * pitch<DP>();
      if (DP == 32) {
        *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(row + 2 * tx);
      } else {
#pragma unroll
        for (int m = 0; m < N; m += 4)
          *reinterpret_cast<float4*>(v + m) = *reinterpret_cast<const float4*>(row + 4 * tx + 16 * m);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < N; ++n) acc[i][n] = fmaf(p[i][kk], v[n], acc[i][n]);
    }
  }
}
// over the 16 threads that share a row
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
template <int DP>
__device__ __forceinline__ void store_rows(float* out, int64_t stride, int r0, int rows, int D,
                                           const float (&acc)[4][DP / 16], const float (&f)[4]) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 4 * ty + i;
    if (r >= rows) continue;
    float* p = out + (int64_t)r * stride;
#pragma unroll
    for (int n = 0; n < DP / 16; ++n)
      if (const int c = out_col<DP>(tx, n); c < D) p[c] = acc[i][n] * f[i];
  }
}

// One CTA: 64 queries of one (sequence, head) and one share of its keys.
template <int DP>
__global__ void __launch_bounds__(NT)
xattn_fwd_simt_kernel(const __grid_constant__ Args a, int tiles) {
  extern __shared__ float4 smem_f4[];
  float* Qs = reinterpret_cast<float*>(smem_f4);
  float* Ks = Qs + TQ * pitch<DP>();
  float* Vs = Ks + TQ * pitch<DP>();
  float* Ps = Vs + TQ * pitch<DP>();
  pdl_wait();
  pdl_trigger();
  int64_t u = blockIdx.x;
  const int sp = (int)(u % a.splits);
  u /= a.splits;
  const int tile = tiles - 1 - (int)(u % tiles);  // causal: the longest first
  u /= tiles;
  const int h = (int)(u % a.H), b = (int)(u / a.H), g = h / a.share;
  const int len = a.len(b), p0 = a.start(b);
  const int q0 = tile * TQ, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int last = min(q0 + TQ, a.Sq) - 1;
  const int seen = a.causal ? min(len, max(0, p0 + last + 1)) : len;
  const int blocks = (seen + TQ - 1) / TQ, per = (blocks + a.splits - 1) / a.splits;
  const float* k = static_cast<const float*>(a.k) + b * a.sk.b + g * a.sk.h;
  const float* v = static_cast<const float*>(a.v) + b * a.sv.b + g * a.sv.h;
  load_tile<DP>(Qs, static_cast<const float*>(a.q) + b * a.sq.b + h * a.sq.h, a.sq.s, q0, a.Sq, a.D);
  float acc[4][DP / 16] = {}, m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
  for (int j = sp * per; j < min(blocks, (sp + 1) * per); ++j) {
    __syncthreads();
    load_tile<DP>(Ks, k, a.sk.s, j * TQ, len, a.D);
    load_tile<DP>(Vs, v, a.sv.s, j * TQ, len, a.D);
    __syncthreads();
    float s[4][4];
    rows_product<DP>(s, Qs, Ks);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = p0 + q0 + 4 * ty + i;
      const int vis = a.causal ? min(len, p + 1) : len;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int key = j * TQ + tx + 16 * c;
        s[i][c] *= a.scale;
        if (a.bias.buckets) s[i][c] += a.bias.clamped(h, key - p);
        if (key >= vis) s[i][c] = -INFINITY;
        mx = fmaxf(mx, s[i][c]);
      }
      mx = fmaxf(m[i], row_max(mx));
      const float ref = mx == -INFINITY ? 0.f : mx;  // no key so far: all weights 0
      const float f = expf(m[i] - ref);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float e = expf(s[i][c] - ref);
        sum += e;
        Ps[(4 * ty + i) * PITCH_P + tx + 16 * c] = e;
      }
      l[i] = l[i] * f + row_sum(sum);
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) acc[i][n] *= f;
    }
    __syncwarp();  // a row's weights are written and read by the same half warp
    add_product<DP>(acc, Ps, Vs);
  }
  float inv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    inv[i] = l[i] == 0.f ? 0.f : 1.f / l[i];
    const int qi = q0 + 4 * ty + i;
    if (tx == 0 && qi < a.Sq)
      (a.splits > 1 ? a.part_lse + (int64_t)sp * a.B * a.H * a.Sq : a.lse)[a.stat(b, h, qi)] =
          m[i] + logf(l[i]);
  }
  if (a.splits > 1)
    store_rows<DP>(a.part_o + (((int64_t)sp * a.B + b) * a.Sq * a.H + h) * a.D, (int64_t)a.H * a.D, q0, a.Sq,
                          a.D, acc, inv);
  else
    store_rows<DP>(static_cast<float*>(a.o) + b * a.so.b + h * a.so.h, a.so.s, q0, a.Sq, a.D, acc, inv);
}

// Rows' weights and score gradients from s and dP of a tile (both overwritten):
// element (i, c) belongs to key `key` and a query at position p whose statistics are
// lse and delta; visible says whether the key counts, and alone whether it is the query's
// only one, of weight 1: no gradient, not a rounding's.
__device__ __forceinline__ void weight_and_grad(float& s, float& dp, bool visible, bool alone, float lse, float delta) {
  const float w = visible ? expf(s - lse) : 0.f;
  dp = visible && !alone ? w * (dp - delta) : 0.f;
  s = w;
}

// dq (and delta, and the bias gradient's partial sums): one CTA per 64 queries.
template <int DP>
__global__ void __launch_bounds__(NT)
xattn_dq_simt_kernel(const __grid_constant__ Args a, int tiles) {
  extern __shared__ float4 smem_f4[];
  float* Qs = reinterpret_cast<float*>(smem_f4);
  float* Os = Qs + TQ * pitch<DP>();
  float* Ks = Os + TQ * pitch<DP>();
  float* Vs = Ks + TQ * pitch<DP>();
  float* Ds = Vs + TQ * pitch<DP>();
  __shared__ float delta[TQ], lse[TQ], diagonal[2 * TQ];
  pdl_wait();
  pdl_trigger();
  int64_t u = blockIdx.x;
  const int tile = tiles - 1 - (int)(u % tiles);
  u /= tiles;
  const int h = (int)(u % a.H), b = (int)(u / a.H), g = h / a.share;
  const int len = a.len(b), p0 = a.start(b);
  const int q0 = tile * TQ, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int last = min(q0 + TQ, a.Sq) - 1;
  const int seen = a.causal ? min(len, max(0, p0 + last + 1)) : len;
  const float* k = static_cast<const float*>(a.k) + b * a.sk.b + g * a.sk.h;
  const float* v = static_cast<const float*>(a.v) + b * a.sv.b + g * a.sv.h;
  const float* o = static_cast<const float*>(a.o) + b * a.so.b + h * a.so.h;
  const float* d_o = static_cast<const float*>(a.d_o) + b * a.sdo.b + h * a.sdo.h;
  load_tile<DP>(Qs, static_cast<const float*>(a.q) + b * a.sq.b + h * a.sq.h, a.sq.s, q0, a.Sq, a.D);
  load_tile<DP>(Os, d_o, a.sdo.s, q0, a.Sq, a.D);
  load_tile<DP>(Ks, o, a.so.s, q0, a.Sq, a.D);
  __syncthreads();
  {  // delta, four threads a row
    const int r = threadIdx.x / 4;
    float d = 0.f;
    for (int c = threadIdx.x % 4; c < DP; c += 4) d = fmaf(Os[r * pitch<DP>() + c], Ks[r * pitch<DP>() + c], d);
    d += __shfl_xor_sync(~0u, d, 1);
    d += __shfl_xor_sync(~0u, d, 2);
    if (threadIdx.x % 4 == 0) {
      delta[r] = d;
      const bool valid = q0 + r < a.Sq;
      if (valid) a.delta[a.stat(b, h, q0 + r)] = d;
      const float l = valid ? a.lse[a.stat(b, h, q0 + r)] : INFINITY;
      lse[r] = l < LSE_LOWEST ? INFINITY : l;  // a row without keys: every weight 0
    }
  }
  float acc[4][DP / 16] = {};
  float db = 0.f;  // thread t < buckets: the bias gradient's bucket t
  for (int j = 0; j * TQ < seen; ++j) {
    __syncthreads();
    load_tile<DP>(Ks, k, a.sk.s, j * TQ, len, a.D);
    load_tile<DP>(Vs, v, a.sv.s, j * TQ, len, a.D);
    __syncthreads();
    float s[4][4], dp[4][4];
    rows_product<DP>(s, Qs, Ks);
    rows_product<DP>(dp, Os, Vs);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i, p = p0 + q0 + r;
      const int vis = q0 + r >= a.Sq ? 0 : a.causal ? min(len, p + 1) : len;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int key = j * TQ + tx + 16 * c;
        s[i][c] *= a.scale;
        if (a.bias.buckets) s[i][c] += a.bias.clamped(h, key - p);
        weight_and_grad(s[i][c], dp[i][c], key < vis, vis == 1, lse[r], delta[r]);
        Ds[r * PITCH_P + tx + 16 * c] = dp[i][c];
      }
    }
    if (a.bias_part != nullptr) {
      // sums along the tile's 127 diagonals, then each bucket's run of them
      __syncthreads();
      if (threadIdx.x < 2 * TQ - 1) {
        const int d = (int)threadIdx.x - (TQ - 1);
        float x = 0.f;
        for (int r = max(0, -d); r < TQ - max(0, d); ++r) x += Ds[r * (PITCH_P + 1) + d];
        diagonal[threadIdx.x] = x;
      }
      __syncthreads();
      if (threadIdx.x < a.bias.buckets) {
        const int2 run = a.bias.range[threadIdx.x];
        const int n0 = j * TQ - (p0 + q0) - (TQ - 1);  // distance of diagonal 0
        const int64_t lo = (int64_t)run.x - n0, hi = (int64_t)run.y - n0;
        for (int x = (int)max((int64_t)0, lo); x <= (int)min((int64_t)(2 * TQ - 2), hi); ++x) db += diagonal[x];
      }
    } else {
      __syncwarp();
    }
    add_product<DP>(acc, Ds, Ks);
  }
  const float f[4] = {a.scale, a.scale, a.scale, a.scale};
  store_rows<DP>(static_cast<float*>(a.dq) + b * a.sdq.b + h * a.sdq.h, a.sdq.s, q0, a.Sq, a.D, acc, f);
  if (a.bias_part != nullptr && threadIdx.x < a.bias.buckets)
    a.bias_part[(((int64_t)h * a.B + b) * tiles + tile) * a.bias.buckets + threadIdx.x] = db;
}

// dk and dv: one CTA per 64 keys of one (sequence, key head), over its query heads.
template <int DP>
__global__ void __launch_bounds__(NT)
xattn_dkv_simt_kernel(const __grid_constant__ Args a, int tiles) {
  extern __shared__ float4 smem_f4[];
  float* Ks = reinterpret_cast<float*>(smem_f4);
  float* Vs = Ks + TQ * pitch<DP>();
  float* Qs = Vs + TQ * pitch<DP>();
  float* Os = Qs + TQ * pitch<DP>();
  float* Ps = Os + TQ * pitch<DP>();
  float* Ds = Ps + TQ * PITCH_P;
  __shared__ float delta[TQ], lse[TQ];
  pdl_wait();
  pdl_trigger();
  int64_t u = blockIdx.x;
  const int tile = (int)(u % tiles);
  u /= tiles;
  const int g = (int)(u % a.G), b = (int)(u / a.G);
  const int len = a.len(b), p0 = a.start(b);
  const int k0 = tile * TQ, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  load_tile<DP>(Ks, static_cast<const float*>(a.k) + b * a.sk.b + g * a.sk.h, a.sk.s, k0, len, a.D);
  load_tile<DP>(Vs, static_cast<const float*>(a.v) + b * a.sv.b + g * a.sv.h, a.sv.s, k0, len, a.D);
  float dk[4][DP / 16] = {}, dv[4][DP / 16] = {};
  // queries before the first that sees key k0 give nothing
  const int i0 = a.causal ? max(0, k0 - p0) / TQ : 0;
  const int end = k0 < len ? a.Sq : 0;
  for (int hh = 0; hh < a.share; ++hh) {
    const int h = g * a.share + hh;
    const float* q = static_cast<const float*>(a.q) + b * a.sq.b + h * a.sq.h;
    const float* d_o = static_cast<const float*>(a.d_o) + b * a.sdo.b + h * a.sdo.h;
    for (int i = i0; i * TQ < end; ++i) {
      __syncthreads();
      load_tile<DP>(Qs, q, a.sq.s, i * TQ, a.Sq, a.D);
      load_tile<DP>(Os, d_o, a.sdo.s, i * TQ, a.Sq, a.D);
      if (threadIdx.x < TQ) {
        const int qi = i * TQ + threadIdx.x;
        const float l = qi < a.Sq ? a.lse[a.stat(b, h, qi)] : INFINITY;
        lse[threadIdx.x] = l < LSE_LOWEST ? INFINITY : l;
        delta[threadIdx.x] = qi < a.Sq ? a.delta[a.stat(b, h, qi)] : 0.f;
      }
      __syncthreads();
      float s[4][4], dp[4][4];
      rows_product<DP>(s, Ks, Qs);
      rows_product<DP>(dp, Vs, Os);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int key = k0 + 4 * ty + r;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int x = tx + 16 * c, qi = i * TQ + x, p = p0 + qi;
          s[r][c] *= a.scale;
          if (a.bias.buckets) s[r][c] += a.bias.clamped(h, key - p);
          const bool visible = key < len && qi < a.Sq && (!a.causal || key <= p);
          weight_and_grad(s[r][c], dp[r][c], visible, len == 1 || (a.causal && p == 0), lse[x], delta[x]);
          Ps[(4 * ty + r) * PITCH_P + x] = s[r][c];
          Ds[(4 * ty + r) * PITCH_P + x] = dp[r][c];
        }
      }
      __syncwarp();
      add_product<DP>(dv, Ps, Os);
      add_product<DP>(dk, Ds, Qs);
    }
  }
  float fk[4], fv[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const bool in = k0 + 4 * ty + r < len;
    fk[r] = in ? a.scale : 0.f, fv[r] = in ? 1.f : 0.f;
    if (!in)  // nothing of what stands behind the sequence's keys
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) dk[r][n] = dv[r][n] = 0.f;
  }
  store_rows<DP>(static_cast<float*>(a.dk) + b * a.sdk.b + g * a.sdk.h, a.sdk.s, k0, a.Sk, a.D, dk, fk);
  store_rows<DP>(static_cast<float*>(a.dv) + b * a.sdv.b + g * a.sdv.h, a.sdv.s, k0, a.Sk, a.D, dv, fv);
}

template <int DP>
constexpr int smem(int tiles, int square) {
  return (tiles * TQ * pitch<DP>() + square * TQ * PITCH_P) * 4;
}

template <int DP>
cudaError_t fwd(const Args& a, cudaStream_t st) {
  const int tiles = (a.Sq + TQ - 1) / TQ;
  const int64_t n = (int64_t)a.B * a.H * tiles * a.splits;
  if (n > INT32_MAX) return cudaErrorInvalidConfiguration;
  static DeviceOnce attr;
  OASES_TRY(attr.run([] {
    return cudaFuncSetAttribute(xattn_fwd_simt_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem<DP>(3, 1));
  }));
  return launch_pdl(xattn_fwd_simt_kernel<DP>, dim3((unsigned)n), dim3(NT), smem<DP>(3, 1), st, a, tiles);
}
template <int DP>
cudaError_t bwd(const Args& a, cudaStream_t st) {
  const int qt = (a.Sq + TQ - 1) / TQ, kt = (a.Sk + TQ - 1) / TQ;
  const int64_t nq = (int64_t)a.B * a.H * qt, nk = (int64_t)a.B * a.G * kt;
  if (nq > INT32_MAX || nk > INT32_MAX) return cudaErrorInvalidConfiguration;
  static DeviceOnce attr;
  OASES_TRY(attr.run([] {
    cudaError_t e = cudaFuncSetAttribute(xattn_dq_simt_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem<DP>(4, 1));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(xattn_dkv_simt_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem<DP>(4, 2));
  }));
  OASES_TRY(launch_pdl(xattn_dq_simt_kernel<DP>, dim3((unsigned)nq), dim3(NT), smem<DP>(4, 1), st, a, qt));
  if (nk == 0) return cudaSuccess;
  return launch_pdl(xattn_dkv_simt_kernel<DP>, dim3((unsigned)nk), dim3(NT), smem<DP>(4, 2), st, a, kt);
}

}  // namespace

cudaError_t xattn_fwd_f32(const Args& a, cudaStream_t st) {
  return a.D <= 32 ? fwd<32>(a, st) : a.D <= 64 ? fwd<64>(a, st) : fwd<128>(a, st);
}
cudaError_t xattn_bwd_f32(const Args& a, cudaStream_t st) {
  return a.D <= 32 ? bwd<32>(a, st) : a.D <= 64 ? bwd<64>(a, st) : bwd<128>(a, st);
}

}  // namespace oases
