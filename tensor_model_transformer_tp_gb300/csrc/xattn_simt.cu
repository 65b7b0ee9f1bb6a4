// Attention over keys of another length, CUDA cores: fp32, where the tensor cores'
// operand types would round the inputs.
//
// A CTA of 256 threads keeps a tile of TR = 64 or 32 rows (queries; keys for dk and dv) and
// goes through blocks of 64 of the other side, the next block on its way to shared memory
// while one is worked on.  Thread (ty, tx) of 16 x 16 holds the scores of RI = TR / 16 rows
// from RI ty on and of columns tx, tx + 16, tx + 32, tx + 48, and of an output tile the same
// rows and DP / 16 columns.  Tiles stand row by row in shared memory with 4 floats of
// padding, so that eight rows read at once (16 bytes each) fall into different banks.  At
// RI = 4 both kinds of product are bound by the FMAs (16 clocks of them a warp against 12 of
// reads), at RI = 2 by the reads (10 against 8): 32 rows are for grids that would leave SMs
// idle (2 sequences of 130, 6 heads of 64, forward and backward: 86 -> 68 us).
#include <math.h>

#include <algorithm>

#include "xattn.cuh"

namespace oases {
namespace {
using namespace xattn;

constexpr int TB = 64, NT = 256, PITCH_P = TB + 4;

template <int DP>
constexpr int pitch() { return DP + 4; }

// rows [r0, r0 + ROWS) of a head into dst, zero from row `rows` and column D on
template <int DP, int ROWS>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int64_t stride, int r0, int rows, int D) {
  constexpr int C = DP / 4;
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
#pragma unroll 4
  for (int i = threadIdx.x; i < ROWS * C; i += NT) {
    const int r = i / C, c = i % C * 4;
    const bool in = r0 + r < rows && c < D;
    const float* from = in ? src + (int64_t)(r0 + r) * stride + c : src;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (r * pitch<DP>() + c) * 4), "l"(from),
                 "r"(in ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void loads_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>  // all but the last LEFT groups have landed
__device__ __forceinline__ void loads_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// s[i][j] = A row (RI ty + i) . B row (tx + 16 j)
template <int DP, int RI>
__device__ __forceinline__ void rows_product(float (&s)[RI][4], const float* A, const float* B) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < DP; d += 4) {
    float4 x[RI], y[4];
#pragma unroll
    for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4*>(A + (RI * ty + i) * pitch<DP>() + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * pitch<DP>() + d);
#pragma unroll
    for (int i = 0; i < RI; ++i)
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
// acc[i][n] += sum over 64 of P[RI ty + i][k] V[k][column n]
template <int DP, int RI>
__device__ __forceinline__ void add_product(float (&acc)[RI][DP / 16], const float* P, const float* V) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  constexpr int N = DP / 16;
#pragma unroll 2
  for (int k = 0; k < TB; k += 4) {
    float p[RI][4];
#pragma unroll
    for (int i = 0; i < RI; ++i)
      *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(P + (RI * ty + i) * PITCH_P + k);
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
      for (int i = 0; i < RI; ++i)
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
template <int DP, int RI>
__device__ __forceinline__ void store_rows(float* out, int64_t stride, int r0, int rows, int D,
                                           const float (&acc)[RI][DP / 16], const float (&f)[RI]) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = r0 + RI * ty + i;
    if (r >= rows) continue;
    float* p = out + (int64_t)r * stride;
#pragma unroll
    for (int n = 0; n < DP / 16; ++n)
      if (const int c = out_col<DP>(tx, n); c < D) p[c] = acc[i][n] * f[i];
  }
}

// One CTA: TR queries of one (sequence, head) and one share of its keys.
template <int DP, int RI>
__global__ void __launch_bounds__(NT)
xattn_fwd_simt_kernel(const __grid_constant__ Args a, int tiles) {
  constexpr int TR = 16 * RI, BLOCK = TB * pitch<DP>();
  extern __shared__ float4 smem_f4[];
  float* Qs = reinterpret_cast<float*>(smem_f4);
  float* Ks = Qs + TR * pitch<DP>();  // [2][K | V]
  float* Ps = Ks + 4 * BLOCK;
  pdl_wait();
  pdl_trigger();
  int64_t u = blockIdx.x;
  const int sp = (int)(u % a.splits);
  u /= a.splits;
  const int tile = tiles - 1 - (int)(u % tiles);  // causal: the longest first
  u /= tiles;
  const int h = (int)(u % a.H), b = (int)(u / a.H), g = h / a.share;
  const int len = a.len(b), p0 = a.start(b);
  const int q0 = tile * TR, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int last = min(q0 + TR, a.Sq) - 1;
  const int seen = a.causal ? min(len, max(0, p0 + last + 1)) : len;
  const int blocks = (seen + TB - 1) / TB, per = (blocks + a.splits - 1) / a.splits;
  const int j0 = sp * per, j1 = min(blocks, j0 + per);
  const float* k = static_cast<const float*>(a.k) + b * a.sk.b + g * a.sk.h;
  const float* v = static_cast<const float*>(a.v) + b * a.sv.b + g * a.sv.h;
  auto load = [&](int j) {
    float* to = Ks + ((j - j0) & 1) * 2 * BLOCK;
    if (j < j1) {
      load_tile<DP, TB>(to, k, a.sk.s, j * TB, len, a.D);
      load_tile<DP, TB>(to + BLOCK, v, a.sv.s, j * TB, len, a.D);
    }
    loads_commit();
  };
  load_tile<DP, TR>(Qs, static_cast<const float*>(a.q) + b * a.sq.b + h * a.sq.h, a.sq.s, q0, a.Sq, a.D);
  load(j0);
  float acc[RI][DP / 16] = {}, m[RI], l[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) m[i] = -INFINITY, l[i] = 0.f;
  for (int j = j0; j < j1; ++j) {
    load(j + 1);
    loads_wait<1>();
    __syncthreads();
    const float* K = Ks + ((j - j0) & 1) * 2 * BLOCK;
    float s[RI][4];
    rows_product<DP, RI>(s, Qs, K);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int p = p0 + q0 + RI * ty + i;
      const int vis = a.causal ? min(len, p + 1) : len;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int key = j * TB + tx + 16 * c;
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
        Ps[(RI * ty + i) * PITCH_P + tx + 16 * c] = e;
      }
      l[i] = l[i] * f + row_sum(sum);
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) acc[i][n] *= f;
    }
    __syncwarp();  // a row's weights are written and read by the same half warp
    add_product<DP, RI>(acc, Ps, K + BLOCK);
    __syncthreads();  // the next loads go where this block stands
  }
  loads_wait<0>();
  float inv[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    inv[i] = l[i] == 0.f ? 0.f : 1.f / l[i];
    const int qi = q0 + RI * ty + i;
    if (tx == 0 && qi < a.Sq)
      (a.splits > 1 ? a.part_lse + (int64_t)sp * a.B * a.H * a.Sq : a.lse)[a.stat(b, h, qi)] =
          m[i] + logf(l[i]);
  }
  if (a.splits > 1)
    store_rows<DP, RI>(a.part_o + (((int64_t)sp * a.B + b) * a.Sq * a.H + h) * a.D, (int64_t)a.H * a.D, q0, a.Sq,
                       a.D, acc, inv);
  else
    store_rows<DP, RI>(static_cast<float*>(a.o) + b * a.so.b + h * a.so.h, a.so.s, q0, a.Sq, a.D, acc, inv);
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

// dq (and delta, and the bias gradient's partial sums): one CTA per TR queries and share
// of the keys.
template <int DP, int RI>
__global__ void __launch_bounds__(NT)
xattn_dq_simt_kernel(const __grid_constant__ Args a, int tiles, int splits) {
  constexpr int TR = 16 * RI, BLOCK = TB * pitch<DP>(), DIAGONALS = TR + TB - 1;
  extern __shared__ float4 smem_f4[];
  float* Qs = reinterpret_cast<float*>(smem_f4);
  float* Os = Qs + TR * pitch<DP>();
  float* Ks = Os + TR * pitch<DP>();  // [2][K | V]
  float* Ds = Ks + 4 * BLOCK;
  __shared__ float delta[TR], lse[TR], diagonal[DIAGONALS + 1];
  pdl_wait();
  pdl_trigger();
  int64_t u = blockIdx.x;
  const int sp = (int)(u % splits);
  u /= splits;
  const int tile = tiles - 1 - (int)(u % tiles);
  u /= tiles;
  const int h = (int)(u % a.H), b = (int)(u / a.H), g = h / a.share;
  const int len = a.len(b), p0 = a.start(b);
  const int q0 = tile * TR, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int last = min(q0 + TR, a.Sq) - 1;
  const int seen = a.causal ? min(len, max(0, p0 + last + 1)) : len;
  const int blocks = (seen + TB - 1) / TB, per = (blocks + splits - 1) / splits;
  const int j0 = sp * per, j1 = min(blocks, j0 + per);
  const float* k = static_cast<const float*>(a.k) + b * a.sk.b + g * a.sk.h;
  const float* v = static_cast<const float*>(a.v) + b * a.sv.b + g * a.sv.h;
  auto load = [&](int j) {
    float* to = Ks + ((j - j0) & 1) * 2 * BLOCK;
    if (j < j1) {
      load_tile<DP, TB>(to, k, a.sk.s, j * TB, len, a.D);
      load_tile<DP, TB>(to + BLOCK, v, a.sv.s, j * TB, len, a.D);
    }
    loads_commit();
  };
  load_tile<DP, TR>(Qs, static_cast<const float*>(a.q) + b * a.sq.b + h * a.sq.h, a.sq.s, q0, a.Sq, a.D);
  load_tile<DP, TR>(Os, static_cast<const float*>(a.d_o) + b * a.sdo.b + h * a.sdo.h, a.sdo.s, q0, a.Sq, a.D);
  // (o where the second block will stand)
  load_tile<DP, TR>(Ks + 2 * BLOCK, static_cast<const float*>(a.o) + b * a.so.b + h * a.so.h, a.so.s, q0, a.Sq, a.D);
  load(j0);
  loads_wait<0>();
  __syncthreads();
  {  // delta, NT / TR threads a row
    constexpr int PER = NT / TR;
    const int r = threadIdx.x / PER;
    float d = 0.f;
    for (int c = threadIdx.x % PER; c < DP; c += PER)
      d = fmaf(Os[r * pitch<DP>() + c], Ks[2 * BLOCK + r * pitch<DP>() + c], d);
#pragma unroll
    for (int x = 1; x < PER; x <<= 1) d += __shfl_xor_sync(~0u, d, x);
    if (threadIdx.x % PER == 0) {
      delta[r] = d;
      const bool valid = q0 + r < a.Sq;
      if (valid && sp == 0) a.delta[a.stat(b, h, q0 + r)] = d;
      const float l = valid ? a.lse[a.stat(b, h, q0 + r)] : INFINITY;
      lse[r] = beyond_weights(l) ? INFINITY : l;  // a row without keys: every weight 0
    }
  }
  __syncthreads();
  float acc[RI][DP / 16] = {};
  // the bias gradient: 8 threads a bucket, bucket threadIdx.x / 8 + 32 x
  float db[MAX_BUCKETS / 32] = {};
  for (int j = j0; j < j1; ++j) {
    load(j + 1);
    loads_wait<1>();
    __syncthreads();
    const float* K = Ks + ((j - j0) & 1) * 2 * BLOCK;
    float s[RI][4], dp[RI][4];
    rows_product<DP, RI>(s, Qs, K);
    rows_product<DP, RI>(dp, Os, K + BLOCK);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int r = RI * ty + i, p = p0 + q0 + r;
      const int vis = q0 + r >= a.Sq ? 0 : a.causal ? min(len, p + 1) : len;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int key = j * TB + tx + 16 * c;
        s[i][c] *= a.scale;
        if (a.bias.buckets) s[i][c] += a.bias.clamped(h, key - p);
        weight_and_grad(s[i][c], dp[i][c], key < vis, vis == 1, lse[r], delta[r]);
        Ds[r * PITCH_P + tx + 16 * c] = dp[i][c];
      }
    }
    if (a.bias_part != nullptr) {
      // sums along the tile's diagonals, then each bucket's run of them
      __syncthreads();
      if (threadIdx.x < DIAGONALS) {
        const int d = (int)threadIdx.x - (TR - 1);  // column less row
        float x = 0.f;
#pragma unroll 4
        for (int r = max(0, -d); r < min(TR, TB - d); ++r) x += Ds[r * (PITCH_P + 1) + d];
        diagonal[threadIdx.x] = x;
      }
      __syncthreads();
      const int n0 = j * TB - (p0 + q0) - (TR - 1);  // distance of diagonal 0
#pragma unroll
      for (int y = 0; y < MAX_BUCKETS / 32; ++y) {
        const int u = (int)threadIdx.x / 8 + 32 * y;
        if (u >= a.bias.buckets) break;
        const int2 run = a.bias.range[u];
        const int64_t lo = (int64_t)run.x - n0, hi = (int64_t)run.y - n0;
        for (int x = (int)max((int64_t)0, lo) + (int)threadIdx.x % 8; x <= (int)min((int64_t)(DIAGONALS - 1), hi); x += 8)
          db[y] += diagonal[x];
      }
    } else {
      __syncwarp();
    }
    add_product<DP, RI>(acc, Ds, K);
    __syncthreads();  // the next loads go where this block stands
  }
  loads_wait<0>();
  float f[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) f[i] = splits > 1 ? 1.f : a.scale;
  if (splits > 1)
    store_rows<DP, RI>(a.piece_dq + (((int64_t)sp * a.B + b) * a.Sq * a.H + h) * a.D, (int64_t)a.H * a.D, q0, a.Sq,
                       a.D, acc, f);
  else
    store_rows<DP, RI>(static_cast<float*>(a.dq) + b * a.sdq.b + h * a.sdq.h, a.sdq.s, q0, a.Sq, a.D, acc, f);
  if (a.bias_part == nullptr) return;
  const int64_t row = (((int64_t)h * a.B + b) * tiles + tile) * splits + sp;
#pragma unroll
  for (int y = 0; y < MAX_BUCKETS / 32; ++y) {
#pragma unroll
    for (int x = 1; x < 8; x <<= 1) db[y] += __shfl_xor_sync(~0u, db[y], x);
    const int u = (int)threadIdx.x / 8 + 32 * y;
    if (threadIdx.x % 8 == 0 && u < a.bias.buckets) a.bias_part[row * a.bias.buckets + u] = db[y];
  }
}

// dk and dv: one CTA per TR keys of one (sequence, key head) and share of its query heads'
// blocks of 64 queries.
template <int DP, int RI>
__global__ void __launch_bounds__(NT)
xattn_dkv_simt_kernel(const __grid_constant__ Args a, int tiles, int splits) {
  constexpr int TR = 16 * RI, BLOCK = TB * pitch<DP>();
  extern __shared__ float4 smem_f4[];
  float* Ks = reinterpret_cast<float*>(smem_f4);
  float* Vs = Ks + TR * pitch<DP>();
  float* Qs = Vs + TR * pitch<DP>();  // [2][Q | dO]
  float* Ps = Qs + 4 * BLOCK;
  float* Ds = Ps + TR * PITCH_P;
  __shared__ float delta[2][TB], lse[2][TB];
  pdl_wait();
  pdl_trigger();
  int64_t u = blockIdx.x;
  const int sp = (int)(u % splits);
  u /= splits;
  const int tile = (int)(u % tiles);
  u /= tiles;
  const int g = (int)(u % a.G), b = (int)(u / a.G);
  const int len = a.len(b), p0 = a.start(b);
  const int k0 = tile * TR, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  // queries before the first that sees key k0 give nothing
  const int i0 = a.causal ? max(0, k0 - p0) / TB : 0;
  const int heads_blocks = k0 < len ? max(0, (a.Sq + TB - 1) / TB - i0) : 0, n = heads_blocks * a.share;
  const int per = (n + splits - 1) / splits, x0 = sp * per, x1 = min(n, x0 + per);
  auto load = [&](int x) {
    if (x < x1) {
      const int h = g * a.share + x / heads_blocks, i = i0 + x % heads_blocks, at = (x - x0) & 1;
      float* to = Qs + at * 2 * BLOCK;
      load_tile<DP, TB>(to, static_cast<const float*>(a.q) + b * a.sq.b + h * a.sq.h, a.sq.s, i * TB, a.Sq, a.D);
      load_tile<DP, TB>(to + BLOCK, static_cast<const float*>(a.d_o) + b * a.sdo.b + h * a.sdo.h, a.sdo.s, i * TB,
                        a.Sq, a.D);
      if (threadIdx.x < TB) {
        const int qi = i * TB + threadIdx.x;
        const float l = qi < a.Sq ? a.lse[a.stat(b, h, qi)] : INFINITY;
        lse[at][threadIdx.x] = beyond_weights(l) ? INFINITY : l;
        delta[at][threadIdx.x] = qi < a.Sq ? a.delta[a.stat(b, h, qi)] : 0.f;
      }
    }
    loads_commit();
  };
  load_tile<DP, TR>(Ks, static_cast<const float*>(a.k) + b * a.sk.b + g * a.sk.h, a.sk.s, k0, len, a.D);
  load_tile<DP, TR>(Vs, static_cast<const float*>(a.v) + b * a.sv.b + g * a.sv.h, a.sv.s, k0, len, a.D);
  load(x0);
  float dk[RI][DP / 16] = {}, dv[RI][DP / 16] = {};
  for (int x = x0; x < x1; ++x) {
    load(x + 1);
    loads_wait<1>();
    __syncthreads();
    const int h = g * a.share + x / heads_blocks, i = i0 + x % heads_blocks, at = (x - x0) & 1;
    const float* Q = Qs + at * 2 * BLOCK;
    float s[RI][4], dp[RI][4];
    rows_product<DP, RI>(s, Ks, Q);
    rows_product<DP, RI>(dp, Vs, Q + BLOCK);
#pragma unroll
    for (int r = 0; r < RI; ++r) {
      const int key = k0 + RI * ty + r;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int y = tx + 16 * c, qi = i * TB + y, p = p0 + qi;
        s[r][c] *= a.scale;
        if (a.bias.buckets) s[r][c] += a.bias.clamped(h, key - p);
        const bool visible = key < len && qi < a.Sq && (!a.causal || key <= p);
        weight_and_grad(s[r][c], dp[r][c], visible, len == 1 || (a.causal && p == 0), lse[at][y], delta[at][y]);
        Ps[(RI * ty + r) * PITCH_P + y] = s[r][c];
        Ds[(RI * ty + r) * PITCH_P + y] = dp[r][c];
      }
    }
    __syncwarp();
    add_product<DP, RI>(dv, Ps, Q + BLOCK);
    add_product<DP, RI>(dk, Ds, Q);
    __syncthreads();  // the next loads go where this block stands
  }
  loads_wait<0>();
  float fk[RI], fv[RI];
#pragma unroll
  for (int r = 0; r < RI; ++r) {
    const bool in = k0 + RI * ty + r < len;
    fk[r] = in ? (splits > 1 ? 1.f : a.scale) : 0.f, fv[r] = in ? 1.f : 0.f;
    if (!in)  // nothing of what stands behind the sequence's keys
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) dk[r][n] = dv[r][n] = 0.f;
  }
  if (splits > 1) {
    const int64_t one = (int64_t)a.B * a.Sk * a.G * a.D;
    float* to = a.piece_dkv + sp * 2 * one + ((int64_t)b * a.Sk * a.G + g) * a.D;
    store_rows<DP, RI>(to, (int64_t)a.G * a.D, k0, a.Sk, a.D, dk, fk);
    store_rows<DP, RI>(to + one, (int64_t)a.G * a.D, k0, a.Sk, a.D, dv, fv);
    return;
  }
  store_rows<DP, RI>(static_cast<float*>(a.dk) + b * a.sdk.b + g * a.sdk.h, a.sdk.s, k0, a.Sk, a.D, dk, fk);
  store_rows<DP, RI>(static_cast<float*>(a.dv) + b * a.sdv.b + g * a.sdv.h, a.sdv.s, k0, a.Sk, a.D, dv, fv);
}

// out = scale times the sum of the shares' [batch][tokens][heads][D], `step` apart.
__global__ void __launch_bounds__(256)
xattn_sum_simt_kernel(const float* part, int splits, int64_t step, float* out, Strides sd, int tokens, int heads, int D,
                      float scale, int64_t n) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int q = 0; q < splits; ++q) {
      const float4 x = *reinterpret_cast<const float4*>(part + q * step + 4 * i);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    int64_t r = 4 * i / D;
    const int c = (int)(4 * i - r * D), h = (int)(r % heads);
    r /= heads;
    const int64_t t = r % tokens, b = r / tokens;
    *reinterpret_cast<float4*>(out + b * sd.b + t * sd.s + h * sd.h + c) =
        make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale);
  }
}
cudaError_t add_shares(const float* part, int splits, int64_t step, void* out, const Strides& sd, const Args& a, int tokens,
                       int heads, float scale, cudaStream_t st) {
  const int64_t n = (int64_t)a.B * tokens * heads * a.D / 4;
  return launch_pdl(xattn_sum_simt_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 8 * sm_count())), dim3(256), 0, st,
                    part, splits, step, static_cast<float*>(out), sd, tokens, heads, a.D, scale, n);
}

template <int DP, int TR>
constexpr int smem(int tiles, int squares) {  // tiles of TR rows beside the two blocks
  return ((tiles * TR + 4 * TB) * pitch<DP>() + squares * TR * PITCH_P) * 4;
}

template <int DP, int RI>
cudaError_t fwd(const Args& a, cudaStream_t st) {
  constexpr int TR = 16 * RI, BYTES = smem<DP, TR>(1, 1);
  static_assert(BYTES <= 232448, "more than 227 KB of shared memory");
  const int tiles = (a.Sq + TR - 1) / TR;
  const int64_t n = (int64_t)a.B * a.H * tiles * a.splits;
  if (n > INT32_MAX) return cudaErrorInvalidConfiguration;
  static DeviceOnce attr;
  OASES_TRY(attr.run([] {
    return cudaFuncSetAttribute(xattn_fwd_simt_kernel<DP, RI>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
  }));
  return launch_pdl(xattn_fwd_simt_kernel<DP, RI>, dim3((unsigned)n), dim3(NT), BYTES, st, a, tiles);
}
template <int DP, int RI>
cudaError_t bwd_q(const Args& a, int splits, cudaStream_t st) {
  constexpr int TR = 16 * RI, BYTES = smem<DP, TR>(2, 1);
  static_assert(BYTES + 2048 <= 232448, "more than 227 KB of shared memory");
  const int tiles = (a.Sq + TR - 1) / TR;
  const int64_t n = (int64_t)a.B * a.H * tiles * splits;
  if (n > INT32_MAX) return cudaErrorInvalidConfiguration;
  static DeviceOnce attr;
  OASES_TRY(attr.run([] {
    return cudaFuncSetAttribute(xattn_dq_simt_kernel<DP, RI>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
  }));
  return launch_pdl(xattn_dq_simt_kernel<DP, RI>, dim3((unsigned)n), dim3(NT), BYTES, st, a, tiles, splits);
}
template <int DP, int RI>
cudaError_t bwd_kv(const Args& a, int splits, cudaStream_t st) {
  constexpr int TR = 16 * RI, BYTES = smem<DP, TR>(2, 2);
  static_assert(BYTES + 1024 <= 232448, "more than 227 KB of shared memory");
  const int tiles = (a.Sk + TR - 1) / TR;
  const int64_t n = (int64_t)a.B * a.G * tiles * splits;
  if (n > INT32_MAX) return cudaErrorInvalidConfiguration;
  static DeviceOnce attr;
  OASES_TRY(attr.run([] {
    return cudaFuncSetAttribute(xattn_dkv_simt_kernel<DP, RI>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
  }));
  return launch_pdl(xattn_dkv_simt_kernel<DP, RI>, dim3((unsigned)n), dim3(NT), BYTES, st, a, tiles, splits);
}

// Rows of a tile: 64, or 32 where 64 would leave SMs without a CTA.
int tile_rows(int64_t pairs, int tokens) { return pairs * ((tokens + 63) / 64) < sm_count() ? 32 : 64; }
// Shares of the other side's blocks: two CTAs an SM, 4 blocks to a share at least.
int shares(int64_t items, int64_t blocks) {
  const int places = 2 * sm_count();
  return items >= places ? 1 : (int)std::max<int64_t>(1, std::min(places / std::max<int64_t>(items, 1), blocks / 4));
}

}  // namespace

F32Cut xattn_f32_cut(const Args& a) {
  F32Cut c;
  const int64_t q = (int64_t)a.B * a.H, kv = (int64_t)a.B * a.G;
  c.q_rows = tile_rows(q, a.Sq);
  c.kv_rows = a.D > 64 ? 32 : tile_rows(kv, a.Sk);  // (64 rows of 128 values: too much shared memory)
  c.q_shares = shares(q * ((a.Sq + c.q_rows - 1) / c.q_rows), (a.Sk + TB - 1) / TB);
  c.kv_shares = shares(kv * ((a.Sk + c.kv_rows - 1) / c.kv_rows), (int64_t)((a.Sq + TB - 1) / TB) * a.share);
  return c;
}

cudaError_t xattn_fwd_f32(const Args& a, cudaStream_t st) {
  const bool few = xattn_f32_cut(a).q_rows == 32;
  return a.D <= 32   ? (few ? fwd<32, 2>(a, st) : fwd<32, 4>(a, st))
         : a.D <= 64 ? (few ? fwd<64, 2>(a, st) : fwd<64, 4>(a, st))
                     : (few ? fwd<128, 2>(a, st) : fwd<128, 4>(a, st));
}
cudaError_t xattn_bwd_f32(const Args& a, cudaStream_t st) {
  const F32Cut c = xattn_f32_cut(a);
  const bool fq = c.q_rows == 32, fk = c.kv_rows == 32;
  const int sq = c.q_shares, sk = c.kv_shares;
  OASES_TRY((a.D <= 32   ? (fq ? bwd_q<32, 2>(a, sq, st) : bwd_q<32, 4>(a, sq, st))
            : a.D <= 64 ? (fq ? bwd_q<64, 2>(a, sq, st) : bwd_q<64, 4>(a, sq, st))
                        : (fq ? bwd_q<128, 2>(a, sq, st) : bwd_q<128, 4>(a, sq, st))));
  OASES_TRY((a.D <= 32   ? (fk ? bwd_kv<32, 2>(a, sk, st) : bwd_kv<32, 4>(a, sk, st))
            : a.D <= 64 ? (fk ? bwd_kv<64, 2>(a, sk, st) : bwd_kv<64, 4>(a, sk, st))
                        : bwd_kv<128, 2>(a, sk, st)));
  if (sq > 1)
    OASES_TRY(add_shares(a.piece_dq, sq, (int64_t)a.B * a.Sq * a.H * a.D, a.dq, a.sdq, a, a.Sq, a.H, a.scale, st));
  if (sk > 1) {
    const int64_t one = (int64_t)a.B * a.Sk * a.G * a.D;
    OASES_TRY(add_shares(a.piece_dkv, sk, 2 * one, a.dk, a.sdk, a, a.Sk, a.G, a.scale, st));
    OASES_TRY(add_shares(a.piece_dkv + one, sk, 2 * one, a.dv, a.sdv, a, a.Sk, a.G, 1.f, st));
  }
  return cudaSuccess;
}

}  // namespace oases
