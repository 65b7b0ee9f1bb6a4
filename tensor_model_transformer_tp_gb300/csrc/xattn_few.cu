// Attention over keys of another length, forward, for a few query rows a key head (one
// token of a sequence being sampled: as many rows as query heads share the key head).
//
// Such a call reads every key and value once and does little with them, so it is bound
// by HBM.  A tile of a matrix product would be nearly empty; here a key's values lie in
// the lanes of a part of a warp, 16 bytes each, and every row's product with it is
// summed by shuffles.  Each such group of lanes goes through its own keys with its own
// running maximum and sum, KU keys at a time, the next ones' loads in flight in the
// registers that these have left (a whole step ahead, in registers of its own, leaves two
// CTAs an SM instead of three: 64 sequences of up to 2000 keys, 16 heads of 64, 50 us
// against 46; through shared memory, 49).  A cluster of CTAs shares the keys that the
// sequence has and joins its groups' results through distributed shared memory; only
// where sequences and key heads are too few for the GPU are the keys split further,
// through memory.  Ragged sequences are taken longest first, rounds of the SMs in snake
// order, so that the CTAs that share an SM have about the same keys together (16 sequences
// of up to 1500 keys, 20 heads of 64: 14 us with the keys in L2, 21 from memory; 59 MB).
// The position bias: R or more away one value on each side, kept in a register; nearer, by
// distance from shared memory where R is at most NEAR, else searched for.
#include <math.h>

#include <algorithm>

#include "sm100_ptx.cuh"
#include "xattn.cuh"

namespace oases {
namespace {
using namespace xattn;

constexpr int WARPS = 8, NT = 32 * WARPS;
constexpr int MAX_CLUSTER = 8;
constexpr int NEAR = 256;  // distances on each side in shared memory

template <typename T>
constexpr int EPL = 16 / (int)sizeof(T);  // values of a lane

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[EPL<T>]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      f[i] = __uint_as_float(w[i]);
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// The bias's table in x's type, and what finds a bucket.
struct Table {
  const void* p;
  Borders border;
  int bidirectional;
  // bias of head h at relative position n, in units of log2(e); finite values stay so
  template <typename T>
  __device__ __forceinline__ float at(int heads, int h, int n) const {
    const int u = border.bucket(bidirectional ? abs(n) : max(-n, 0)) + (bidirectional && n > 0 ? border.n + 1 : 0);
    const float v = ld_elem(static_cast<const T*>(p), (int64_t)u * heads + h);
    return fabsf(v) < INFINITY ? fminf(fmaxf(v * LOG2E, -3.402823466e38f), 3.402823466e38f) : v;
  }
};

// LPK lanes a key, R rows (query i, query head hh of the group: row i share + hh).
template <typename T, int LPK, int R, bool BIAS>
__global__ void __launch_bounds__(NT, R == 1 ? 3 : 2)
xattn_few_kernel(const __grid_constant__ Args a, const __grid_constant__ Table table, int rows, int sms) {
  constexpr int E = EPL<T>, GROUPS = 32 / LPK, KU = R == 4 ? 2 : 4, D_MAX = LPK * E;
  __shared__ float red_o[WARPS][R][D_MAX], red_m[WARPS][R], red_l[WARPS][R];
  __shared__ float out_o[R][D_MAX], out_m[R], out_l[R];
  __shared__ float near[BIAS ? R : 1][BIAS ? 2 * NEAR + 1 : 1];
  __shared__ int lens[NT], order[NT];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane % LPK, grp = lane / LPK;
  const int csize = gridDim.x / a.splits, rank = blockIdx.x % csize, sp = blockIdx.x / csize;
  int y = blockIdx.y;
  if (a.kv_lens && a.B > 1 && a.B <= NT) {
    // place y of the rounds' snake order, in the sequences by falling length
    const int round = y / sms, at = y % sms, n = min(sms, (int)gridDim.y - round * sms);
    if (round & 1) y = round * sms + n - 1 - at;
    const int t = threadIdx.x;
    if (t < a.B) lens[t] = a.len(t);
    __syncthreads();
    if (t < a.B) {
      int rank = 0;
      for (int x = 0; x < a.B; ++x) rank += lens[x] > lens[t] || (lens[x] == lens[t] && x < t);
      order[rank] = t;
    }
    __syncthreads();
    y = order[y / a.G] * a.G + y % a.G;
  }
  const int g = y % a.G, b = y / a.G;
  const int len = a.len(b), p0 = a.start(b);
  const int seen = a.causal ? min(len, max(0, p0 + a.Sq)) : len;
  // this CTA's keys: an even share, in whole steps of a CTA's groups
  constexpr int STEP = WARPS * GROUPS * KU;
  const int parts = csize * a.splits, part = sp * csize + rank;
  const int share = ((seen + parts - 1) / parts + STEP - 1) / STEP * STEP;
  const int k_begin = min(seen, part * share), k_end = min(seen, k_begin + share);
  const bool cols = sub * E < a.D;

  float q[R][E], acc[R][E], m[R], l[R];
  int vis[R], pos[R];
  float left[R], right[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = r / a.share, h = g * a.share + r % a.share;
    const bool in = r < rows;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in && cols)
      v = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + b * a.sq.b + i * a.sq.s + h * a.sq.h + sub * E);
    unpack<T>(v, q[r]);
    pos[r] = p0 + i;
    left[r] = right[r] = 0.f;
    if (BIAS && in) {
      left[r] = table.at<T>(a.H, h, -a.bias.R);
      right[r] = table.at<T>(a.H, h, a.bias.R);
    }
    vis[r] = !in ? 0 : a.causal ? min(len, p0 + i + 1) : len;
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[r][e] *= a.scale * LOG2E;
      acc[r][e] = 0.f;
    }
  }
  const T* kp = static_cast<const T*>(a.k) + b * a.sk.b + g * a.sk.h + sub * E;
  const T* vp = static_cast<const T*>(a.v) + b * a.sv.b + g * a.sv.h + sub * E;
  // a step's keys are loaded once the step before has used its own, and its values likewise
  uint4 kv[KU], vv[KU];
  auto load = [&](uint4 (&to)[KU], const T* from, int64_t stride, int k0) {
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const int key = k0 + u * GROUPS;
      to[u] = make_uint4(0, 0, 0, 0);
      if (key < k_end && cols) to[u] = *reinterpret_cast<const uint4*>(from + key * stride);
    }
  };
  const int k_first = k_begin + warp * GROUPS * KU + grp;
  load(kv, kp, a.sk.s, k_first);
  load(vv, vp, a.sv.s, k_first);
  const bool by_distance = BIAS && a.bias.R <= NEAR;
  if (by_distance) {
    const int n = 2 * a.bias.R + 1;
    for (int x = threadIdx.x; x < rows * n; x += NT)
      near[x / n][x % n] = table.at<T>(a.H, g * a.share + x / n % a.share, x % n - a.bias.R);
    __syncthreads();
  }
  for (int k0 = k_first; k0 - grp < k_end; k0 += STEP) {
    float s[R][KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      float f[E];
      unpack<T>(kv[u], f);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) d = fmaf(q[r][e], f[e], d);
        s[r][u] = d;
      }
    }
    load(kv, kp, a.sk.s, k0 + STEP);
#pragma unroll
    for (int o = LPK / 2; o; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int u = 0; u < KU; ++u) s[r][u] += __shfl_xor_sync(~0u, s[r][u], o);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int h = g * a.share + r % a.share;
      float mx = m[r];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int key = k0 + u * GROUPS;
        if (BIAS && r < rows) {
          const int n = key - pos[r];
          s[r][u] += n <= -a.bias.R   ? left[r]
                     : n >= a.bias.R ? right[r]
                     : by_distance   ? near[r][n + a.bias.R]
                                     : table.at<T>(a.H, h, n);
        }
        if (key >= k_end || key >= vis[r]) s[r][u] = -INFINITY;
        mx = fmaxf(mx, s[r][u]);
      }
      const float ref = mx == -INFINITY ? 0.f : mx;  // no key so far: all weights 0
      const float f = exp2f(m[r] - ref);
      m[r] = mx;
      l[r] *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[r][e] *= f;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        s[r][u] = exp2f(s[r][u] - ref);
        l[r] += s[r][u];
      }
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      float f[E];
      unpack<T>(vv[u], f);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] = fmaf(s[r][u], f[e], acc[r][e]);
    }
    load(vv, vp, a.sv.s, k0 + STEP);
  }
  // the warp's groups, then the CTA's warps, then the cluster's CTAs
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = LPK; o < 32; o <<= 1) {
      const float mo = __shfl_xor_sync(~0u, m[r], o), lo = __shfl_xor_sync(~0u, l[r], o);
      const float top = fmaxf(m[r], mo), ref = top == -INFINITY ? 0.f : top;
      const float f = exp2f(m[r] - ref), fo = exp2f(mo - ref);
      m[r] = top;
      l[r] = l[r] * f + lo * fo;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[r][e] = acc[r][e] * f + __shfl_xor_sync(~0u, acc[r][e], o) * fo;
    }
    if (grp == 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) red_o[warp][r][sub * E + e] = acc[r][e];
      if (sub == 0) {
        red_m[warp][r] = m[r];
        red_l[warp][r] = l[r];
      }
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < R * D_MAX; x += NT) {
    const int r = x / D_MAX, d = x % D_MAX;
    float top = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, red_m[w][r]);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = exp2f(red_m[w][r] - ref);
      sum = fmaf(red_l[w][r], f, sum);
      v = fmaf(red_o[w][r][d], f, v);
    }
    out_o[r][d] = v;
    if (d == 0) {
      out_m[r] = top;
      out_l[r] = sum;
    }
  }
  if (csize > 1) ptx::cluster_sync();
  else __syncthreads();
  // rank k writes rows k, k + csize, ...
  const uint32_t so = ptx::smem_u32(&out_o[0][0]), sm = ptx::smem_u32(out_m), sl = ptx::smem_u32(out_l);
  for (int x = threadIdx.x; x < R * D_MAX; x += NT) {
    const int r = x / D_MAX, d = x % D_MAX;
    if (r % csize != rank || r >= rows || d >= a.D) continue;
    float top = -INFINITY, sum = 0.f, v = 0.f;
    if (csize == 1) {
      top = out_m[r], sum = out_l[r], v = out_o[r][d];
    } else {
      for (int c = 0; c < csize; ++c) top = fmaxf(top, ptx::ld_cluster(ptx::mapa(sm + 4 * r, c)));
      const float ref = top == -INFINITY ? 0.f : top;
      for (int c = 0; c < csize; ++c) {
        const float f = exp2f(ptx::ld_cluster(ptx::mapa(sm + 4 * r, c)) - ref);
        sum = fmaf(ptx::ld_cluster(ptx::mapa(sl + 4 * r, c)), f, sum);
        v = fmaf(ptx::ld_cluster(ptx::mapa(so + 4 * x, c)), f, v);
      }
    }
    const int i = r / a.share, h = g * a.share + r % a.share;
    const float o = sum == 0.f ? 0.f : v / sum, lse = (top + log2f(sum)) * LN2;
    if (a.splits > 1) {
      a.part_o[((((int64_t)sp * a.B + b) * a.Sq + i) * a.H + h) * a.D + d] = o;
      if (d == 0) a.part_lse[(int64_t)sp * a.B * a.H * a.Sq + a.stat(b, h, i)] = lse;
    } else {
      st_elem(static_cast<T*>(a.o) + b * a.so.b + i * a.so.s + h * a.so.h, d, o);
      if (d == 0) a.lse[a.stat(b, h, i)] = lse;
    }
  }
  if (csize > 1) ptx::cluster_sync();  // no CTA leaves while another reads its results
}

template <typename T, int LPK, int R, bool BIAS>
cudaError_t launch(const Args& a, const Table& tb, int rows, int csize, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(csize * a.splits, a.B * a.G);
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = csize;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = csize > 1 ? 2 : 1;
  ++g_launch_count;
  return cudaLaunchKernelEx(&cfg, xattn_few_kernel<T, LPK, R, BIAS>, a, tb, rows, sm_count());
}
template <typename T, int LPK, bool BIAS>
cudaError_t launch_bias(const Args& a, const Table& tb, int rows, int csize, cudaStream_t st) {
  return rows == 1   ? launch<T, LPK, 1, BIAS>(a, tb, rows, csize, st)
         : rows == 2 ? launch<T, LPK, 2, BIAS>(a, tb, rows, csize, st)
                     : launch<T, LPK, 4, BIAS>(a, tb, rows, csize, st);
}
template <typename T, int LPK>
cudaError_t launch_rows(const Args& a, const Table& tb, int rows, int csize, cudaStream_t st) {
  return a.bias.buckets ? launch_bias<T, LPK, true>(a, tb, rows, csize, st)
                        : launch_bias<T, LPK, false>(a, tb, rows, csize, st);
}

// CTAs of a cluster: two an SM in all, with 256 keys each at least (at 320 sequences and
// key heads of up to 1500 keys of 64 values, clusters of 1, 2, 4, 8: 15, 19, 21, 34 us:
// a CTA's start and the join cost more than its keys).
int cluster_size(const Args& a) {
  int c = 1;
  while (c < MAX_CLUSTER && (int64_t)a.B * a.G * c < 2 * sm_count() && a.Sk >= 512 * c) c *= 2;
  return c;
}

}  // namespace

// Up to 4 rows a key head, and no more (sequence, key head) pairs than a grid's second
// dimension holds.  The other side is the kernel of 128-row tiles, a tile to each query head,
// which reads the keys once for each.  From a cold L2, bf16, here against there:
//   16 x 8192 keys, 4 key heads of 128: 1 query of 1, 2, 4 heads a key head 71, 69, 97 us against
//   67, 88, 167; 4 queries of 1 head 97 against 67
//   64 x 2000 keys, 4 key heads of 64: 44, 44, 58 against 48, 83, 138; 4 queries 58 against 48
// so that this one is for heads that share keys (where they do not, a key head's tile has all of
// its rows, and is as fast for one query and faster for four).  Eight heads a key head, there: 323 and 265.
bool xattn_few_takes(const Args& a) {
  return (int64_t)a.Sq * a.share <= 4 && (int64_t)a.B * a.G <= 65535;
}
// Shares of the keys beyond the cluster's: two CTAs an SM, and 256 keys to a CTA at least
// (4 sequences of up to 8192 keys, 8 heads on 2 of 128: 24 us, 30 with 512).
int xattn_few_splits(const Args& a) {
  const int c = cluster_size(a);
  const int64_t ctas = (int64_t)a.B * a.G * c, places = 2 * sm_count();
  if (c < MAX_CLUSTER || ctas >= places) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(places / ctas, a.Sk / (256 * c)));
}
cudaError_t xattn_few(const Args& a, const void* table, const Borders& border, bool bidirectional,
                      cudaStream_t st) {
  const Table tb{table, border, bidirectional ? 1 : 0};
  const int rows = a.Sq * a.share, c = cluster_size(a), chunks = a.D * (int)dtype_size(a.t) / 16;
  if (a.t == DType::BF16)
    return chunks <= 4   ? launch_rows<__nv_bfloat16, 4>(a, tb, rows, c, st)
           : chunks <= 8 ? launch_rows<__nv_bfloat16, 8>(a, tb, rows, c, st)
                         : launch_rows<__nv_bfloat16, 16>(a, tb, rows, c, st);
  return chunks <= 8    ? launch_rows<float, 8>(a, tb, rows, c, st)
         : chunks <= 16 ? launch_rows<float, 16>(a, tb, rows, c, st)
                        : launch_rows<float, 32>(a, tb, rows, c, st);
}

}  // namespace oases
