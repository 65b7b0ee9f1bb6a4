// fp32 GEMM on the CUDA cores with an epilogue given as a type, for the
// operators' fp32 form (TF32 tensor cores would round the operands to 11 bits):
//   D[m, n] = sum_k A(m, k) B(n, k).
//
// 64 x 64 output tiles, 128 threads of 8 x 4 outputs each, kept as pairs along
// m for the packed fp32x2 FMA; K goes 32 at a time through two shared-memory
// buffers, the next step's elements in registers meanwhile.  The models in fp32
// are small, so a product has few tiles: a cluster of S CTAs splits K, and the
// partial tiles meet through distributed shared memory, each CTA summing (in
// the order of the splits) and finishing 64 / S rows.  In a DUAL tile, B rows
// 0..31 come from n0 and 32..63 from b_off further down (gate and up), and the
// epilogue sees both products of an output.  Several products (a backward's dx
// and weight gradients) share a launch: alone, none of them fills the SMs.
#pragma once
#include <algorithm>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace oases {
namespace f32 {

constexpr int BM = 64, BN = 64, BK = 32, NT = 128;
constexpr int MAX_DIM = 32 * 65535;  // rows and columns: tiles of 32 and 64 fit a grid dimension
constexpr int CLUSTER = 8;  // largest split of a contraction

// Operand tiles in shared memory are [BK][64] with each k's sixteen groups of
// four rows permuted by k / 4, so that the transposing stores of a K-major
// operand (eight k / 4 by four rows per warp) meet no bank twice.
__device__ __forceinline__ int at_of(int k, int row) { return k * 64 + (((row >> 2) ^ ((k >> 2) & 7)) << 2) + (row & 3); }

struct Args {
  int M, N, K;  // N: outputs per row (of each product, DUAL)
  const float* a;
  int64_t lda;
  const float* b;
  int64_t ldb;
  int b_off = 0;   // DUAL: row offset of the second product's B
  int padded = 0;  // a's rows go on with finite values up to a multiple of four elements
  int kspan = 0;   // K per CTA of the cluster, a multiple of BK
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// One step's 64 x 32 elements of an operand, four per thread and register
// group: K-major rows are read 4 along k, MN-major ones 4 along the row index.
template <bool KM, bool VEC>
struct Loader {
  float4 r[4];
  // rows: the operand's row of tile row i, or -1 past the matrix
  template <typename RowOf>
  __device__ __forceinline__ void load(const float* p, int64_t ld, int k0, int kend, RowOf row_of) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int idx = threadIdx.x + NT * i;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (KM) {
        const int row = row_of(idx / 8), k = k0 + idx % 8 * 4;
        if (row >= 0) {
          const float* q = p + (int64_t)row * ld + k;
          if (VEC) {
            if (k < kend) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(q);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (k + j < kend) v[j] = q[j];
          }
        }
      } else {
        const int k = k0 + idx / 16, m = idx % 16 * 4;
        if (k < kend) {
          const float* q = p + (int64_t)k * ld;
          if (VEC) {
            const int row = row_of(m);
            if (row >= 0) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(q + row);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = row_of(m + j);
              if (row >= 0) v[j] = q[row];
            }
          }
        }
      }
      r[i] = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  __device__ __forceinline__ void store(float* s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int idx = threadIdx.x + NT * i;
      if (KM) {
        const int row = idx / 8, k = idx % 8 * 4;
        float* q = s + at_of(k, row);  // k .. k+3 share the permutation
        q[0] = r[i].x;
        q[64] = r[i].y;
        q[128] = r[i].z;
        q[192] = r[i].w;
      } else {
        *reinterpret_cast<float4*>(s + at_of(idx / 16, idx % 16 * 4)) = r[i];
      }
    }
  }
};

// Epi: struct with DUAL and
//   device void tile(m, n0, const float (&v)[4], col, M, N): outputs n0 + col .. + 3
//   of row m (v[i] for columns inside the matrix only), or, DUAL,
//   device void tile(m, n0, const float (&a)[4], const float (&b)[4], col, M, N).
// Sixteen consecutive threads (8, DUAL) hold one row of a tile, in order.
// One tile, m0 .. and n0 .., by S CTAs of the cluster, rank0 .. rank0 + S - 1.
// (m0 past the matrix: a CTA of the cluster with no tile.)
template <class Epi, bool A_K, bool B_K, bool VEC>
__device__ __forceinline__ void tile_body(const Args& g, const Epi& e, int m0, int n0, int S, int rank0,
                                          float* smem) {
  constexpr int TN = Epi::DUAL ? BN / 2 : BN;
  const int rank = (int)blockIdx.x - rank0;
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int k0 = min(m0 < g.M ? g.K : 0, rank * g.kspan), kend = min(m0 < g.M ? g.K : 0, k0 + g.kspan);
  auto row_a = [&](int i) { return m0 + i < g.M ? m0 + i : -1; };
  auto row_b = [&](int i) {
    if (Epi::DUAL) {
      const int c = n0 + i % TN;
      return c < g.N ? c + (i < TN ? 0 : g.b_off) : -1;
    }
    return n0 + i < g.N ? n0 + i : -1;
  };
  float *As = smem, *Bs = smem + 2 * BK * 64;
  Loader<A_K, VEC> la;
  Loader<B_K, VEC> lb;
  uint64_t acc[4][4];  // pairs of rows (8 ty + 2 i, + 1), columns 4 tx + j
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
  if (k0 < kend) {
    la.load(g.a, g.lda, k0, kend, row_a);
    lb.load(g.b, g.ldb, k0, kend, row_b);
    la.store(As);
    lb.store(Bs);
  }
  __syncthreads();
  int buf = 0;
  for (int k = k0; k < kend; k += BK, buf ^= 1) {
    const bool more = k + BK < kend;
    if (more) {
      la.load(g.a, g.lda, k + BK, kend, row_a);
      lb.load(g.b, g.ldb, k + BK, kend, row_b);
    }
    const float *pa = As + buf * BK * 64, *pb = Bs + buf * BK * 64;
#pragma unroll
    for (int kk = 0; kk < BK; ++kk) {
      const ulonglong2 a0 = *reinterpret_cast<const ulonglong2*>(pa + at_of(kk, 8 * ty));
      const ulonglong2 a1 = *reinterpret_cast<const ulonglong2*>(pa + at_of(kk, 8 * ty + 4));
      const float4 b0 = *reinterpret_cast<const float4*>(pb + at_of(kk, 4 * tx));
      const uint64_t a[4] = {a0.x, a0.y, a1.x, a1.y};
      const float b[4] = {b0.x, b0.y, b0.z, b0.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t bb = f2_splat(b[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = f2_fma(a[i], bb, acc[i][j]);
      }
    }
    if (more) {
      la.store(As + (buf ^ 1) * BK * 64);
      lb.store(Bs + (buf ^ 1) * BK * 64);
    }
    __syncthreads();
  }
  // the partial tile, [64][64], in the buffers' place
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = h ? f2_hi(acc[i][j]) : f2_lo(acc[i][j]);
      *reinterpret_cast<float4*>(smem + (8 * ty + 2 * i + h) * BN + 4 * tx) =
          make_float4(v[0], v[1], v[2], v[3]);
    }
  if (gridDim.x > 1)
    ptx::cluster_sync();
  else
    __syncthreads();
  const uint32_t base = ptx::smem_u32(smem);
  uint32_t from[CLUSTER];
#pragma unroll
  for (int s = 0; s < CLUSTER; ++s) from[s] = s < S ? ptx::mapa(base, (uint32_t)(rank0 + s)) : 0u;
  auto total = [&](int at, float (&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
    for (int s = 0; s < CLUSTER; ++s)
      if (s < S) {
        const float4 q = ld_cluster4(from[s] + 4u * at);
        v[0] += q.x;
        v[1] += q.y;
        v[2] += q.z;
        v[3] += q.w;
      }
  };
  const int rows = BM / S;  // this CTA finishes rows rank * rows ..
  constexpr int PER = TN / 4;  // threads per row
  for (int i = tid; i < rows * PER; i += NT) {
    const int r = rank * rows + i / PER, col = i % PER * 4, m = m0 + r;
    if constexpr (Epi::DUAL) {
      float a[4], b[4];
      total(r * BN + col, a);
      total(r * BN + TN + col, b);
      e.tile(m, n0, a, b, col, g.M, g.N);
    } else {
      float v[4];
      total(r * BN + col, v);
      e.tile(m, n0, v, col, g.M, g.N);
    }
  }
  if (gridDim.x > 1) {
    __syncwarp();
    ptx::cluster_sync();  // no CTA leaves while another reads its partial tile
  }
}

constexpr int SMEM_FLOATS = 2 * 2 * BK * 64;
static_assert(SMEM_FLOATS >= BM * BN, "the partial tile takes the buffers' place");

template <class Epi, bool A_K, bool B_K, bool VEC>
__global__ void __launch_bounds__(NT, 4) gemm_f32_kernel(const Args g, const Epi e) {
  __shared__ __align__(16) float smem[SMEM_FLOATS];
  pdl_wait();
  pdl_trigger();
  tile_body<Epi, A_K, B_K, VEC>(g, e, blockIdx.z * BM, blockIdx.y * (Epi::DUAL ? BN / 2 : BN),
                                gridDim.x, 0, smem);
}

// C (+)= scale * D + bias + resid, each optional; resid may be C.
struct Out {
  static constexpr bool DUAL = false;
  float* c;
  int64_t ld;
  const float *scale, *bias, *resid;
  int accumulate;
  __device__ __forceinline__ void tile(int m, int n0, const float (&v)[4], int col, int M, int N) const {
    if (m >= M) return;
    const float s = product_factor(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + col + i;
      if (n >= N) break;
      const int64_t at = (int64_t)m * ld + n;
      float x = s * v[i];
      if (bias) x += bias[n];
      if (resid) x += resid[at];
      if (accumulate) x += c[at];
      c[at] = x;
    }
  }
};

// Products with MN-major B in one launch; A is K-major where a_k.  Product i
// splits its contraction over split[i] CTAs, so a cluster takes CLUSTER /
// split[i] of its tiles; its clusters are end[i - 1] .. end[i] - 1.
struct Group {
  Args g[3];
  Out e[3];
  int a_k[3], vec[3], tn[3], split[3], end[3];
};
static __global__ void __launch_bounds__(NT, 4) gemm_f32_group_kernel(const Group q) {
  __shared__ __align__(16) float smem[SMEM_FLOATS];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.y, i = c < q.end[0] ? 0 : c < q.end[1] ? 1 : 2;
  const int S = q.split[i], rank0 = (int)blockIdx.x / S * S;
  const int r = (c - (i ? q.end[i - 1] : 0)) * ((int)gridDim.x / S) + (int)blockIdx.x / S;
  const int m0 = r / q.tn[i] * BM, n0 = r % q.tn[i] * BN;
  if (q.a_k[i]) {
    if (q.vec[i])
      tile_body<Out, true, false, true>(q.g[i], q.e[i], m0, n0, S, rank0, smem);
    else
      tile_body<Out, true, false, false>(q.g[i], q.e[i], m0, n0, S, rank0, smem);
  } else {
    if (q.vec[i])
      tile_body<Out, false, false, true>(q.g[i], q.e[i], m0, n0, S, rank0, smem);
    else
      tile_body<Out, false, false, false>(q.g[i], q.e[i], m0, n0, S, rank0, smem);
  }
}

// CTAs that split a contraction over K: a CTA is left the K-steps that an even
// share of the launch's would give it with four CTAs per SM, two at least.
inline int split_of(int64_t launch_steps, int K) {
  const int64_t share = std::max<int64_t>(2, launch_steps / (4 * 152)), steps = (K + BK - 1) / BK;
  int S = 1;
  while (S < CLUSTER && steps > S * share) S *= 2;
  return S;
}
inline int span_of(int K, int S) { return ((K + S - 1) / S + BK - 1) / BK * BK; }
// 16-byte loads: every row starts on one and the extents read are whole ones.
// What a padded row of A has past K meets zeros of B, past M no output.
inline bool vector_loads(const Args& g, bool a_k, bool b_k) {
  auto ok4 = [](const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 4 == 0; };
  return ok4(g.a, g.lda) && ok4(g.b, g.ldb) && (g.padded || (a_k ? g.K : g.M) % 4 == 0) &&
         (b_k ? g.K : g.N) % 4 == 0;
}
inline void configure(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attrs, dim3 grid, cudaStream_t st) {
  *cfg = {};
  cfg->gridDim = grid;
  cfg->blockDim = dim3(NT);
  cfg->stream = st;
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = grid.x;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg->attrs = attrs;
  cfg->numAttrs = 2;
  ++g_launch_count;
}

// split: CTAs per contraction, 0: as is best for a launch of its own.
template <class Epi, bool A_K, bool B_K>
cudaError_t launch(Args g, const Epi& e, cudaStream_t st, int split = 0) {
  constexpr int TN = Epi::DUAL ? BN / 2 : BN;
  if (g.M == 0 || g.N == 0) return cudaSuccess;
  const int64_t tm = (g.M + BM - 1) / BM, tn = (g.N + TN - 1) / TN;
  if (tm > 65535 || tn > 65535) return cudaErrorInvalidConfiguration;
  const int S = split ? split : split_of(tm * tn * ((g.K + BK - 1) / BK), g.K);
  g.kspan = span_of(g.K, S);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attrs[2];
  configure(&cfg, attrs, dim3((unsigned)S, (unsigned)tn, (unsigned)tm), st);
  return vector_loads(g, A_K, B_K)
             ? cudaLaunchKernelEx(&cfg, gemm_f32_kernel<Epi, A_K, B_K, true>, g, e)
             : cudaLaunchKernelEx(&cfg, gemm_f32_kernel<Epi, A_K, B_K, false>, g, e);
}

// Up to three products with MN-major B; those with no output (e.c null) are left out.
// The contractions are split as if none were: a product's bits do not depend on
// which others are wanted.
static inline cudaError_t launch_group(const Args (&g)[3], const Out (&e)[3], const bool (&a_k)[3],
                                cudaStream_t st) {
  Group q = {};
  int n = 0;
  int64_t tiles[3], steps = 0;
  for (int i = 0; i < 3; ++i) {
    if (g[i].M == 0 || g[i].N == 0) continue;
    const int64_t tm = (g[i].M + BM - 1) / BM, tn = (g[i].N + BN - 1) / BN;
    steps += tm * tn * ((g[i].K + BK - 1) / BK);
    if (!e[i].c) continue;
    tiles[n] = tm * tn;
    q.g[n] = g[i];
    q.e[n] = e[i];
    q.a_k[n] = a_k[i];
    q.vec[n] = vector_loads(g[i], a_k[i], false);
    q.tn[n] = (int)tn;
    ++n;
  }
  if (n == 0) return cudaSuccess;
  int64_t clusters = 0;
  for (int i = 0; i < n; ++i) {
    q.split[i] = split_of(steps, q.g[i].K);
    q.g[i].kspan = span_of(q.g[i].K, q.split[i]);
    const int per = CLUSTER / q.split[i];
    clusters += (tiles[i] + per - 1) / per;
    q.end[i] = (int)std::min<int64_t>(clusters, INT32_MAX);
  }
  for (int i = n; i < 3; ++i) {
    q.split[i] = 1;
    q.end[i] = q.end[n - 1];
  }
  if (clusters > 65535) {  // more than a grid dimension holds
    for (int i = 0; i < n; ++i) {
      const cudaError_t err = q.a_k[i] ? launch<Out, true, false>(q.g[i], q.e[i], st, q.split[i])
                                       : launch<Out, false, false>(q.g[i], q.e[i], st, q.split[i]);
      if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attrs[2];
  configure(&cfg, attrs, dim3(CLUSTER, (unsigned)clusters), st);
  return cudaLaunchKernelEx(&cfg, gemm_f32_group_kernel, q);
}

}  // namespace f32
}  // namespace oases
