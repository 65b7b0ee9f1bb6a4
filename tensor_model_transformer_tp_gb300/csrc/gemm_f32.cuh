// fp32 GEMM on the CUDA cores with an epilogue given as a type, for the
// operators' fp32 form (TF32 tensor cores would round the operands to 11 bits):
//   D[m, n] = sum_k A(m, k) B(n, k).
//
// 64 x 64 output tiles, 64 threads of 8 x 8 outputs each, kept as pairs along
// m for the packed fp32x2 FMA; K goes 16 at a time through two shared-memory
// buffers, the next step's elements in registers meanwhile.  The models in fp32
// are small, so a product has few tiles: a cluster of S CTAs splits K, and the
// partial tiles meet through distributed shared memory, each CTA summing (in
// the order of the splits) and finishing 64 / S rows.  In a DUAL tile, B rows
// 0..31 come from n0 and 32..63 from b_off further down (gate and up), and the
// epilogue sees both products of an output.
#pragma once
#include "common.cuh"
#include "sm100_ptx.cuh"

namespace oases {
namespace f32 {

constexpr int BM = 64, BN = 64, BK = 16, NT = 64, LDS = 68;  // LDS: row pitch in shared memory

struct Args {
  int M, N, K;  // N: outputs per row (of each product, DUAL)
  const float* a;
  int64_t lda;
  const float* b;
  int64_t ldb;
  int b_off;  // DUAL: row offset of the second product's B
  int kspan;  // K per CTA of the cluster, a multiple of BK
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// One step's 64 x 16 elements of an operand, four per thread and register
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
        const int row = row_of(idx / 4), k = k0 + idx % 4 * 4;
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
        const int row = idx / 4, k = idx % 4 * 4;
        s[k * LDS + row] = r[i].x;
        s[(k + 1) * LDS + row] = r[i].y;
        s[(k + 2) * LDS + row] = r[i].z;
        s[(k + 3) * LDS + row] = r[i].w;
      } else {
        *reinterpret_cast<float4*>(s + idx / 16 * LDS + idx % 16 * 4) = r[i];
      }
    }
  }
};

// Epi: struct with DUAL and
//   device void tile(m, n0, const float (&v)[4], col, M, N): outputs n0 + col .. + 3
//   of row m (v[i] for columns inside the matrix only), or, DUAL,
//   device void tile(m, n0, const float (&a)[4], const float (&b)[4], col, M, N).
// Sixteen consecutive threads (8, DUAL) hold one row of a tile, in order.
template <class Epi, bool A_K, bool B_K, bool VEC>
__global__ void __launch_bounds__(NT) gemm_f32_kernel(const Args g, const Epi e) {
  __shared__ __align__(16) float smem[2 * 2 * BK * LDS];
  static_assert(2 * 2 * BK * LDS >= BM * BN, "the partial tile takes the buffers' place");
  constexpr int TN = Epi::DUAL ? BN / 2 : BN;
  const int S = gridDim.x, rank = blockIdx.x;
  const int m0 = blockIdx.z * BM, n0 = blockIdx.y * TN;
  const int tid = threadIdx.x, tx = tid % 8, ty = tid / 8;
  const int k0 = min(g.K, rank * g.kspan), kend = min(g.K, k0 + g.kspan);
  pdl_wait();
  pdl_trigger();
  auto row_a = [&](int i) { return m0 + i < g.M ? m0 + i : -1; };
  auto row_b = [&](int i) {
    if (Epi::DUAL) {
      const int c = n0 + i % TN;
      return c < g.N ? c + (i < TN ? 0 : g.b_off) : -1;
    }
    return n0 + i < g.N ? n0 + i : -1;
  };
  float *As = smem, *Bs = smem + 2 * BK * LDS;
  Loader<A_K, VEC> la;
  Loader<B_K, VEC> lb;
  uint64_t acc[4][8];  // pairs of rows (8 ty + 2 i, + 1), columns 8 tx + j
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0ull;
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
    const float *pa = As + buf * BK * LDS + 8 * ty, *pb = Bs + buf * BK * LDS + 8 * tx;
#pragma unroll
    for (int kk = 0; kk < BK; ++kk) {
      const ulonglong2 a0 = *reinterpret_cast<const ulonglong2*>(pa + kk * LDS);
      const ulonglong2 a1 = *reinterpret_cast<const ulonglong2*>(pa + kk * LDS + 4);
      const float4 b0 = *reinterpret_cast<const float4*>(pb + kk * LDS);
      const float4 b1 = *reinterpret_cast<const float4*>(pb + kk * LDS + 4);
      const uint64_t a[4] = {a0.x, a0.y, a1.x, a1.y};
      const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint64_t bb = f2_splat(b[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = f2_fma(a[i], bb, acc[i][j]);
      }
    }
    if (more) {
      la.store(As + (buf ^ 1) * BK * LDS);
      lb.store(Bs + (buf ^ 1) * BK * LDS);
    }
    __syncthreads();
  }
  // the partial tile, [64][64], in the buffers' place
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float* q = smem + (8 * ty + 2 * i + h) * BN + 8 * tx;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = h ? f2_hi(acc[i][j]) : f2_lo(acc[i][j]);
      *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  if (S > 1)
    ptx::cluster_sync();
  else
    __syncthreads();
  const uint32_t base = ptx::smem_u32(smem);
  uint32_t from[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) from[s] = s < S ? ptx::mapa(base, (uint32_t)s) : 0u;
  auto total = [&](int at, float (&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s)
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
  if (S > 1) {
    __syncwarp();
    ptx::cluster_sync();  // no CTA leaves while another reads its partial tile
  }
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
    const float s = scale ? *scale : 1.f;
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

template <class Epi, bool A_K, bool B_K>
cudaError_t launch(Args g, const Epi& e, cudaStream_t st) {
  constexpr int TN = Epi::DUAL ? BN / 2 : BN;
  if (g.M == 0 || g.N == 0) return cudaSuccess;
  const int64_t tm = (g.M + BM - 1) / BM, tn = (g.N + TN - 1) / TN;
  if (tm > 65535 || tn > 65535) return cudaErrorInvalidConfiguration;
  // split K while the SMs hold fewer than four CTAs each and a CTA keeps two steps
  int S = 1;
  while (S < 8 && tm * tn * S * 2 <= 152 * 6 && g.K >= S * 2 * 2 * BK) S *= 2;
  g.kspan = ((g.K + S - 1) / S + BK - 1) / BK * BK;
  auto ok4 = [](const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 4 == 0; };
  // 16-byte loads: every row starts on one and the extents read are whole ones
  const bool vec = ok4(g.a, g.lda) && ok4(g.b, g.ldb) && (A_K || B_K ? g.K % 4 == 0 : true) &&
                   (A_K || g.M % 4 == 0) && (B_K || g.N % 4 == 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S, (unsigned)tn, (unsigned)tm);
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = S;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  ++g_launch_count;
  return vec ? cudaLaunchKernelEx(&cfg, gemm_f32_kernel<Epi, A_K, B_K, true>, g, e)
             : cudaLaunchKernelEx(&cfg, gemm_f32_kernel<Epi, A_K, B_K, false>, g, e);
}

}  // namespace f32
}  // namespace oases
