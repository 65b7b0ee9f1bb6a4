// Output epilogue of gemm_core.cuh:
//   C[m, n] (+)= scale * (D[m, n] + prior[m, n]) + bias[n] + resid[m, n]
// each term optional.
#pragma once
#include "gemm_core.cuh"

namespace oases {
namespace core {

struct EpiOut {
  static constexpr bool DUAL = false, PAD_ROWS = false;
  static constexpr int STG = 4096, WBARS = 0;  // 32 rows x 128 bytes
  struct Params {
    CUtensorMap c;             // boxes of 32 rows x 128 bytes of C
    int f32;                   // C's type: fp32, else bf16
    int accumulate;            // C (fp32) += by TMA reduction
    const float* scale;        // one device value, or null (1)
    const float* prior;        // fp32 [M, N], leading dimension N
    const __nv_bfloat16* bias;  // [N]
    const __nv_bfloat16* resid;  // [M, N]
    int slab_rows;             // rows between the outputs of two splits of the contraction
  };
  struct Warp : WarpBase {
    float alpha;
    template <int BN>
    __device__ __forceinline__ void before(const Params& e, const Problem&, int, int, int) {
      alpha = e.scale ? *e.scale : 1.f;
    }
    // CW accumulator columns from n, this lane's row m
    template <int CW>
    __device__ __forceinline__ void chunk(const Params& e, const Problem& p, int m, int n,
                                          float (&v)[CW]) {
      const bool row = m < p.M;
      if (e.prior && row) {
        const float* q = e.prior + (int64_t)m * p.N + n;
#pragma unroll
        for (int i = 0; i < CW; i += 4)
          if (n + i < p.N) {
            const float4 t = *reinterpret_cast<const float4*>(q + i);
            v[i] += t.x;
            v[i + 1] += t.y;
            v[i + 2] += t.z;
            v[i + 3] += t.w;
          }
      }
      if (e.scale) {
#pragma unroll
        for (int i = 0; i < CW; ++i) v[i] *= alpha;
      }
      if (e.bias) add8<CW>(e.bias + n, p.N - n, v);
      if (e.resid && row) add8<CW>(e.resid + (int64_t)m * p.N + n, p.N - n, v);
    }
    // v[i] += src[i] for i < left, left a multiple of 8
    template <int CW>
    __device__ __forceinline__ void add8(const __nv_bfloat16* src, int left, float (&v)[CW]) {
#pragma unroll
      for (int i = 0; i < CW; i += 8)
        if (i < left) {
          const uint4 u = *reinterpret_cast<const uint4*>(src + i);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2(w[k]);
            add2_inplace(v[i + 2 * k], v[i + 2 * k + 1], f.x, f.y);
          }
        }
    }
    template <int BN>
    __device__ __forceinline__ void tile(const Params& e, const Problem& p, int mw, int n0, int half,
                                         int z, uint32_t trow) {
      const int m = mw + lane;
      if (!e.f32) {
#pragma unroll 1
        for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 64) {
          const int n = n0 + c;
          if (n >= p.N) break;
          float v[64];
          ptx::tmem_ld32(trow + c, *reinterpret_cast<float(*)[32]>(v));
          ptx::tmem_ld32(trow + c + 32, *reinterpret_cast<float(*)[32]>(v + 32));
          chunk<64>(e, p, m, n, v);
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1]);
          wait_free();
          stage_row(w);
          store_box(&e.c, n, mw + z * e.slab_rows);
        }
      } else {
#pragma unroll 1
        for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
          const int n = n0 + c;
          if (n >= p.N) break;
          float v[32];
          ptx::tmem_ld32(trow + c, v);
          chunk<32>(e, p, m, n, v);
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
          wait_free();
          stage_row(w);
          if (e.accumulate)
            reduce_box(&e.c, n, mw);
          else
            store_box(&e.c, n, mw + z * e.slab_rows);
        }
      }
    }
  };
};

// Fills the output part of EpiOut's parameters: C [rows, N], leading dimension ld.
inline bool out_map(EpiOut::Params* e, void* c, DType t, int rows, int N, int64_t ld) {
  e->f32 = t == DType::F32;
  return tensor_map(&e->c, c, e->f32 != 0, N, rows, ld, e->f32 ? 32 : 64, 32);
}

}  // namespace core
}  // namespace oases
