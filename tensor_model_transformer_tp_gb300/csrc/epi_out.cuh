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
    const float* scale;        // one device value (product_factor), or null
    const float* prior;        // fp32 [M, N], leading dimension N
    const __nv_bfloat16* bias;  // [N]
    const __nv_bfloat16* resid;  // [M, N]
    int slab_rows;             // rows between the outputs of two splits of the contraction
  };
  struct Warp : WarpBase {
    float alpha;
    template <int BN>
    __device__ __forceinline__ void before(const Params& e, const Problem&, int, int, int) {
      alpha = product_factor(e.scale);
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
      // the warps' halves of the columns are whole 64-column boxes
      constexpr int MID = (BN / 2 + 63) / 64 * 64;
      const int c0 = half ? MID : 0, c1 = half ? BN : MID;
      if (!e.f32) {
#pragma unroll 1
        for (int c = c0; c < c1; c += 64) {
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
        for (int c = c0; c < c1; c += 32) {
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

// The outputs of products whose contractions were split, in one launch (block row y
// takes out y):  out (+)= scale * (sum of the splits' partial products, in their
// order) + bias + resid, each optional; [rows, N] from slabs of [slab / N, N] fp32.
struct SlabSum {
  const float* slabs;
  int splits;
  int64_t slab;
  const float* scale;
  const __nv_bfloat16 *bias, *resid;
  void* out;
  int f32, accumulate;  // out's type: fp32, else bf16; += (fp32)
  int64_t n;
  int N;
};
struct SlabSums {
  SlabSum q[3];
};
static __global__ void __launch_bounds__(256) slab_sum_kernel(const SlabSums all) {
  pdl_wait();
  pdl_trigger();
  const SlabSum q = all.q[blockIdx.y];
  const float s = product_factor(q.scale);
  for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) * 4; i < q.n;
       i += (int64_t)gridDim.x * blockDim.x * 4) {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int z = 0; z < q.splits; ++z) {
      const float4 t = *reinterpret_cast<const float4*>(q.slabs + z * q.slab + i);
      a[0] += t.x;
      a[1] += t.y;
      a[2] += t.z;
      a[3] += t.w;
    }
    const int c = (int)(i % q.N);  // N is a multiple of 8
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] *= s;
      if (q.bias) a[k] += __bfloat162float(q.bias[c + k]);
      if (q.resid) a[k] += __bfloat162float(q.resid[i + k]);
    }
    if (!q.f32) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(q.out) + i) =
          make_uint2(pack2(a[0], a[1]), pack2(a[2], a[3]));
    } else {
      float4* out = reinterpret_cast<float4*>(static_cast<float*>(q.out) + i);
      if (q.accumulate) {
        const float4 t = *out;
        a[0] += t.x;
        a[1] += t.y;
        a[2] += t.z;
        a[3] += t.w;
      }
      *out = make_float4(a[0], a[1], a[2], a[3]);
    }
  }
}

// Rows of a slab: whole tiles, so that the rows of one never reach the next.
inline int slab_rows(int rows) { return (rows + 255) / 256 * 256; }
inline size_t slab_bytes(int rows, int N, int splits) {  // a multiple of 256: N of 8
  return splits > 1 ? (size_t)slab_rows(rows) * N * 4 * splits : 0;
}

// The split products of an operator, summed by one launch at its end.
struct Slabs {
  SlabSums all = {};
  int count = 0;
  char* ws;  // slab_bytes() for each, in turn
  explicit Slabs(void* p) : ws(static_cast<char*>(p)) {}
  // Output [M, N] of o, contiguous, in o.splits parts or at once; the optional terms
  // and `accumulate` are in e, and go to the sum where there are parts.
  bool output(Operands* o, int splits, EpiOut::Params* e, void* out, DType t) {
    o->splits = splits;
    if (splits == 1) return out_map(e, out, t, o->M, o->N, o->N);
    SlabSum& q = all.q[count++];
    q = {reinterpret_cast<float*>(ws), splits, (int64_t)slab_rows(o->M) * o->N, e->scale, e->bias,
         e->resid, out, t == DType::F32, e->accumulate, (int64_t)o->M * o->N, o->N};
    ws += slab_bytes(o->M, o->N, splits);
    *e = {};
    e->slab_rows = slab_rows(o->M);
    return out_map(e, const_cast<float*>(q.slabs), DType::F32, e->slab_rows * splits, o->N, o->N);
  }
  cudaError_t sum(cudaStream_t st) {
    if (count == 0) return cudaSuccess;
    int64_t n = 0;
    for (int i = 0; i < count; ++i) n = std::max(n, all.q[i].n);
    const dim3 grid((unsigned)std::min<int64_t>((n / 4 + 255) / 256, 152 * 8), (unsigned)count);
    return launch_pdl(slab_sum_kernel, grid, dim3(256), 0, st, all);
  }
};

// How a product [M, N] over K with few tiles is cut: columns per tile and splits
// of the contraction, by the clocks of the longest path: a K-slice takes about
// 512 of a CTA pair for 256 columns, 430 for 192 and 480 for 128 (operand bytes
// bound the narrow tiles), a tile 3000 more, and a split's partial products are
// written and read back at about 1600 bytes per clock, with a launch of 6000.
struct Cut {
  int bn, splits;
};
// narrow: tiles of fewer than 256 columns are possible.
inline Cut cut_of(int M, int N, int K, int slots, bool narrow) {
  const int nkb = (K + BKE - 1) / BKE, mp = (M + 2 * BM - 1) / (2 * BM);
  const int bn[3] = {256, 192, 128}, clk[3] = {512, 430, 480};
  Cut best{256, 1};
  double least = 1e30;
  for (int splits = 1; splits <= 8; ++splits) {
    const int kbs = (nkb + splits - 1) / splits;
    if (splits > 1 && kbs < 8) break;
    for (int i = 0; i < 3; ++i) {
      if (i > 0 && (splits > 1 || !narrow)) continue;  // a split has tiles enough
      const int64_t tiles = (int64_t)mp * ((N + bn[i] - 1) / bn[i]) * splits;
      double c = (double)((tiles + slots - 1) / slots) * ((double)kbs * clk[i] + 3000);
      if (splits > 1) c += 6000 + splits * (double)M * N * 8 / 1600;
      if (c < least * 0.97) {
        least = c;
        best = {bn[i], splits};
      }
    }
  }
  slices_per_split(K, &best.splits);
  return best;
}

// Splits of the contractions of N products that belong together: sizes[i] = {M, N, K}.
// In one launch where launch_group would take them (the operands stay in L2), no tile
// longer than an even share; else each as it is best alone.  The weight gradients of
// many rows and small weights are split too: 65536 x 512 x 1024 (dx, dw1, dw2) 625 ->
// 230 us, 8000 x 256 x 512 the backward 50 -> 30, the head's at 65536 x 256 x 8000
// 1176 -> 815.
template <int N>
bool split_together(const int (&sizes)[N][3]) {
  int64_t bytes = 0;
  for (const auto& q : sizes) bytes += operand_bytes(q[0], q[1], q[2]);
  return bytes <= GROUP_BYTES;
}
template <int N>
void splits_of(const int (&sizes)[N][3], bool together, int (&splits)[N]) {
  int64_t slices[N], all = 0;
  for (int i = 0; i < N; ++i) {
    const int* q = sizes[i];
    slices[i] = tiles256(q[0], q[1]) * ((q[2] + BKE - 1) / BKE + TILE_COST);
    all += slices[i];
  }
  for (int i = 0; i < N; ++i) {
    const int* q = sizes[i];
    splits[i] = together ? even_splits(tiles256(q[0], q[1]), q[2], all - slices[i], pair_count())
                         : cut_of(q[0], q[1], q[2], pair_count(), false).splits;
  }
}

}  // namespace core
}  // namespace oases
