// Tensor-core kernels of the linear head's cross entropy (bf16): the main loop
// of gemm_core.cuh over tiles of rows x vocabulary, with the softmax in its
// epilogues, so that no logit leaves the chip.
#include "ce.cuh"
#include "epi_out.cuh"

namespace oases {
namespace {

using core::Problem;
using core::WarpBase;
using core::pack2;

constexpr float LOG2E = 1.4426950408889634f;
constexpr int64_t PART_BYTES = 256ll << 20;   // partial maxima and sums of the forward
// g of one piece of the backward.  A piece's dx is added to the others' in fp32,
// so pieces are long; 8192 x 50304 x 2560 takes 3.60 ms with 64 MB, 3.50 with 128,
// 3.42 with 256, 3.36 with 512, 3.30 with 1024; 2041 x 50257 x 1024 the same from
// 128 on.
constexpr int64_t PIECE_BYTES = 256ll << 20;
constexpr int MIN_PIECE = 4096;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- forward -------------------------------------------------------------------
// Bound by the product: 4096 x 32000 x 4096 runs at 1.8 PFLOP/s, 2041 x 50257 x
// 1024 in 105 us (the exponentials, 2048 clocks of a 256-column tile's 8192 at
// hidden 1024, hide behind the next tile's main loop); few rows by reading w:
// 37 x 50257 x 1024 in 19 us, 5.5 TB/s with the join.
// Each warp reduces its half of a tile's columns of its 32 rows, one row per
// lane, to (r, s): r the maximum of the logits, s the sum of e^(l - r) as
// 2^((l - r) log2 e); -inf and 0 where every logit is -inf.  The target's logit
// goes out as it is met.  The maximum is a logit as it is, not one rounded to
// base-2 units, and its own term is 1: so s >= 1, lse = r + log s is no less than
// any logit, and the loss of a row whose target has all the weight is 0.
struct EpiStat {
  static constexpr bool DUAL = false, PAD_ROWS = false;
  // Nothing is staged: the 8 KB keep the ring at six stages.  With seven, 2041 x 50257
  // x 1024 takes 133 us against 128 with the join, hidden 512 70 against 65.
  static constexpr int STG = 1024, WBARS = 0;
  struct Params {
    float2* part;  // [slots][M]
    float* at;     // [M]
    const int64_t* target;
  };
  struct Warp : WarpBase {
    int64_t t;
    template <int BN>
    __device__ __forceinline__ void before(const Params& e, const Problem& p, int mw, int, int) {
      const int m = mw + lane;
      t = m < p.M ? e.target[m] : -1;
    }
    template <int BN>
    __device__ __forceinline__ void tile(const Params& e, const Problem& p, int mw, int n0, int half,
                                         int, uint32_t trow) {
      const int m = mw + lane, nh = n0 + half * (BN / 2);
      if (nh >= p.N) return;
      float r = -INFINITY, s = 0.f;
#pragma unroll 1
      for (int c = 0; c < BN / 2; c += 64) {
        const int n = nh + c;
        if (n >= p.N) break;
        float v[64];
        ptx::tmem_ld32x2(trow + half * (BN / 2) + c, trow + half * (BN / 2) + c + 32,
                         *reinterpret_cast<float(*)[32]>(v), *reinterpret_cast<float(*)[32]>(v + 32));
        const int left = p.N - n;
        if (left < 64) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= left) v[i] = -INFINITY;
        }
        const int64_t d = t - n;
        const bool here = d >= 0 && d < min(64, left);
        if (__any_sync(0xffffffffu, here)) {
          float a = 0.f;
#pragma unroll
          for (int i = 0; i < 64; ++i) a = d == i ? v[i] : a;
          if (here && m < p.M) e.at[m] = a;
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = v[k];
#pragma unroll
        for (int i = 4; i < 64; ++i) mx[i % 4] = fmaxf(mx[i % 4], v[i]);
        const float top = fmaxf(r, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        const float ref = top == -INFINITY ? 0.f : top;
        s *= ex2((r - ref) * LOG2E);
        r = top;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        const uint64_t l2 = f2_splat(LOG2E), nr = f2_splat(-ref);
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const uint64_t q = f2_mul(f2_add(f2_pack(v[i], v[i + 1]), nr), l2);
          sum[i % 4] += ex2(f2_lo(q));
          sum[i % 4 + 1] += ex2(f2_hi(q));
        }
        s += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      if (m < p.M) e.part[(int64_t)(nh / (BN / 2)) * p.M + m] = make_float2(r, s);
    }
  };
};

// Joins the (r, s) of a row's slots in a fixed order: RB rows per block (whole
// sectors of `part` per slot), 512 / RB threads per row over the slots.
template <int RB>
__global__ void __launch_bounds__(512)
ce_join_kernel(const float2* part, int slots, const float* at, const int64_t* target, int64_t ignore,
               int V, int M, float* loss, float* lse) {
  constexpr int Y = 512 / RB;
  __shared__ float2 red[Y][RB + 1];
  pdl_wait();
  pdl_trigger();
  const int x = threadIdx.x % RB, y = threadIdx.x / RB, m = blockIdx.x * RB + x;
  float r = -INFINITY, s = 0.f;
  auto join = [&](float2 q) {
    const float top = fmaxf(r, q.x), ref = top == -INFINITY ? 0.f : top;
    s = s * exp2f((r - ref) * LOG2E) + q.y * exp2f((q.x - ref) * LOG2E);
    r = top;
  };
  if (m < M) {
#pragma unroll 4
    for (int i = y; i < slots; i += Y) join(part[(int64_t)i * M + m]);
  }
  red[y][x] = make_float2(r, s);
#pragma unroll
  for (int o = Y / 2; o; o >>= 1) {
    __syncthreads();
    if (y < o) {
      join(red[y + o][x]);
      red[y][x] = make_float2(r, s);
    }
  }
  if (y == 0 && m < M) {
    const float l = (r == -INFINITY ? 0.f : r) + logf(s);
    lse[m] = l;
    const int64_t t = target[m];
    loss[m] = row_loss(t, ignore, V, l, t >= 0 && t < V ? at[m] : 0.f);
  }
}

// ---- backward ------------------------------------------------------------------
// g / s of a piece, rounded to bf16: r (2^((l - lse) log2 e) - [v == target]), the
// difference first: a logit that has all the weight gives 1, not what the rounding of
// lse log2 e leaves (7e-4 off at logits of 16000).  Rows without a loss are 0 whatever
// their logits are.
struct EpiG {
  static constexpr bool DUAL = false, PAD_ROWS = false;
  static constexpr int STG = 4096, WBARS = 0;
  struct Params {
    CUtensorMap g;  // boxes of 32 rows x 64 columns of the piece
    CeRows rows;
    const float* lse;
    int v0;  // first column of the piece
  };
  struct Warp : WarpBase {
    int64_t t;
    float r, l;  // row factor, lse
    bool dead;
    template <int BN>
    __device__ __forceinline__ void before(const Params& e, const Problem& p, int mw, int, int) {
      const int m = mw + lane;
      t = -1;
      r = l = 0.f;
      dead = true;
      if (m < p.M) {
        t = e.rows.target[m];
        dead = t == e.rows.ignore;
        r = row_factor(e.rows, t, m);
        l = e.lse[m];
        t -= e.v0;
      }
    }
    template <int BN>
    __device__ __forceinline__ void tile(const Params& e, const Problem& p, int mw, int n0, int half,
                                         int, uint32_t trow) {
#pragma unroll 1
      for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 64) {
        const int n = n0 + c;
        if (n >= p.N) break;
        float v[64];
        ptx::tmem_ld32x2(trow + c, trow + c + 32, *reinterpret_cast<float(*)[32]>(v),
                         *reinterpret_cast<float(*)[32]>(v + 32));
        const uint64_t le = f2_splat(LOG2E), nl = f2_splat(-l);
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const uint64_t q = f2_mul(f2_add(f2_pack(v[i], v[i + 1]), nl), le);
          v[i] = ex2(f2_lo(q));
          v[i + 1] = ex2(f2_hi(q));
        }
        const int64_t d = t - n;
        if (__any_sync(0xffffffffu, d >= 0 && d < 64)) {
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] -= d == i ? 1.f : 0.f;
        }
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = dead ? 0u : pack2(v[2 * i] * r, v[2 * i + 1] * r);
        wait_free();
        stage_row(w);
        store_box(&e.g, n, mw);
      }
    }
  };
};

// Tiles of the logits: 128 columns while one row block holds every row (the
// product is bound by reading w, and 128-column tiles spread it over more SMs),
// else 256-column CTA-pair tiles.
int stat_slots(const CeShape& s) { return (s.V + (s.M <= 128 ? 63 : 127)) / (s.M <= 128 ? 64 : 128); }
// Rows per pass of the forward: the partial results of a pass fit PART_BYTES.
int fwd_rows(const CeShape& s) {
  const int64_t fit = PART_BYTES / (8ll * stat_slots(s)) / 256 * 256;
  return (int)std::min<int64_t>(s.M, std::max<int64_t>(fit, 256));
}

struct BwdPlan {
  int piece, splits, dw_splits;  // columns of a piece, splits of dx and of dw
  bool together;                 // dx and dw of a piece may share a launch
  int64_t ld;
  size_t dx, total;  // g of a piece comes first, then the earlier pieces' dx
};
BwdPlan bwd_plan(const CeShape& s) {  // the same whichever gradients are wanted
  BwdPlan b;
  const int64_t fit = PIECE_BYTES / (2ll * s.M) / 256 * 256;
  const int pieces = (int)((s.V + std::max<int64_t>(fit, MIN_PIECE) - 1) / std::max<int64_t>(fit, MIN_PIECE));
  b.piece = pieces == 1 ? s.V : ((s.V + pieces - 1) / pieces + 255) / 256 * 256;
  b.ld = ((int64_t)b.piece + 63) / 64 * 64;  // rows on 128-byte lines
  const int sizes[2][3] = {{s.M, s.H, b.piece}, {b.piece, s.H, s.M}};
  int splits[2];
  // dx of few rows has few tiles, each a contraction over the whole vocabulary:
  // split over the SMs, up to 128 rows in a launch of its own (it reads w at
  // 5.5 TB/s; with dw's tiles, which only write, 49 x 2024 x 40704 took 95 us
  // against 30 + 61 apart)
  b.together = s.M > 128 && core::split_together(sizes);
  core::splits_of(sizes, b.together, splits);
  b.splits = pieces > 1 ? 1 : splits[0];  // a piece's dx is added to the others'
  b.dw_splits = splits[1];
  if (pieces == 1 && s.M <= 128) {
    b.splits = std::max(1, std::min(core::sm_count() / ((s.H + 127) / 128), s.V / 512));
    core::slices_per_split(s.V, &b.splits);
  }
  b.dx = align256((size_t)s.M * b.ld * 2);
  b.total = b.dx;
  if (pieces > 1) b.total += align256((size_t)s.M * s.H * 4);
  b.total += core::slab_bytes(s.M, s.H, b.splits) + core::slab_bytes(b.piece, s.H, b.dw_splits);
  return b;
}

}  // namespace

size_t ce_tc_fwd_bytes(const CeShape& s) {
  const size_t rows = fwd_rows(s);
  return align256(rows * stat_slots(s) * 8) + align256(rows * 4);
}

cudaError_t ce_tc_fwd(const CeShape& s, const void* x, const void* w, const int64_t* target,
                      float* loss, float* lse, char* ws, cudaStream_t st) {
  const int step = fwd_rows(s), slots = stat_slots(s);
  EpiStat::Params e;
  e.part = reinterpret_cast<float2*>(ws);
  e.at = reinterpret_cast<float*>(ws + align256((size_t)step * slots * 8));
  for (int m0 = 0; m0 < s.M; m0 += step) {
    const int M = std::min(step, s.M - m0);
    e.target = target + m0;
    core::Operands o{M, s.V, s.H, static_cast<const __nv_bfloat16*>(x) + (int64_t)m0 * s.H, s.H, w, s.H};
    OASES_TRY(s.M <= 128 ? (core::launch<EpiStat, 128, true, true, 1>(o, e, st))
                         : (core::launch<EpiStat, 256, true, true, 2>(o, e, st)));
    OASES_TRY(ce_join(e.part, slots, e.at, e.target, s, M, loss + m0, lse + m0, st));
  }
  return cudaSuccess;
}

cudaError_t ce_join(const float2* part, int slots, const float* at, const int64_t* target,
                    const CeShape& s, int M, float* loss, float* lse, cudaStream_t st) {
  // few rows: more threads per row, for the latency of the chain of joins
  if (M <= 512)
    return launch_pdl(ce_join_kernel<4>, dim3((M + 3) / 4), dim3(512), 0, st, part, slots, at, target,
                      s.ignore, s.V, M, loss, lse);
  return launch_pdl(ce_join_kernel<16>, dim3((M + 15) / 16), dim3(512), 0, st, part, slots, at, target,
                    s.ignore, s.V, M, loss, lse);
}

size_t ce_tc_bwd_bytes(const CeShape& s) { return bwd_plan(s).total; }

cudaError_t ce_tc_bwd(const CeShape& s, const void* x, const void* w, const CeRows& rows,
                      const float* lse, void* dx, void* dw, char* ws, cudaStream_t st) {
  using core::EpiOut;
  const BwdPlan b = bwd_plan(s);
  void* g = ws;
  float* dx32 = reinterpret_cast<float*>(ws + b.dx);
  const bool few = s.M <= 128;
  for (int v0 = 0; v0 < s.V; v0 += b.piece) {
    const int n = std::min(b.piece, s.V - v0);
    const bool first = v0 == 0, last = v0 + n == s.V;
    const __nv_bfloat16* wp = static_cast<const __nv_bfloat16*>(w) + (int64_t)v0 * s.H;
    {
      EpiG::Params e;
      if (!core::tensor_map(&e.g, g, false, n, s.M, b.ld, 64, 32)) return cudaErrorInvalidValue;
      e.rows = rows;
      e.lse = lse;
      e.v0 = v0;
      core::Operands o{s.M, n, s.H, x, s.H, wp, s.H};
      OASES_TRY(few ? (core::launch<EpiG, 128, true, true, 1>(o, e, st))
                    : (core::launch<EpiG, 256, true, true, 2>(o, e, st)));
    }
    core::Product prod[2] = {{{s.M, s.H, n, g, b.ld, wp, s.H}, true},
                             {{n, s.H, s.M, g, b.ld, x, s.H}, false}};
    EpiOut::Params ep[2] = {};
    core::Slabs slabs(dx32 + (b.piece < s.V ? align256((size_t)s.M * s.H * 4) / 4 : 0));
    if (dx) {
      if (last) {
        ep[0].scale = rows.scale;
        ep[0].prior = first ? nullptr : dx32;
      } else {
        ep[0].accumulate = !first;
      }
      if (!slabs.output(&prod[0].o, b.splits, &ep[0], last ? dx : dx32, last ? DType::BF16 : DType::F32))
        return cudaErrorInvalidValue;
    }
    if (dw) {
      char* out = static_cast<char*>(dw) + (size_t)v0 * s.H * dtype_size(s.grad_t);
      ep[1].scale = rows.scale;
      ep[1].accumulate = s.accumulate;
      if (!slabs.output(&prod[1].o, b.dw_splits, &ep[1], out, s.grad_t)) return cudaErrorInvalidValue;
    }
    bool taken = false;
    if (b.together && dx && dw) OASES_TRY((core::launch_group<EpiOut, 2>(prod, ep, &taken, st)));
    if (!taken) {
      if (dx)
        OASES_TRY(few ? (core::launch<EpiOut, 128, true, false, 1>(prod[0].o, ep[0], st))
                      : (core::launch<EpiOut, 256, true, false, 2>(prod[0].o, ep[0], st)));
      if (dw) OASES_TRY((core::launch<EpiOut, 256, false, false, 2>(prod[1].o, ep[1], st)));
    }
    OASES_TRY(slabs.sum(st));
  }
  return cudaSuccess;
}

int ce_read_and_clear_error() { return core::read_and_clear_error(); }

}  // namespace oases
