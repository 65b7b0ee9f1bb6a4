// Tensor-core kernels of the gated feed-forward block (bf16): the main loop of
// gemm_core.cuh with the block's element-wise parts in its epilogues.
#include "epi_out.cuh"
#include "glu.cuh"
#include "mx_block.cuh"

namespace oases {
namespace {

using core::Problem;
using core::WarpBase;
using core::pack2;
using core::unpack2;

// ---- projections, activation and product -------------------------------------
// Tiles of 256 rows x 128 columns of a and the same of b (DUAL): every
// accumulator pair (a, b) of an output is in one thread, so h, and what is kept
// of a and b, leave from registers and the projections never go to memory.
template <int KEEP>
struct EpiDual {
  static constexpr bool DUAL = true;
  static constexpr bool PAD_ROWS = KEEP == OASES_GLU_KEEP_MXFP8;  // scales of the rows past M
  static constexpr int STG = 4096;
  struct Params {
    CUtensorMap h, a, b;  // boxes of 32 rows x 64 columns of h, pre's halves
    const __nv_bfloat16* bias;
    int act, want_h;
    uint8_t *codes, *scales;
    int64_t ldq, code_stride, scale_stride;
    int kgroups;
  };
  struct Warp : WarpBase {
    __device__ __forceinline__ void before(const Params&, const Problem&, int, int, int) {}
    __device__ __forceinline__ void add_bias(const __nv_bfloat16* src, int left, float (&v)[32]) {
#pragma unroll
      for (int i = 0; i < 32; i += 8)
        if (i < left) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + i));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2(w[k]);
            add2_inplace(v[i + 2 * k], v[i + 2 * k + 1], f.x, f.y);
          }
        }
    }
    // 32 columns of one row to E4M3 codes at q; returns the scale byte.
    // Columns at and past `left` (a multiple of 8) are not part of the matrix.
    __device__ __forceinline__ uint32_t keep8(const float (&v)[32], int left, bool row, uint8_t* q) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) amax = fmaxf(amax, i < left ? fabsf(v[i]) : 0.f);
      const int xe = block_exponent(amax);
      const float mul = pow2_neg(xe);
      if (row) {
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          if (i < left) {
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
              w[k] = (uint32_t)e4m3x2(v[i + 4 * k] * mul, v[i + 4 * k + 1] * mul) |
                     ((uint32_t)e4m3x2(v[i + 4 * k + 2] * mul, v[i + 4 * k + 3] * mul) << 16);
            *reinterpret_cast<uint2*>(q + i) = make_uint2(w[0], w[1]);
          }
      }
      return (uint32_t)(xe + 127);
    }
    template <int BN>
    __device__ __forceinline__ void tile(const Params& e, const Problem& p, int mw, int n0, int half,
                                         int, uint32_t trow) {
      const int m = mw + lane, c = half * (BN / 4), n = n0 + c;
      const bool row = m < p.M;
      if (KEEP == OASES_GLU_KEEP_MXFP8) {
        // scale bytes of columns n .. n+63 (blocks j, j+1 of a group of four);
        // rows and blocks past the matrix get 127
        if (n >= (p.N + 127) / 128 * 128) return;
      } else {
        if (n >= p.N) return;
      }
      uint32_t wh[32], wa[KEEP == OASES_GLU_KEEP_PRE ? 32 : 1], wb[KEEP == OASES_GLU_KEEP_PRE ? 32 : 1];
      uint32_t sa = 0, sb = 0;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float a[32], b[32];
        ptx::tmem_ld32x2(trow + c + 32 * hh, trow + BN / 2 + c + 32 * hh, a, b);
        const int left = p.N - (n + 32 * hh);
        if (e.bias) {
          add_bias(e.bias + n + 32 * hh, left, a);
          add_bias(e.bias + p.N + n + 32 * hh, left, b);
        }
        if (KEEP == OASES_GLU_KEEP_PRE) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            wa[16 * hh + i] = pack2(a[2 * i], a[2 * i + 1]);
            wb[16 * hh + i] = pack2(b[2 * i], b[2 * i + 1]);
          }
        }
        if (KEEP == OASES_GLU_KEEP_MXFP8) {
          uint8_t* q = e.codes + (int64_t)m * e.ldq + n + 32 * hh;
          const uint32_t xa = keep8(a, left, row, q), xb = keep8(b, left, row, q + e.code_stride);
          sa |= (row && left > 0 ? xa : 127u) << (8 * hh);
          sb |= (row && left > 0 ? xb : 127u) << (8 * hh);
        }
        if (e.act == OASES_ACT_SILU) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float f0, f1, s;
            silu(a[2 * i], f0, s);
            silu(a[2 * i + 1], f1, s);
            wh[16 * hh + i] = pack2(f0 * b[2 * i], f1 * b[2 * i + 1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            gelu2_inplace(a[2 * i], a[2 * i + 1]);
            wh[16 * hh + i] = pack2(a[2 * i] * b[2 * i], a[2 * i + 1] * b[2 * i + 1]);
          }
        }
      }
      if (KEEP == OASES_GLU_KEEP_MXFP8) {
        // two bytes of each operand's scale tile: row m, blocks n / 32, n / 32 + 1
        uint8_t* s = e.scales + ((int64_t)(m / 128) * e.kgroups + n / 128) * 512 + (m % 32) * 16 +
                     ((m % 128) / 32) * 4 + (n / 32) % 4;
        *reinterpret_cast<uint16_t*>(s) = (uint16_t)sa;
        *reinterpret_cast<uint16_t*>(s + e.scale_stride) = (uint16_t)sb;
      }
      if (n >= p.N || mw >= p.M) return;
      if (e.want_h) {
        wait_free();
        stage_row(wh);
        store_box(&e.h, n, mw);
      }
      if constexpr (KEEP == OASES_GLU_KEEP_PRE) {
        wait_free();
        stage_row(wa);
        store_box(&e.a, n, mw);
        wait_free();
        stage_row(wb);
        store_box(&e.b, n, mw);
      }
    }
  };
};

// ---- gradients of the projections --------------------------------------------
// dh = dy W2 stays in the accumulator; the epilogue reads a and b of its
// elements and writes da = dh b act'(a), db = dh act(a) and h = act(a) b.
template <bool EIGHT>
struct EpiGrad {
  static constexpr bool DUAL = false, PAD_ROWS = false;
  static constexpr int STG = 4096;
  struct Params {
    CUtensorMap da, db, h;  // boxes of 32 rows x 64 columns
    const __nv_bfloat16* pre;  // [M, 2F]
    const uint8_t *codes, *scales;
    int64_t ldq, code_stride, scale_stride;
    int kgroups, act;
  };
  struct Warp : WarpBase {
    __device__ __forceinline__ void before(const Params&, const Problem&, int, int, int) {}
    // 32 columns of one row; zeros past `left` columns (a multiple of 8)
    __device__ __forceinline__ void load_pre(const __nv_bfloat16* src, int left, bool row, float (&v)[32]) {
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (row && i < left) u = __ldg(reinterpret_cast<const uint4*>(src + i));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = unpack2(w[k]);
          v[i + 2 * k] = f.x;
          v[i + 2 * k + 1] = f.y;
        }
      }
    }
    __device__ __forceinline__ void load8(const uint8_t* q, uint32_t s, int left, bool row, float (&v)[32]) {
      const float x = scale_value(s);
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint2 u = make_uint2(0, 0);
        if (row && i < left) u = __ldg(reinterpret_cast<const uint2*>(q + i));
        const uint32_t w[2] = {u.x, u.y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = e4m3x2_values((uint16_t)(w[k / 2] >> (16 * (k % 2))));
          v[i + 2 * k] = f.x * x;
          v[i + 2 * k + 1] = f.y * x;
        }
      }
    }
    template <int BN>
    __device__ __forceinline__ void tile(const Params& e, const Problem& p, int mw, int n0, int half,
                                         int, uint32_t trow) {
      const int m = mw + lane;
      const bool row = m < p.M;
#pragma unroll 1
      for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 64) {
        const int n = n0 + c;
        if (n >= p.N) break;
        uint32_t wa[32], wb[32], wh[32];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int nn = n + 32 * hh, left = p.N - nn;
          float a[32], b[32], d[32];
          if (EIGHT) {
            const uint8_t* q = e.codes + (int64_t)m * e.ldq + nn;
            uint32_t sa = 127, sb = 127;
            if (row && left > 0) {
              const uint8_t* s = e.scales + ((int64_t)(m / 128) * e.kgroups + nn / 128) * 512 +
                                 (m % 32) * 16 + ((m % 128) / 32) * 4 + (nn / 32) % 4;
              sa = __ldg(s);
              sb = __ldg(s + e.scale_stride);
            }
            load8(q, sa, left, row, a);
            load8(q + e.code_stride, sb, left, row, b);
          } else {
            const __nv_bfloat16* q = e.pre + (int64_t)m * 2 * p.N + nn;
            load_pre(q, left, row, a);
            load_pre(q + p.N, left, row, b);
          }
          ptx::tmem_ld32(trow + c + 32 * hh, d);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float f0, f1, g0, g1;
            act_both_fast(e.act, a[2 * i], f0, g0);
            act_both_fast(e.act, a[2 * i + 1], f1, g1);
            const float d0 = d[2 * i], d1 = d[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
            wa[16 * hh + i] = pack2(d0 * b0 * g0, d1 * b1 * g1);
            wb[16 * hh + i] = pack2(d0 * f0, d1 * f1);
            wh[16 * hh + i] = pack2(f0 * b0, f1 * b1);
          }
        }
        wait_free();
        stage_row(wa);
        store_box(&e.da, n, mw);
        wait_free();
        stage_row(wb);
        store_box(&e.db, n, mw);
        wait_free();
        stage_row(wh);
        store_box(&e.h, n, mw);
      }
    }
  };
};

// Maps of the 32 x 64 boxes of pre's (or dpre's) two halves and of h.
bool halves(CUtensorMap* a, CUtensorMap* b, void* pre, const GluShape& s) {
  __nv_bfloat16* q = static_cast<__nv_bfloat16*>(pre);
  return core::tensor_map(a, q, false, s.F, s.M, 2 * (int64_t)s.F, 64, 32) &&
         core::tensor_map(b, q + s.F, false, s.F, s.M, 2 * (int64_t)s.F, 64, 32);
}

template <int KEEP>
cudaError_t project(const GluShape& s, const void* x, const void* w1, const void* b1, void* h,
                    void* pre, void* kept8, cudaStream_t st) {
  using E = EpiDual<KEEP>;
  typename E::Params e = {};
  e.bias = static_cast<const __nv_bfloat16*>(b1);
  e.act = s.act;
  e.want_h = h != nullptr;
  if (h && !core::tensor_map(&e.h, h, false, s.F, s.M, s.F, 64, 32)) return cudaErrorInvalidValue;
  if (pre && !halves(&e.a, &e.b, pre, s)) return cudaErrorInvalidValue;
  if (kept8) {
    e.codes = static_cast<uint8_t*>(kept8);
    e.scales = e.codes + saved_scale_offset(s);
    e.ldq = s.ldq;
    e.code_stride = (int64_t)s.M * s.ldq;
    e.scale_stride = mx_sf_bytes(s.M, s.F);
    e.kgroups = (s.F + 127) / 128;
  }
  core::Operands o{s.M, s.F, s.H, x, s.H, w1, s.H};
  o.b_off = s.F;
  return core::launch<E, 256, true, true, 2>(o, e, st);
}

template <bool EIGHT>
cudaError_t grad(const GluShape& s, const void* dy, const void* w2, const void* pre,
                 const void* kept8, void* dpre, void* h, cudaStream_t st) {
  using E = EpiGrad<EIGHT>;
  typename E::Params e = {};
  e.act = s.act;
  if (!halves(&e.da, &e.db, dpre, s) || !core::tensor_map(&e.h, h, false, s.F, s.M, s.F, 64, 32))
    return cudaErrorInvalidValue;
  e.pre = static_cast<const __nv_bfloat16*>(pre);
  if (EIGHT) {
    e.codes = static_cast<const uint8_t*>(kept8);
    e.scales = e.codes + saved_scale_offset(s);
    e.ldq = s.ldq;
    e.code_stride = (int64_t)s.M * s.ldq;
    e.scale_stride = mx_sf_bytes(s.M, s.F);
    e.kgroups = (s.F + 127) / 128;
  }
  core::Operands o{s.M, s.F, s.H, dy, s.H, w2, s.F};
  if (s.M <= 128) return core::launch<E, 128, true, false, 1>(o, e, st);
  return core::launch<E, 256, true, false, 2>(o, e, st);
}

}  // namespace

cudaError_t glu_project_tc(const GluShape& s, const void* x, const void* w1, const void* b1,
                           void* h, void* pre, void* kept8, cudaStream_t st) {
  if (s.M <= GLU_FEW_ROWS && h) return glu_project_few(s, x, w1, b1, h, pre, kept8, st);
  if (kept8) return project<OASES_GLU_KEEP_MXFP8>(s, x, w1, b1, h, nullptr, kept8, st);
  if (pre) return project<OASES_GLU_KEEP_PRE>(s, x, w1, b1, h, pre, nullptr, st);
  return project<OASES_GLU_KEEP_NONE>(s, x, w1, b1, h, nullptr, nullptr, st);
}

cudaError_t glu_grad_tc(const GluShape& s, const void* dy, const void* w2, const void* pre,
                        const void* kept8, void* dpre, void* h, cudaStream_t st) {
  return kept8 ? grad<true>(s, dy, w2, nullptr, kept8, dpre, h, st)
               : grad<false>(s, dy, w2, pre, nullptr, dpre, h, st);
}

cudaError_t glu_down_tc(const GluShape& s, const void* h, const void* w2, const void* b2,
                        const void* resid, void* y, cudaStream_t st) {
  if (s.M <= GLU_FEW_ROWS) return glu_down_few(s, h, w2, b2, resid, y, st);
  using E = core::EpiOut;
  E::Params e = {};
  if (!core::out_map(&e, y, DType::BF16, s.M, s.H, s.H)) return cudaErrorInvalidValue;
  e.bias = static_cast<const __nv_bfloat16*>(b2);
  e.resid = static_cast<const __nv_bfloat16*>(resid);
  core::Operands o{s.M, s.H, s.F, h, s.F, w2, s.F};
  const int tiles256 = (s.M + 127) / 128 * ((s.H + 255) / 256);
  if (2 * tiles256 < core::sm_count() || s.H <= 128)
    return core::launch<E, 128, true, true, 2>(o, e, st);
  return core::launch<E, 256, true, true, 2>(o, e, st);
}

int glu_read_and_clear_error() {
  const int v = core::read_and_clear_error(), w = glu_few_read_and_clear_error();
  return v ? v : w;
}

}  // namespace oases
