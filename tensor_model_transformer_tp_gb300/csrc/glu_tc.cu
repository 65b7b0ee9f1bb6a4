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
// Bound by the product (4096 x 4096 x 11008 runs at 1.7 PFLOP/s with the second
// product, the rate the power limit sustains) where hidden is large, and by the
// writes of what is kept where it is small: at 4096 x 1024 x 4096 it takes 40 us
// keeping nothing and 57 keeping 67 MB of a and b, the same through plain stores
// as through TMA.
template <int KEEP>
struct EpiDual {
  static constexpr bool DUAL = true;
  static constexpr bool PAD_ROWS = KEEP == OASES_GLU_KEEP_MXFP8;  // scales of the rows past M
  // a buffer each for h and for what is kept of a and b: a tile's stores drain
  // while the next tile is computed
  static constexpr int STG = KEEP == OASES_GLU_KEEP_PRE ? 3 * 4096 : 4096, WBARS = 0;
  struct Params {
    CUtensorMap h, a, b;  // boxes of 32 rows x 64 columns of h, pre's halves
    const __nv_bfloat16* bias;
    int act;
    uint8_t *codes, *scales;
    int64_t ldq, code_stride, scale_stride;
    int kgroups;
  };
  struct Warp : WarpBase {
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
      wait_free();
      stage_row(wh);
      store_box(&e.h, n, mw);
      if constexpr (KEEP == OASES_GLU_KEEP_PRE) {
        stage_row(wa, 4096);
        store_box(&e.a, n, mw, 4096);
        stage_row(wb, 8192);
        store_box(&e.b, n, mw, 8192);
      }
    }
  };
};

// ---- gradients of the projections --------------------------------------------
// dh = dy W2 stays in the accumulator; the epilogue reads a and b of its
// elements and writes da = dh b act'(a), db = dh act(a) and h = act(a) b, 32
// columns of a warp's 32 rows at a time.  Two staging sets of three 2 KB
// buffers (64-byte rows, 64-byte swizzle) alternate: TMA brings a and b of the
// next 32 columns into one while the other's are turned, in place, into da and
// db, with h beside them, and stored.  (With one row per lane loaded straight
// from global memory, a cache-line lookup per lane, and the activation chosen
// per element, the kernel took 73 us at 4096 x 1024 x 4096; staged 61, with the
// choice outside the loops 48.)
// EIGHT: a and b come from the 8-bit form, 32 bytes of a row per lane (whole
// sectors), loaded one step ahead.
// What bounds it: the product takes 24 us there, the 100 MB it writes 25 at the
// 4 TB/s that fills reach, and it takes their sum; without its loads it takes 39,
// without loads and stores 24, without the arithmetic between them 45.  That is
// latency: the issue slots are 70% idle and DRAM at a third of its rate, because a, b
// and da, db share a staging set, and a request for the next a and b waits until every
// earlier store has read shared memory.  A warp's loads, arithmetic and stores so run
// one after the other.
template <bool EIGHT>
struct EpiGrad {
  static constexpr bool DUAL = false, PAD_ROWS = false;
  static constexpr int STG = 2 * 6144, WBARS = EIGHT ? 0 : 2;
  struct Params {
    CUtensorMap a, b;       // boxes of 32 rows x 32 columns of pre's halves
    CUtensorMap da, db, h;  // of dpre's halves and of h
    const uint8_t *codes, *scales;
    int64_t ldq, code_stride, scale_stride;
    int kgroups, act;
  };
  struct Warp : WarpBase {
    uint32_t count, asked;  // 32-column steps taken by this warp, and requested
    uint4 ca[2], cb[2];  // EIGHT: codes of the next step
    uint32_t sa, sb;     // and their scale bytes
    __device__ __forceinline__ void init() { count = asked = 0; }
    // Request a and b of columns n .. n+31 for the step `step`.
    __device__ __forceinline__ void request(const Params& e, const Problem& p, int mw, int n, uint32_t step) {
      if constexpr (EIGHT) {
        const int m = mw + lane, left = p.N - n;
        sa = sb = 127;
        ca[0] = ca[1] = cb[0] = cb[1] = make_uint4(0, 0, 0, 0);
        if (m < p.M && left > 0) {
          // codes rows are padded to 16 bytes, so a 16-byte load is whole
          const uint8_t* q = e.codes + (int64_t)m * e.ldq + n;
          const uint8_t* s = e.scales + sf_offset(m, n / MXB, e.kgroups);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (16 * i < left) {
              ca[i] = __ldg(reinterpret_cast<const uint4*>(q) + i);
              cb[i] = __ldg(reinterpret_cast<const uint4*>(q + e.code_stride) + i);
            }
          sa = __ldg(s);
          sb = __ldg(s + e.scale_stride);
        }
      } else if (lane == 0) {
        ptx::bulk_wait_read0();  // the set's last stores have read it
        const uint32_t set = step & 1u, at = stg_s + set * 6144;
        ptx::mbar_arrive_expect_tx(bars + 8 * set, 4096);
        ptx::tma_load_2d(at, &e.a, bars + 8 * set, n, mw);
        ptx::tma_load_2d(at + 2048, &e.b, bars + 8 * set, n, mw);
      }
      asked = step + 1;
    }
    __device__ __forceinline__ void finish() {  // a request that no step took
      if (!EIGHT && asked > count) ptx::mbar_wait(bars + 8 * (count & 1u), (count >> 1) & 1u);
    }
    template <int BN>
    __device__ __forceinline__ void before(const Params& e, const Problem& p, int mw, int n0, int half) {
      const int n = n0 + half * (BN / 2);
      if (mw < p.M && n < p.N) request(e, p, mw, n, count);
    }
    __device__ __forceinline__ void codes_to(const uint4& c, float x, float* v) {
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = e4m3x2_values((uint16_t)(w[k / 2] >> (16 * (k % 2))));
        v[2 * k] = f.x * x;
        v[2 * k + 1] = f.y * x;
      }
    }
    template <int BN>
    __device__ __forceinline__ void tile(const Params& e, const Problem& p, int mw, int n0, int half,
                                         int, uint32_t trow) {
#pragma unroll 1
      for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
        const int n = n0 + c;
        if (n >= p.N) break;
        const bool more = c + 32 < (half + 1) * (BN / 2) && n + 32 < p.N;
        const uint32_t set = count & 1u;
        float a[32], b[32], d[32];
        if constexpr (EIGHT) {
          const float xa = scale_value(sa), xb = scale_value(sb);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            codes_to(ca[i], xa, a + 16 * i);
            codes_to(cb[i], xb, b + 16 * i);
          }
          if (more) request(e, p, mw, n + 32, count + 1);
          wait_free_but_one();
        } else {
          if (more) request(e, p, mw, n + 32, count + 1);
          if (!__all_sync(0xffffffffu, ptx::mbar_wait(bars + 8 * set, (count >> 1) & 1u))) {
            if (lane == 0) atomicExch(&core::g_core_error, 4);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            unpack8(*row_unit(stg + set * 6144, lane, u), a + 8 * u);
            unpack8(*row_unit(stg + set * 6144 + 2048, lane, u), b + 8 * u);
          }
        }
        ptx::tmem_ld32(trow + c, d);
        uint32_t wa[16], wb[16], wh[16];
        if (e.act == OASES_ACT_SILU)
          gradients<OASES_ACT_SILU>(a, b, d, wa, wb, wh);
        else
          gradients<OASES_ACT_GELU>(a, b, d, wa, wb, wh);
        put_row(stg + set * 6144, lane, wa);
        put_row(stg + set * 6144 + 2048, lane, wb);
        put_row(stg + set * 6144 + 4096, lane, wh);
        ptx::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::tma_store_2d(&e.da, stg_s + set * 6144, n, mw);
          ptx::tma_store_2d(&e.db, stg_s + set * 6144 + 2048, n, mw);
          ptx::tma_store_2d(&e.h, stg_s + set * 6144 + 4096, n, mw);
          ptx::bulk_commit();
        }
        ++count;
      }
    }
    // EIGHT: at most the last step's stores still read shared memory
    __device__ __forceinline__ void wait_free_but_one() {
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();
    }
    __device__ __forceinline__ void unpack8(uint4 q, float* v) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2(w[k]);
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
      }
    }
  };
};

template <int KEEP>
cudaError_t project(const GluShape& s, const void* x, const void* w1, const void* b1, void* h,
                    void* pre, void* kept8, cudaStream_t st) {
  using E = EpiDual<KEEP>;
  typename E::Params e = {};
  e.bias = static_cast<const __nv_bfloat16*>(b1);
  e.act = s.act;
  if (!core::tensor_map(&e.h, h, false, s.F, s.M, s.ldh, 64, 32)) return cudaErrorInvalidValue;
  if (pre && !halves(&e.a, &e.b, pre, 2 * (int64_t)s.F, s, 64)) return cudaErrorInvalidValue;
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
  if (!halves(&e.da, &e.db, dpre, s.ldp, s, 32) ||
      !core::tensor_map(&e.h, h, false, s.F, s.M, s.ldh, 32, 32))
    return cudaErrorInvalidValue;
  if (!EIGHT) {
    if (!halves(&e.a, &e.b, pre, 2 * (int64_t)s.F, s, 32)) return cudaErrorInvalidValue;
  } else {
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
  if (s.M <= GLU_FEW_ROWS) return glu_project_few(s, x, w1, b1, h, pre, kept8, st);
  if (kept8) return project<OASES_GLU_KEEP_MXFP8>(s, x, w1, b1, h, nullptr, kept8, st);
  if (pre) return project<OASES_GLU_KEEP_PRE>(s, x, w1, b1, h, pre, nullptr, st);
  return project<OASES_GLU_KEEP_NONE>(s, x, w1, b1, h, nullptr, nullptr, st);
}

cudaError_t glu_grad_tc(const GluShape& s, const void* dy, const void* w2, const void* pre,
                        const void* kept8, void* dpre, void* h, cudaStream_t st) {
  return kept8 ? grad<true>(s, dy, w2, nullptr, kept8, dpre, h, st)
               : grad<false>(s, dy, w2, pre, nullptr, dpre, h, st);
}

namespace {

using core::EpiOut;

// dx, dw2 and dw1 and the splits of their contractions, the same ones whichever of
// them are wanted: a gradient does not depend on what else is asked for.
struct GradSplits {
  int sizes[3][3], splits[3];
  bool together;
  explicit GradSplits(const GluShape& s)
      : sizes{{s.M, s.H, 2 * s.F}, {s.H, s.F, s.M}, {2 * s.F, s.H, s.M}} {
    together = core::split_together(sizes);
    core::splits_of(sizes, together, splits);
  }
  size_t bytes() const {
    size_t n = 0;
    for (int i = 0; i < 3; ++i) n += core::slab_bytes(sizes[i][0], sizes[i][1], splits[i]);
    return n;
  }
};

}  // namespace

size_t glu_grads_tc_bytes(const GluShape& s) { return GradSplits(s).bytes(); }

cudaError_t glu_grads_tc(const GluShape& s, const void* x, const void* dy, const void* w1,
                         const void* dpre, const void* h, void* dx, void* dw1, void* dw2, char* ws,
                         cudaStream_t st) {
  core::Product prod[3] = {{{s.M, s.H, 2 * s.F, dpre, s.ldp, w1, s.H}, true},
                           {{s.H, s.F, s.M, dy, s.H, h, s.ldh}, false},
                           {{2 * s.F, s.H, s.M, dpre, s.ldp, x, s.H}, false}};
  EpiOut::Params ep[3] = {};
  void* const out[3] = {dx, dw2, dw1};
  const GradSplits g(s);
  core::Slabs slabs(ws);
  for (int i = 0; i < 3; ++i) {
    ep[i].accumulate = i > 0 && s.accumulate;
    if (out[i] && !slabs.output(&prod[i].o, g.splits[i], &ep[i], out[i], i > 0 ? s.grad_t : s.dx_t))
      return cudaErrorInvalidValue;
  }
  bool taken = false;
  if (g.together && dx && dw1 && dw2)
    OASES_TRY((core::launch_group<EpiOut, 3>(prod, ep, &taken, st)));
  if (!taken) {
    if (dw2) OASES_TRY((core::launch<EpiOut, 256, false, false, 2>(prod[1].o, ep[1], st)));
    if (dw1) OASES_TRY((core::launch<EpiOut, 256, false, false, 2>(prod[2].o, ep[2], st)));
    if (dx) OASES_TRY((core::launch<EpiOut, 256, true, false, 2>(prod[0].o, ep[0], st)));
  }
  return slabs.sum(st);
}

size_t glu_down_tc_bytes(const GluShape& s) {
  if (s.M <= GLU_FEW_ROWS) return 0;
  return core::slab_bytes(s.M, s.H, core::cut_of(s.M, s.H, s.F, core::pair_count(), true).splits);
}

cudaError_t glu_down_tc(const GluShape& s, const void* h, const void* w2, const void* b2,
                        const void* resid, void* y, char* ws, cudaStream_t st) {
  if (s.M <= GLU_FEW_ROWS) return glu_down_few(s, h, w2, b2, resid, y, st);
  const core::Cut c = core::cut_of(s.M, s.H, s.F, core::pair_count(), true);
  core::Operands o{s.M, s.H, s.F, h, s.ldh, w2, s.F};
  EpiOut::Params e = {};
  e.bias = static_cast<const __nv_bfloat16*>(b2);
  e.resid = static_cast<const __nv_bfloat16*>(resid);
  core::Slabs slabs(ws);
  if (!slabs.output(&o, c.splits, &e, y, DType::BF16)) return cudaErrorInvalidValue;
  if (c.bn == 128) return core::launch<EpiOut, 128, true, true, 2>(o, e, st);
  if (c.bn == 192) return core::launch<EpiOut, 192, true, true, 2>(o, e, st);
  OASES_TRY((core::launch<EpiOut, 256, true, true, 2>(o, e, st)));
  return slabs.sum(st);
}

int glu_read_and_clear_error() {
  const int v = core::read_and_clear_error(), w = glu_few_read_and_clear_error(),
            u = glu_again_read_and_clear_error();
  return v ? v : w ? w : u;
}

}  // namespace oases
