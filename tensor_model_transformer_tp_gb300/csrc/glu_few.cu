// Gated feed-forward block, forward, for few rows (a token of each of a few
// sequences): both products are bound by reading the weights once, so the
// weights are the M = 128 side of the MMA and the rows its N = 16 .. 128 side:
//   D[w, m] = sum_k W[w, k] x[m, k].
// A CTA owns 128 weight rows (up: 64 of Wg and the same 64 of Wu, so a and b of
// an output meet in one CTA) and a cluster of S CTAs splits the contraction;
// the partial D of the cluster meet through distributed shared memory, where
// each CTA sums, in the order of the splits, and finishes its share of the
// outputs.  Two CTAs per SM keep 190 KB of weight tiles in flight per SM.
// With the weights in memory, one row at 2560 x 6912 (106 MB) takes 22.5 us for
// both products, 4.7 TB/s; 16 rows at 4096 x 11008 (271 MB) 48.5, 5.6 TB/s; 61
// rows at 1024 x 2736 (17 MB) 13.8, two kernels' fixed costs.  One CTA per SM of
// twelve stages took 24.1, 59.8 and 15.2, four of three 23.8, 51.0 and 15.6, and
// asking for the second product's weights to be brought into L2 as the first's
// CTAs end 24.7, 53.5 and 13.9.  On the 256-row tiles of gemm_core.cuh the three
// took 53, 83 and 22, and 128 rows at 2560 x 6912 48 against 40.
//
// The second product's weight tiles are requested before the first kernel has
// finished: they depend on nothing that it writes, and every earlier kernel of
// the stream is complete when a dependent launch may start.
#include "gemm_core.cuh"
#include "glu.cuh"
#include "mx_block.cuh"

namespace oases {
namespace {

constexpr int BKE = 64, NTHREADS = 192;

template <int NT>
struct Few {
  static constexpr int W_BYTES = 128 * 128, X_BYTES = NT * 128, STAGE = W_BYTES + X_BYTES;
  static constexpr int STAGES = (108 * 1024) / STAGE;
  static constexpr int BAR_BYTES = 8 * (2 * STAGES + 1) + 8;
  static constexpr int SMEM = STAGES * STAGE + BAR_BYTES + 1024;
  static constexpr int TMEM_COLS = NT < 32 ? 32 : NT;
  static_assert(NT * 512 <= STAGES * STAGE, "the partial outputs take the stages' place");
};

struct FewArgs {
  int M, N, K;        // rows, outputs per row (ffn or hidden), contraction
  int kbs;            // K-slices per CTA of the cluster
  int split;          // CTAs of a cluster; the clusters follow one another in gridDim.x
  int act, keep;
  const __nv_bfloat16 *bias, *resid;
  __nv_bfloat16 *out;   // h [M, N] or y [M, N]
  __nv_bfloat16 *pre;   // [M, 2N]
  int64_t ldx, ldo;     // leading dimensions of x and out
  uint8_t *codes, *scales;
  int64_t ldq, code_stride, scale_stride;
  int kgroups;
};

template <int NT, bool UP>
__global__ void __launch_bounds__(NTHREADS)
glu_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const FewArgs g) {
  using C = Few<NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::STAGES * C::STAGE;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::STAGES + s); };
  const uint32_t done = bars + 8u * (2 * C::STAGES), tslot = done + 8;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int S = g.split, rank = (int)blockIdx.x % S;
  const int n0 = (int)blockIdx.x / S * (UP ? 64 : 128);
  const int nkb = (g.K + BKE - 1) / BKE;
  const int kb0 = min(nkb, rank * g.kbs), n = min(nkb, kb0 + g.kbs) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(done, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 5) {
    ptx::tmem_alloc(tslot, C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + (tslot - base));

  if (warp == 4) {
    if (lane == 0) {
      auto load_w = [&](int s, int kb) {
        ptx::mbar_arrive_expect_tx(full(s), C::STAGE);
        const uint32_t sw = base + s * C::STAGE;
        if (UP) {
          ptx::tma_load_2d(sw, &tmW, full(s), kb * BKE, n0);
          ptx::tma_load_2d(sw + 8192, &tmW, full(s), kb * BKE, g.N + n0);
        } else {
          ptx::tma_load_2d(sw, &tmW, full(s), kb * BKE, n0);
        }
      };
      auto load_x = [&](int s, int kb) {
        ptx::tma_load_2d(base + s * C::STAGE + C::W_BYTES, &tmX, full(s), kb * BKE, 0);
      };
      const int head = min(n, C::STAGES);
      bool ok = true;
      if (UP) pdl_wait();
      for (int i = 0; i < head; ++i) load_w(i, kb0 + i);
      if (!UP) pdl_wait();
      for (int i = 0; i < head; ++i) load_x(i, kb0 + i);
      int last = head;
      for (int i = head; i < n; ++i) {
        const int s = i % C::STAGES;
        if (!ptx::mbar_wait(empty(s), (uint32_t)(i / C::STAGES - 1) & 1u)) { ok = false; break; }
        load_w(s, kb0 + i);
        load_x(s, kb0 + i);
        last = i + 1;
      }
      // every load has landed before the CTA goes on
      for (int i = max(0, last - C::STAGES); i < last; ++i)
        if (!ptx::mbar_wait(full(i % C::STAGES), (uint32_t)(i / C::STAGES) & 1u)) ok = false;
      if (!ok) atomicExch(&core::g_core_error, 11);
    }
    __syncwarp();
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t IDESC = ptx::idesc_bf16_f32(128, NT, false, false);
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int s = i % C::STAGES;
        if (!ptx::mbar_wait(full(s), (uint32_t)(i / C::STAGES) & 1u)) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t sw = base + s * C::STAGE;
        const uint64_t ad = ptx::smem_desc_sw128(sw, 16, 1024);
        const uint64_t bd = ptx::smem_desc_sw128(sw + C::W_BYTES, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < BKE / 16; ++kk)
          ptx::mma_bf16(tmem, ad + 2 * kk, bd + 2 * kk, IDESC, (i | kk) != 0 ? 1u : 0u);
        ptx::mma_commit(empty(s));
      }
      ptx::mma_commit(done);  // all MMAs issued by this thread are complete
      if (!ok) atomicExch(&core::g_core_error, 12);
    }
    __syncwarp();
  }
  pdl_wait();
  pdl_trigger();
  // Every warp: this CTA's products are complete (and with them its loads).
  const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(done, 0));
  if (!ok && lane == 0) atomicExch(&core::g_core_error, 13);
  __syncthreads();
  ptx::tc_fence_after();
  // partial D to red[m][w], in the stages' place
  float* red = reinterpret_cast<float*>(gbase);
  if (warp < 4) {
#pragma unroll 1
    for (int c = 0; c < NT; c += 16) {
      float v[16], u[16];
      // (one 16-column load; the second address repeats it)
      ptx::tmem_ld16x2(tmem + ((uint32_t)(warp * 32) << 16) + c, tmem + ((uint32_t)(warp * 32) << 16) + c,
                       v, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) red[(c + i) * 128 + warp * 32 + lane] = n > 0 ? v[i] : 0.f;
    }
  }
  ptx::tc_fence_before();
  if (S > 1)
    ptx::cluster_sync();
  else
    __syncthreads();
  uint32_t from[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) from[s] = s < S ? ptx::mapa(base, (uint32_t)s) : 0u;
  auto total = [&](int at) {
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < S) v += ptx::ld_cluster(from[s] + 4u * at);
    return v;
  };
  constexpr int W = UP ? 64 : 128;  // outputs of a row in this cluster
  for (int i = rank * NTHREADS + (int)threadIdx.x; i < g.M * W; i += S * NTHREADS) {
    const int m = i / W, r = i % W, c = n0 + r;
    const bool in = c < g.N;
    if (UP) {
      float a = total(m * 128 + r), b = total(m * 128 + 64 + r);
      if (g.bias && in) {
        a += __bfloat162float(g.bias[c]);
        b += __bfloat162float(g.bias[g.N + c]);
      }
      if (g.keep == OASES_GLU_KEEP_PRE && in) {
        g.pre[(int64_t)m * 2 * g.N + c] = __float2bfloat16_rn(a);
        g.pre[(int64_t)m * 2 * g.N + g.N + c] = __float2bfloat16_rn(b);
      } else if (g.keep == OASES_GLU_KEEP_MXFP8) {
        // a warp holds 32 consecutive columns of a row: one scale block of each
        float ta = in ? fabsf(a) : 0.f, tb = in ? fabsf(b) : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, o));
          tb = fmaxf(tb, __shfl_xor_sync(0xffffffffu, tb, o));
        }
        const int xa = block_exponent(ta), xb = block_exponent(tb);
        if (in) {
          uint8_t* q = g.codes + (int64_t)m * g.ldq + c;
          q[0] = (uint8_t)e4m3x2(a * pow2_neg(xa), 0.f);
          q[g.code_stride] = (uint8_t)e4m3x2(b * pow2_neg(xb), 0.f);
        }
        if (lane == 0) {
          uint8_t* s = g.scales + sf_offset(m, c / MXB, g.kgroups);
          s[0] = (uint8_t)(xa + 127);
          s[g.scale_stride] = (uint8_t)(xb + 127);
        }
      }
      if (in) g.out[m * g.ldo + c] = __float2bfloat16_rn(act_fast(g.act, a) * b);
    } else if (in) {
      float v = total(m * 128 + r);
      if (g.bias) v += __bfloat162float(g.bias[c]);
      const int64_t at = m * g.ldo + c;  // resid's too
      if (g.resid) v += __bfloat162float(g.resid[at]);
      g.out[at] = __float2bfloat16_rn(v);
    }
  }
  if (UP && g.keep == OASES_GLU_KEEP_MXFP8) {  // scales of the rows past M
    for (int i = rank * NTHREADS + (int)threadIdx.x; i < (128 - g.M) * 2; i += S * NTHREADS) {
      uint8_t* s = g.scales + sf_offset(g.M + i / 2, n0 / MXB + i % 2, g.kgroups);
      s[0] = 127;
      s[g.scale_stride] = 127;
    }
  }
  __syncwarp();
  // no CTA leaves while another reads its partial D
  if (S > 1)
    ptx::cluster_sync();
  else
    __syncthreads();
  if (warp == 5) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
}

// The largest cluster for which two CTAs per SM hold the whole grid.
int few_split(int tiles, int nkb) {
  int S = 1;
  while (S < 8 && 2 * S * tiles <= 2 * core::sm_count() && 4 * S <= nkb) S *= 2;
  return S;
}

template <int NT, bool UP>
cudaError_t launch_few(FewArgs g, const void* w, const void* x, int tiles, cudaStream_t st) {
  using C = Few<NT>;
  CUtensorMap mw, mx;
  if (!core::tensor_map(&mw, w, false, g.K, UP ? 2 * (int64_t)g.N : g.N, g.K, BKE, UP ? 64 : 128) ||
      !core::tensor_map(&mx, x, false, g.K, g.M, g.ldx, BKE, NT))
    return cudaErrorInvalidValue;
  const int nkb = (g.K + BKE - 1) / BKE, S = few_split(tiles, nkb);
  g.kbs = (nkb + S - 1) / S;
  g.split = S;
  auto kern = glu_few_kernel<NT, UP>;
  static DeviceOnce attr;
  const cudaError_t ea = attr.run([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (ea != cudaSuccess) return ea;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S * tiles);  // x: wide weights have more than 65535 tiles
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = C::SMEM;
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
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, g);
}

template <bool UP>
cudaError_t dispatch(const FewArgs& g, const void* w, const void* x, int tiles, cudaStream_t st) {
  if (g.M <= 16) return launch_few<16, UP>(g, w, x, tiles, st);
  if (g.M <= 32) return launch_few<32, UP>(g, w, x, tiles, st);
  if (g.M <= 64) return launch_few<64, UP>(g, w, x, tiles, st);
  return launch_few<128, UP>(g, w, x, tiles, st);
}

}  // namespace

cudaError_t glu_project_few(const GluShape& s, const void* x, const void* w1, const void* b1,
                            void* h, void* pre, void* kept8, cudaStream_t st) {
  FewArgs g = {};
  g.M = s.M;
  g.N = s.F;
  g.K = s.H;
  g.act = s.act;
  g.bias = static_cast<const __nv_bfloat16*>(b1);
  g.out = static_cast<__nv_bfloat16*>(h);
  g.ldx = s.H;
  g.ldo = s.ldh;
  int tiles = (s.F + 63) / 64;
  if (kept8) {
    g.keep = OASES_GLU_KEEP_MXFP8;
    g.codes = static_cast<uint8_t*>(kept8);
    g.scales = g.codes + saved_scale_offset(s);
    g.ldq = s.ldq;
    g.code_stride = (int64_t)s.M * s.ldq;
    g.scale_stride = mx_sf_bytes(s.M, s.F);
    g.kgroups = (s.F + 127) / 128;
    tiles = 2 * g.kgroups;  // whole scale tiles
  } else if (pre) {
    g.keep = OASES_GLU_KEEP_PRE;
    g.pre = static_cast<__nv_bfloat16*>(pre);
  }
  return dispatch<true>(g, w1, x, tiles, st);
}

cudaError_t glu_down_few(const GluShape& s, const void* h, const void* w2, const void* b2,
                         const void* resid, void* y, cudaStream_t st) {
  FewArgs g = {};
  g.M = s.M;
  g.N = s.H;
  g.K = s.F;
  g.bias = static_cast<const __nv_bfloat16*>(b2);
  g.resid = static_cast<const __nv_bfloat16*>(resid);
  g.out = static_cast<__nv_bfloat16*>(y);
  g.ldx = s.ldh;
  g.ldo = s.H;
  return dispatch<false>(g, w2, h, (s.H + 127) / 128, st);
}

int glu_few_read_and_clear_error() { return core::read_and_clear_error(); }

}  // namespace oases
