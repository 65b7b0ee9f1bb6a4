// Gated feed-forward block, backward, with the projections computed again (bf16):
// a = x Wg^T + bg, b = x Wu^T + bu and dh = dy W2 of a tile of 256 rows x 128
// columns in one CTA pair's tensor memory, so that da = dh b act'(a), db = dh
// act(a) and h = act(a) b come from fp32 accumulators and neither a, b nor dh
// goes to memory.
//
// The roles of gemm_core.cuh: warp 0 loads, warp 1 issues the pair's MMAs, warps
// 2..9 are the epilogue.  Tensor memory: a in columns 0..127 and b in 128..255
// (one MMA of N = 256, gate rows of W1 in the even CTA and up rows in the odd
// one), dh in 256..383 or, every other tile, 384..511.  A tile begins with dh,
// while the epilogue still reads the tile before; a and b follow once it is done.
//
// At 1531 x 2048 x 5464 it takes 92 us; the projections to bf16 and back through
// memory, then the gradients, 57 + 44; at 1017 x 952 x 5344 43 against 29 + 31.  A
// K-slice takes 340 ns on average: 128-column MMAs of dh run at about half the
// rate of the 256-column ones, and rows of W2 do not start on 128-byte lines.
#include "glu.cuh"

namespace oases {
namespace {

constexpr int BM = 128, BKE = 64, NTHREADS = 320, TN = 128;
constexpr int A_BYTES = BM * 128, STAGE = 2 * A_BYTES;  // B: 128 rows of W1, or 64 columns of W2
constexpr int STG = 3 * 2048;                            // an epilogue warp's da, db and h
constexpr int STAGES = 5;
constexpr int EPI_OFF = STAGES * STAGE;
constexpr int BARS = EPI_OFF + 8 * STG;
constexpr int SMEM = BARS + 8 * (2 * STAGES + 3) + 8 + 1024;
static_assert(SMEM <= 227 * 1024, "shared memory");

struct Again {
  CUtensorMap x, w1, dy, w2;
  CUtensorMap da, db, h;  // boxes of 32 rows x 32 columns
  const __nv_bfloat16* b1;
  int M, H, F, act, num_mp, num_n, group;
};

__global__ void __launch_bounds__(NTHREADS, 1) glu_again_kernel(const __grid_constant__ Again g) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  auto full = [&](int s) { return base + BARS + 8u * s; };
  auto empty = [&](int s) { return base + BARS + 8u * (STAGES + s); };
  const uint32_t tfull = base + BARS + 8u * (2 * STAGES), tempty = tfull + 8, drain = tfull + 16;
  const uint32_t tslot = tfull + 24;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)ptx::cluster_rank();
  const int tiles = g.num_mp * g.num_n, first = blockIdx.x / 2, stride = gridDim.x / 2;
  const int nkb = (g.H + BKE - 1) / BKE;
  // row blocks fastest inside groups of g.group, as in gemm_core.cuh
  auto place = [&](int t, int& m0, int& n0) {
    const int q = t / (g.group * g.num_n), gm = min(g.group, g.num_mp - q * g.group);
    const int i = t - q * g.group * g.num_n;
    n0 = i / gm * TN;
    m0 = ((q * g.group + i % gm) * 2 + rank) * BM;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    ptx::mbar_init(tfull, 1);
    ptx::mbar_init(tempty, 16);  // the epilogue warps of the pair
    ptx::mbar_init(drain, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(tslot, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + (tslot - base));
  ptx::cluster_sync();  // the partner's barriers are initialised
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, iphase = 0;  // bit s: stage s loaded, parity of its last load
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride) {
        int m0, n0;
        place(t, m0, n0);
        for (int kb = 0; kb < 2 * nkb; ++kb) {
          const bool grad = kb < nkb;  // dy and W2, then x and W1
          const int k0 = (grad ? kb : kb - nkb) * BKE;
          if (!ptx::mbar_wait(empty(stage), phase ^ 1u)) { ok = false; break; }
          const uint32_t fb = ptx::mapa(full(stage), 0);
          if (rank == 0)
            ptx::mbar_arrive_expect_tx(full(stage), 2 * (grad ? A_BYTES + A_BYTES / 2 : STAGE));
          const uint32_t sa = base + stage * STAGE, sb = sa + A_BYTES;
          if (grad) {
            ptx::tma_load_2d_pair(sa, &g.dy, fb, k0, m0);
            ptx::tma_load_2d_pair(sb, &g.w2, fb, n0 + rank * 64, k0);
          } else {
            ptx::tma_load_2d_pair(sa, &g.x, fb, k0, m0);
            ptx::tma_load_2d_pair(sb, &g.w1, fb, k0, n0 + rank * g.F);
          }
          issued |= 1u << stage;
          iphase = (iphase & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // every load this thread issued has landed before the CTA leaves
      for (int s = 0; s < STAGES; ++s)
        if ((issued >> s) & 1u)
          if (!ptx::mbar_wait(rank == 0 ? full(s) : empty(s), (iphase >> s) & 1u)) ok = false;
      if (!ok) atomicExch(&core::g_core_error, 21);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {  // the even CTA issues the pair's MMAs
      constexpr uint32_t ID_DH = ptx::idesc_bf16_f32(2 * BM, TN, false, true);
      constexpr uint32_t ID_AB = ptx::idesc_bf16_f32(2 * BM, 2 * TN, false, false);
      int stage = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += stride, ++n) {
        for (int kb = 0; kb < 2 * nkb; ++kb) {
          const bool grad = kb < nkb;
          // a and b of the tile before have been read (and with them its dh, so
          // that the next tile's dh may take that place)
          if (kb == nkb && n > 0 && !ptx::mbar_wait(tempty, (uint32_t)(n - 1) & 1u)) { ok = false; break; }
          if (!ptx::mbar_wait(full(stage), phase)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t sa = base + stage * STAGE, sb = sa + A_BYTES;
          const uint64_t ad = ptx::smem_desc_sw128(sa, 16, 1024);
          const uint64_t bd = grad ? ptx::smem_desc_sw128(sb, 8192, 1024) : ptx::smem_desc_sw128(sb, 16, 1024);
          const uint32_t to = tmem + (grad ? 256u + 128u * (n & 1) : 0u);
          const int kb1 = grad ? kb : kb - nkb;
#pragma unroll
          for (int kk = 0; kk < BKE / 16; ++kk)
            ptx::mma_bf16_pair(to, ad + 2 * kk, bd + (uint64_t)(grad ? 128 * kk : 2 * kk),
                               grad ? ID_DH : ID_AB, (kb1 | kk) != 0 ? 1u : 0u);
          ptx::mma_commit_pair_mc(empty(stage), 3);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (ok) ptx::mma_commit_pair_mc(tfull, 3);
      }
      // all MMAs issued by this thread are complete before TMEM is freed
      ptx::mma_commit_pair(drain);
      if (!ptx::mbar_wait(drain, 0)) ok = false;
      if (!ok) atomicExch(&core::g_core_error, 22);
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stg = gbase + EPI_OFF + (warp - 2) * STG;
    const uint32_t stg_s = base + EPI_OFF + (warp - 2) * STG;
    int n = 0;
    for (int t = first; t < tiles; t += stride, ++n) {
      // the decision is warp-uniform: tcgen05.ld is warp-collective
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(tfull, (uint32_t)n & 1u))) {
        if (lane == 0) atomicExch(&core::g_core_error, 23);
        break;
      }
      ptx::tc_fence_after();
      int m0, n0;
      place(t, m0, n0);
      const int mw = m0 + quarter * 32;
      const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
      if (mw < g.M) {
#pragma unroll 1
        for (int c = half * 64; c < half * 64 + 64; c += 32) {
          const int col = n0 + c, left = g.F - col;
          if (left <= 0) break;
          float a[32], b[32], d[32];
          ptx::tmem_ld32x2(trow + c, trow + 128 + c, a, b);
          ptx::tmem_ld32(trow + 256 + 128 * (n & 1) + c, d);
          if (g.b1) {
            add_bias(g.b1 + col, left, a);
            add_bias(g.b1 + g.F + col, left, b);
          }
          uint32_t wa[16], wb[16], wh[16];
          if (g.act == OASES_ACT_SILU)
            gradients<OASES_ACT_SILU>(a, b, d, wa, wb, wh);
          else
            gradients<OASES_ACT_GELU>(a, b, d, wa, wb, wh);
          if (lane == 0) ptx::bulk_wait_read0();  // the last stores have read the staging
          __syncwarp();
          put_row(stg, lane, wa);
          put_row(stg + 2048, lane, wb);
          put_row(stg + 4096, lane, wh);
          ptx::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_2d(&g.da, stg_s, col, mw);
            ptx::tma_store_2d(&g.db, stg_s + 2048, col, mw);
            ptx::tma_store_2d(&g.h, stg_s + 4096, col, mw);
            ptx::bulk_commit();
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa(tempty, 0));
    }
    if (lane == 0) ptx::bulk_wait0();  // stores performed before the CTA retires
  }
  ptx::tc_fence_before();
  __syncthreads();
  // the pair's MMAs and every cross-CTA arrival are complete before either CTA
  // frees TMEM or leaves
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
  ptx::cluster_sync();
}

}  // namespace

cudaError_t glu_grad_again_tc(const GluShape& s, const void* x, const void* dy, const void* w1,
                              const void* b1, const void* w2, void* dpre, void* h, cudaStream_t st) {
  Again g = {};
  const int64_t F2 = 2 * (int64_t)s.F;
  if (!core::tensor_map(&g.x, x, false, s.H, s.M, s.H, BKE, BM) ||
      !core::tensor_map(&g.w1, w1, false, s.H, F2, s.H, BKE, BM) ||
      !core::tensor_map(&g.dy, dy, false, s.H, s.M, s.H, BKE, BM) ||
      !core::tensor_map(&g.w2, w2, false, s.F, s.H, s.F, 64, BKE) ||
      !halves(&g.da, &g.db, dpre, s.ldp, s, 32) ||
      !core::tensor_map(&g.h, h, false, s.F, s.M, s.ldh, 32, 32))
    return cudaErrorInvalidValue;
  g.b1 = static_cast<const __nv_bfloat16*>(b1);
  g.M = s.M;
  g.H = s.H;
  g.F = s.F;
  g.act = s.act;
  g.num_mp = (s.M + 2 * BM - 1) / (2 * BM);
  g.num_n = (s.F + TN - 1) / TN;
  g.group = 4ll * s.M * s.H > core::A_L2_BYTES ? std::min(core::GROUP_M, g.num_mp) : g.num_mp;
  static DeviceOnce attr;
  const cudaError_t ea = attr.run([&] {
    return cudaFuncSetAttribute(glu_again_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  });
  if (ea != cudaSuccess) return ea;
  const int64_t tiles = (int64_t)g.num_mp * g.num_n, slots = core::pair_count();
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t rounds = (tiles + slots - 1) / slots;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles + rounds - 1) / rounds) * 2);
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = 2;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  ++g_launch_count;
  return cudaLaunchKernelEx(&cfg, glu_again_kernel, g);
}

int glu_again_read_and_clear_error() { return core::read_and_clear_error(); }

}  // namespace oases
