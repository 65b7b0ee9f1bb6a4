// Attention over keys of another length, backward, on the 5th-generation tensor cores
// (bf16 in, fp32 between the products).
//
//   P = e^(s - lse), delta = rowsum(dO * O), dP = dO V^T, dS = P (dP - delta),
//   dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO, and dS summed by bucket.
// Two kernels own disjoint outputs, so there are no atomics:
//   dq kernel   persistent: items of 128 queries, looped over blocks of 128 keys
//   dkv kernel  a CTA per 128 keys of a key head, looped over its query heads and
//               blocks of 64 queries
// and dS is formed twice (9 products of the definition's 7).  Both are pipelines of one
// TMA warp, two MMA-issuing threads (one for S and dP, one for the accumulations: a
// thread that issued both would wait at one's barrier while the other's operands are
// ready) and 16 element-wise warps, four per TMEM lane quarter.  P and dS are rounded
// to bf16, the operand type; the bias's gradient sums dS before that.
//
// The bias's gradient (dkv kernel).  A warp's 32 x 16 scores that lie R or more from the
// diagonal on one side belong to one bucket: every thread adds its own.  Nearer ones are
// summed along their 47 diagonals, by passing a running sum from lane to lane as the column
// advances (lane r adds element (r, c) at step c, so a sum that moves one lane a step
// stays on its diagonal), and the sums of each bucket's run of diagonals are added to
// the warp's own buckets in shared memory: a fixed order throughout.
#include <math.h>

#include <algorithm>

#include "xattn_tc.cuh"

namespace oases {

__device__ int g_xattn_bwd_error;

namespace {
using namespace xattn;

constexpr uint64_t WAIT = 1ull << 29;  // cycles before a wait gives up (~0.25 s)
constexpr int NT = 608, ACC_WARP = 18, EW = 16;
constexpr int BOX64 = 64 * 64 * 2;  // one TMA box of 64 rows
constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t IDESC_N64 = ptx::idesc_bf16_f32(128, 64, false, false);

__device__ __forceinline__ void wait_failed(int site) { atomicCAS(&g_xattn_bwd_error, 0, site); }
__device__ __forceinline__ bool wait1(uint32_t bar, uint32_t parity) { return ptx::mbar_wait(bar, parity, WAIT); }
// Warp-uniform bounded wait (every lane waits; the warp agrees on the outcome).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait1(bar, parity));
}
// A row's lse in base 2; a query without keys: every weight 0.
__device__ __forceinline__ float lse2_of(float lse) { return lse == -INFINITY ? INFINITY : lse * LOG2E; }

struct Plan {
  Args a;
  int tiles, items;  // dq: 128-query tiles; dkv: 128-key tiles
  float scale_log2;
};

// delta: 16 lanes a row, 16 bytes each.
__global__ void __launch_bounds__(256)
xattn_delta_kernel(const __grid_constant__ Args a, int64_t rows) {
  pdl_wait();
  pdl_trigger();
  const int64_t r = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 16;  // (batch, query, head)
  const int c = threadIdx.x % 16 * 8;
  float d = 0.f;
  int64_t at = 0;
  if (r < rows) {
    const int64_t bq = r / a.H, b = bq / a.Sq;
    const int h = (int)(r - bq * a.H), qi = (int)(bq - b * a.Sq);
    at = a.stat((int)b, h, qi);
    if (c < a.D) {
      const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.o) + b * a.so.b +
                                                      qi * a.so.s + h * a.so.h + c);
      const uint4 y = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.d_o) + b * a.sdo.b +
                                                      qi * a.sdo.s + h * a.sdo.h + c);
      const uint32_t u[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(w[i] << 16), d);
        d = fmaf(__uint_as_float(u[i] & 0xffff0000u), __uint_as_float(w[i] & 0xffff0000u), d);
      }
    }
  }
#pragma unroll
  for (int o = 8; o; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
  if (r < rows && c == 0) a.delta[at] = d;
}

// ---- dq ---------------------------------------------------------------------------------
// 608 threads: warp 0 TMA (per item K_0 and V_0, then Q and dO, then the K_j and V_j
// rings, which run on across items), warp 1 TMEM and the S and dP MMAs, warps 2..17
// element-wise (lanes 32 (w % 4) .. of a block, columns 32 ((w - 2) / 4) ..), warp 18 the
// dQ MMAs.  TMEM: S 0..127, dP 128..255, dQ 256.., dS (packed bf16) 384..447.  S and dP
// have one buffer each: the element-wise warps load their columns and release both at
// once, so the next block's are formed while they work.
template <int DP>
struct DqSmem {
  static constexpr int TILE = tile_bytes<DP>();
  static constexpr int KST = DP == 64 ? 4 : 3, VST = DP == 64 ? 4 : 2;
  static constexpr int Q = 0, DO = TILE, K = 2 * TILE, V = K + KST * TILE;
  static constexpr int BAR = V + VST * TILE;
  static constexpr int NBAR = 8 + 2 * KST + 2 * VST;
  static constexpr int BYTES = BAR + 8 * NBAR + 16 + 1024;
  static_assert(BYTES <= 232448, "more than 227 KB of shared memory");
};

struct DqItem {
  int h, b, q0, p0, len, n, tile;  // head, sequence, first query and its position, keys, key blocks
};
__device__ __forceinline__ DqItem dq_item(const Plan& p, int i) {
  const Args& a = p.a;
  const int bh = a.H * a.B;
  DqItem it;
  it.tile = p.tiles - 1 - i / bh;
  const int r = i % bh;
  it.h = r % a.H;
  it.b = r / a.H;
  it.q0 = it.tile * 128;
  it.len = a.len(it.b);
  it.p0 = a.start(it.b) + it.q0;
  const int rows = min(128, a.Sq - it.q0);
  const int vis = a.causal ? min(it.len, max(0, it.p0 + rows)) : it.len;
  it.n = (vis + 127) / 128;
  return it;
}

template <int DP, bool BIAS>
__global__ void __launch_bounds__(NT, 1)
xattn_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                const __grid_constant__ Plan p) {
  using L = DqSmem<DP>;
  constexpr int TILE = L::TILE, KST = L::KST, VST = L::VST;
  constexpr uint32_t IDESC_DQ = ptx::idesc_bf16_f32(128, DP, false, true);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::BAR;
  const uint32_t qdo_full = bars, qdo_empty = bars + 8u, sdp_full = bars + 16u, sdp_empty = bars + 24u;
  const uint32_t ds_full = bars + 32u, ds_empty = bars + 40u, bar_fin = bars + 48u, sdp_drain = bars + 56u;
  auto k_full = [&](uint32_t s) { return bars + 8u * (8 + s); };
  auto k_empty = [&](uint32_t s) { return bars + 8u * (8 + KST + s); };
  auto v_full = [&](uint32_t s) { return bars + 8u * (8 + 2 * KST + s); };
  auto v_empty = [&](uint32_t s) { return bars + 8u * (8 + 2 * KST + VST + s); };
  const uint32_t tslot = bars + 8u * L::NBAR;
  const Args& a = p.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int cta = blockIdx.x, G = gridDim.x;

  if (tid == 0) {
    ptx::mbar_init(qdo_full, 1);
    ptx::mbar_init(qdo_empty, 1);
    ptx::mbar_init(sdp_full, 1);
    ptx::mbar_init(sdp_empty, EW);
    ptx::mbar_init(ds_full, EW);
    ptx::mbar_init(ds_empty, 1);
    ptx::mbar_init(bar_fin, 1);
    ptx::mbar_init(sdp_drain, 1);
    for (int s = 0; s < 2 * KST + 2 * VST; ++s) ptx::mbar_init(k_full(s), 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tq);
    ptx::prefetch_tmap(&tdo);
    ptx::prefetch_tmap(&tk);
    ptx::prefetch_tmap(&tv);
  }
  if (warp == 1) {
    ptx::tmem_alloc(tslot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + (tslot - base));
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dq = tmem + 256, t_ds = tmem + 384;
  pdl_wait();
  pdl_trigger();
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t ke = 0, nq = 0;  // ring entries (of K and of V) and Q/dO tiles loaded
      auto load_kv = [&](int r, int g, int b) {
        const uint32_t sk = ke % KST, uk = ke / KST, sv = ke % VST, uv = ke / VST;
        if (uk > 0 && !wait1(k_empty(sk), (uk - 1) & 1)) return false;
        ptx::mbar_arrive_expect_tx(k_full(sk), TILE);
        load_tile<DP, 128>(base + L::K + sk * TILE, &tk, k_full(sk), r, g, b);
        bool landed = true;
        if (uv > 0) landed = wait1(v_empty(sv), (uv - 1) & 1);
        if (landed) {
          ptx::mbar_arrive_expect_tx(v_full(sv), TILE);
          load_tile<DP, 128>(base + L::V + sv * TILE, &tv, v_full(sv), r, g, b);
          ++ke;
        } else {  // (K's load of this entry must land too before the CTA exits)
          (void)wait1(k_full(sk), uk & 1);
        }
        return landed;
      };
      for (int k = 0; ok; ++k) {
        const int i = persistent_item(k, cta, G);
        if (i >= p.items) break;
        const DqItem it = dq_item(p, i);
        if (it.n == 0) continue;
        const int g = it.h / a.share;
        ok = load_kv(0, g, it.b);
        // Q and dO are free once the previous item's last S and dP are done
        if (ok && nq > 0 && !wait1(qdo_empty, (nq - 1) & 1)) ok = false;
        if (!ok) break;
        ptx::mbar_arrive_expect_tx(qdo_full, 2 * TILE);
        load_tile<DP, 128>(base + L::Q, &tq, qdo_full, it.q0, it.h, it.b);
        load_tile<DP, 128>(base + L::DO, &tdo, qdo_full, it.q0, it.h, it.b);
        ++nq;
        for (int j = 1; j < it.n && ok; ++j) ok = load_kv(j * 128, g, it.b);
      }
      if (!ok) wait_failed(101);
      // every load issued has landed before the CTA may exit
      bool dr = true;
      for (uint32_t s = 0; s < KST; ++s)
        if (ke > s) dr = wait1(k_full(s), ((ke - 1 - s) / KST) & 1) && dr;
      for (uint32_t s = 0; s < VST; ++s)
        if (ke > s) dr = wait1(v_full(s), ((ke - 1 - s) / VST) & 1) && dr;
      if (nq > 0) dr = wait1(qdo_full, (nq - 1) & 1) && dr;
      if (!dr) wait_failed(102);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t g = 0, nq = 0;  // blocks (= ring entries) and items with blocks so far
      for (int k = 0; ok; ++k) {
        const int i = persistent_item(k, cta, G);
        if (i >= p.items) break;
        const DqItem it = dq_item(p, i);
        if (it.n == 0) continue;
        if (!wait1(qdo_full, nq & 1)) {
          ok = false;
          wait_failed(103);
          break;
        }
        ++nq;
        for (int j = 0; j < it.n && ok; ++j, ++g) {  // S_j = Q K_j^T, dP_j = dO V_j^T
          const uint32_t sk = g % KST, sv = g % VST;
          // (the element-wise warps have loaded the previous block's S and dP)
          if (!wait1(k_full(sk), (g / KST) & 1) || !wait1(v_full(sv), (g / VST) & 1) ||
              (g >= 1 && !wait1(sdp_empty, (g - 1) & 1))) {
            ok = false;
            wait_failed(104);
            break;
          }
          ptx::tc_fence_after();
          const uint32_t kt = base + L::K + sk * TILE, vt = base + L::V + sv * TILE;
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk)
            ptx::mma_bf16(t_s, kmajor_desc(base + L::Q, kk), kmajor_desc(kt, kk), IDESC_S, kk > 0);
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk)
            ptx::mma_bf16(t_dp, kmajor_desc(base + L::DO, kk), kmajor_desc(vt, kk), IDESC_S, kk > 0);
          ptx::mma_commit(sdp_full);
          ptx::mma_commit(v_empty(sv));
          if (j + 1 == it.n) ptx::mma_commit(qdo_empty);  // the item's last read of Q and dO
        }
      }
      ptx::mma_commit(sdp_drain);  // completes once every MMA this thread issued has
      if (!wait1(sdp_drain, 0)) {
        ok = false;
        wait_failed(107);
      }
    }
  } else if (warp == ACC_WARP) {
    if (lane == 0) {
      uint32_t g = 0, nk = 0;  // blocks, items with blocks finished
      for (int k = 0; ok; ++k) {
        const int i = persistent_item(k, cta, G);
        if (i >= p.items) break;
        const DqItem it = dq_item(p, i);
        if (it.n == 0) continue;
        for (int j = 0; j < it.n && ok; ++j, ++g) {  // dQ += dS_j K_j
          const uint32_t sk = g % KST;
          if (!wait1(ds_full, g & 1)) {
            ok = false;
            wait_failed(106);
            break;
          }
          ptx::tc_fence_after();
          const uint32_t kt = base + L::K + sk * TILE;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            ptx::mma_bf16_ts(t_dq, t_ds + 8u * kk, mnmajor_desc(kt, kk), IDESC_DQ, (j > 0 || kk > 0) ? 1u : 0u);
          // S_j, dP_j (which also read K_j) completed before dS_j could be handed over,
          // so K_j is free once these MMAs are
          ptx::mma_commit(ds_empty);
          ptx::mma_commit(k_empty(sk));
        }
        if (!ok) break;
        ptx::mma_commit(bar_fin);  // the item's dQ is complete once this does
        ++nk;
      }
      // every MMA this thread issued is complete before the CTA may exit
      if (nk > 0 && !wait1(bar_fin, (nk - 1) & 1)) {
        ok = false;
        wait_failed(111);
      }
      if (!ok) {  // one more commit drains whatever was issued after the last finished item
        ptx::mma_commit(bar_fin);
        (void)wait1(bar_fin, nk & 1);
      }
    }
  } else {
    const int qq = warp & 3, sub = (warp - 2) >> 2;  // lane quarter; columns 32 sub .. + 31
    const int row = qq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qq * 32) << 16;
    uint32_t g = 0, nf = 0;
    // this row's LSE (base 2) and delta of an item, read one item ahead
    auto stats = [&](int i, float& lse2, float& dlt) {
      lse2 = INFINITY;
      dlt = 0.f;
      if (i >= p.items) return;
      const DqItem it = dq_item(p, i);
      if (it.q0 + row < a.Sq) {
        const int64_t at = a.stat(it.b, it.h, it.q0 + row);
        lse2 = lse2_of(a.lse[at]);
        dlt = a.delta[at];
      }
    };
    float lse2_next, dlt_next;
    stats(persistent_item(0, cta, G), lse2_next, dlt_next);
    for (int k = 0; ok; ++k) {
      const int i = persistent_item(k, cta, G);
      if (i >= p.items) break;
      const DqItem it = dq_item(p, i);
      const int qi = it.q0 + row;
      const bool valid_q = qi < a.Sq;
      const float lse2 = lse2_next, dlt = dlt_next;
      stats(persistent_item(k + 1, cta, G), lse2_next, dlt_next);
      const int w0 = it.p0 + qq * 32;  // position of the warp's first query
      float left = 0.f, right = 0.f;
      if (BIAS) {
        left = *a.bias.at(it.h, -a.bias.R);
        right = *a.bias.at(it.h, a.bias.R);
      }
      for (int j = 0; j < it.n && ok; ++j, ++g) {
        if (!warp_wait(sdp_full, g & 1)) {
          ok = false;
          if (lane == 0) wait_failed(108);
          break;
        }
        ptx::tc_fence_after();
        float v[32], w[32];
        ptx::tmem_ld32x2(t_s + lane_off + sub * 32, t_dp + lane_off + sub * 32, v, w);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sdp_empty);  // the TMEM buffers may be overwritten
        const int kb = j * 128 + sub * 32;
        // 32 x 32 scores wholly visible need no mask (warp-uniform)
        const bool full = it.q0 + qq * 32 + 32 <= a.Sq && kb + 32 <= it.len && (!a.causal || kb + 31 <= w0);
        const bool on_right = BIAS && kb - (w0 + 31) >= a.bias.R;
        const bool on_left = BIAS && !on_right && kb + 31 - w0 <= -a.bias.R;
        const bool near = BIAS && !on_left && !on_right;
        const float shift = (on_right ? right : on_left ? left : 0.f) - lse2;
        float mul = p.scale_log2;
        if (near) {
          const float* bv = a.bias.at(it.h, kb - w0) - lane;
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = fmaf(v[c], p.scale_log2, __ldg(bv + c));
          mul = 1.f;
        }
        uint32_t pk[16];  // dS as packed bf16 pairs (keys 2i, 2i+1 of these 32)
        if (full) {
          const uint64_t sc = f2_splat(mul), sh = f2_splat(shift), nd = f2_splat(-dlt);
#pragma unroll
          for (int i2 = 0; i2 < 16; ++i2) {
            const uint64_t x = f2_fma(f2_pack(v[2 * i2], v[2 * i2 + 1]), sc, sh);
            const uint64_t pr = f2_pack(fast_exp2(f2_lo(x)), fast_exp2(f2_hi(x)));
            const uint64_t ds = f2_mul(pr, f2_add(f2_pack(w[2 * i2], w[2 * i2 + 1]), nd));
            pk[i2] = pack2(f2_lo(ds), f2_hi(ds));
          }
        } else {
          // keys kb + c with c >= nvis are past the diagonal or the sequence's keys (all
          // of them for a row past the queries)
          const int nvis = valid_q ? (a.causal ? min(w0 + lane + 1, it.len) : it.len) - kb : 0;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float e = fast_exp2(fmaf(v[c], mul, shift));
            v[c] = c < nvis ? e * (w[c] - dlt) : 0.f;
          }
#pragma unroll
          for (int i2 = 0; i2 < 16; ++i2) pk[i2] = pack2(v[2 * i2], v[2 * i2 + 1]);
        }
        // the dS columns are free once the previous block's dQ MMAs are done
        if (g >= 1 && !warp_wait(ds_empty, (g - 1) & 1)) {
          ok = false;
          if (lane == 0) wait_failed(109);
          break;
        }
        ptx::tc_fence_after();
        ptx::tmem_st16_nowait(t_ds + lane_off + sub * 16, pk);
        // the keys behind the sequence's, where the tensor goes on: their rows of K
        // cleared (S and dP of this block, which also read the tile, are complete)
        if (j * 128 + 128 > it.len && it.len < a.Sk) {
          const int r = (warp - 2) * 8 + lane / 4;
          if (j * 128 + r >= it.len) {
            uint8_t* kr = gbase + L::K + g % KST * TILE + r * 128 + (lane & 3) * 32;
#pragma unroll
            for (int c = 0; c < DP / 64; ++c) {
              *reinterpret_cast<uint4*>(kr + c * BOX) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(kr + c * BOX + 16) = make_uint4(0, 0, 0, 0);
            }
          }
          ptx::fence_async_smem();
          __syncwarp();
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ds_full);
      }
      if (!ok) break;
      bool fin = true;
      float v0[32];
      if (it.n > 0) {
        // the item's last accumulation is complete (or the MMA thread gave up)
        fin = warp_wait(bar_fin, nf & 1);
        ++nf;
        ptx::tc_fence_after();
        // tcgen05.ld is warp-collective: every lane loads (DP = 64: what the last two
        // column groups load is not used)
        ptx::tmem_ld32(t_dq + lane_off + sub * 32, v0);
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) v0[c] = 0.f;
      }
      if (fin && valid_q && sub * 32 < DP) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.dq) + it.b * a.sdq.b + qi * a.sdq.s + it.h * a.sdq.h + sub * 32;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (sub * 32 + 8 * u < a.D)
            *reinterpret_cast<uint4*>(out + 8 * u) =
                make_uint4(pack2(v0[8 * u] * a.scale, v0[8 * u + 1] * a.scale),
                           pack2(v0[8 * u + 2] * a.scale, v0[8 * u + 3] * a.scale),
                           pack2(v0[8 * u + 4] * a.scale, v0[8 * u + 5] * a.scale),
                           pack2(v0[8 * u + 6] * a.scale, v0[8 * u + 7] * a.scale));
      }
      if (!fin) {
        ok = false;
        if (lane == 0) wait_failed(112);
      }
    }
  }
  if (!ok) atomicCAS(&g_xattn_bwd_error, 0, 3);
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ---- dk, dv -------------------------------------------------------------------------------
// 608 threads: warp 0 TMA (K and V once, then Q_i and dO_i into a ring, each stage with
// its queries' lse and delta), warp 1 TMEM and the S^T and dP^T MMAs (N = 64, two buffers),
// warps 2..17 element-wise (lanes 32 (w % 4) .., one key row each, columns 16 ((w - 2) / 4) ..),
// warp 18 the dV and dK MMAs.  A warp writes P^T and dS^T, packed, over the first 8 of
// its own 16 columns of S^T and dP^T: one 16-query step of the accumulations' A operand,
// read from tensor memory.  (From shared memory the operands' reads bound the kernel:
// 224 KB a block at 128 bytes a clock against 1024 clocks of products, 160 KB so.)
// TMEM: buffer b's S^T at 128 b .. + 63, dP^T at + 64 .., dV 256 .., dK 384 ..
template <int DP, bool BIAS>
struct KvSmem {
  static constexpr int TILE = tile_bytes<DP>(), T64 = TILE / 2;
  static constexpr int QST = DP == 64 ? 8 : BIAS ? 4 : 5;
  static constexpr int K = 0, V = TILE, Q = 2 * TILE, DO = Q + QST * T64;
  static constexpr int STAT = DO + QST * T64;                              // [stage][lse2[64] | delta[64]] fp32
  static constexpr int BUCKET = STAT + QST * 2 * 64 * 4;                   // [16][MAX_BUCKETS] fp32
  static constexpr int DIAG = BUCKET + (BIAS ? EW * MAX_BUCKETS * 4 : 0);  // [16][48] fp32
  static constexpr int BAR = DIAG + (BIAS ? EW * 48 * 4 : 0);
  static constexpr int NBAR = 9 + 2 * QST;
  static constexpr int USED = BAR + 8 * NBAR + 16;
  // the tiles need 1024-byte alignment: the window starts so aligned on this GPU, and
  // the kernel checks that what rounding takes is there
  static constexpr int BYTES = USED + 1024 <= 232448 ? USED + 1024 : 232448;
  static_assert(USED <= 232448, "more than 227 KB of shared memory");
};

template <int DP, bool BIAS>
__global__ void __launch_bounds__(NT, 1)
xattn_dkv_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                 const __grid_constant__ Plan p) {
  using L = KvSmem<DP, BIAS>;
  constexpr int TILE = L::TILE, T64 = L::T64, QST = L::QST;
  constexpr uint32_t IDESC_ACC = ptx::idesc_bf16_f32(128, DP, false, true);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  if (base - raw + L::USED > (uint32_t)L::BYTES) {  // (uniform: every thread leaves)
    if (threadIdx.x == 0) wait_failed(6);
    return;
  }
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::BAR;
  const uint32_t bar_kv = bars, bar_fin = bars + 8u, sdp_drain = bars + 16u;
  auto sdp_full = [&](int b) { return bars + 8u * (3 + b); };   // S^T and dP^T formed
  auto pd_full = [&](int b) { return bars + 8u * (5 + b); };    // P^T and dS^T written over them
  auto pd_empty = [&](int b) { return bars + 8u * (7 + b); };   // and read
  auto q_full = [&](int s) { return bars + 8u * (9 + s); };
  auto q_empty = [&](int s) { return bars + 8u * (9 + QST + s); };
  const uint32_t tslot = bars + 8u * L::NBAR;
  float* stat = reinterpret_cast<float*>(gbase + L::STAT);
  const Args& a = p.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (tid == 0) {
    ptx::mbar_init(bar_kv, 1);
    ptx::mbar_init(bar_fin, 1);
    ptx::mbar_init(sdp_drain, 1);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(sdp_full(b), 1);
      ptx::mbar_init(pd_full(b), EW);
      ptx::mbar_init(pd_empty(b), 1);
    }
    for (int s = 0; s < 2 * QST; ++s) ptx::mbar_init(q_full(s), 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tk);
    ptx::prefetch_tmap(&tv);
    ptx::prefetch_tmap(&tq);
    ptx::prefetch_tmap(&tdo);
  }
  if (warp == 1) {
    ptx::tmem_alloc(tslot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + (tslot - base));
  auto t_st = [&](int b) { return tmem + (uint32_t)(b * 128); };
  auto t_dpt = [&](int b) { return tmem + (uint32_t)(b * 128 + 64); };
  const uint32_t t_dv = tmem + 256, t_dk = tmem + 384;
  pdl_wait();
  pdl_trigger();
  bool ok = true;

  // key tile 0 (causal: the most query blocks) first
  int u = blockIdx.x;
  const int g = u % a.G;
  u /= a.G;
  const int bb = u % a.B, k0 = u / a.B * 128;
  const int len = a.len(bb), p0 = a.start(bb);
  const int i0 = a.causal ? max(0, k0 - p0) / 64 : 0;  // blocks before see none of these keys
  const int per_head = k0 < len ? max(0, (a.Sq + 63) / 64 - i0) : 0;
  const int n = per_head * a.share;
  // block ii: of query head g share + ii / per_head, its query block i0 + ii % per_head

  if (warp == 0) {
    if (lane == 0 && n > 0) {
      ptx::mbar_arrive_expect_tx(bar_kv, 2 * TILE);
      load_tile<DP, 128>(base + L::K, &tk, bar_kv, k0, g, bb);
      load_tile<DP, 128>(base + L::V, &tv, bar_kv, k0, g, bb);
    }
    // lse (log2 units) and delta of block ii's 64 queries, two of each per lane; the
    // next block's are loaded before the wait for its stage
    int hh = 0, i = i0 - 1;  // of the block loaded last
    auto ld_stat = [&](int ii, float (&v)[4]) {
      if (++i == i0 + per_head) {
        i = i0;
        ++hh;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int qi = i * 64 + lane + 32 * x;
        const bool in = ii < n && qi < a.Sq;
        const int64_t at = in ? a.stat(bb, g * a.share + hh, qi) : 0;
        v[x] = in ? lse2_of(a.lse[at]) : INFINITY;
        v[2 + x] = in ? a.delta[at] : 0.f;
      }
    };
    float cur[4];
    if (n > 0) ld_stat(0, cur);
    int nl = 0;  // query blocks whose loads were issued
    for (int ii = 0; ii < n; ++ii) {
      const int s = ii % QST, ci = i, ch = hh;
      float nxt[4];
      ld_stat(ii + 1, nxt);
      bool w = true;
      if (lane == 0 && ii >= QST) w = wait1(q_empty(s), ((ii / QST) & 1) ^ 1);
      if (!__shfl_sync(0xffffffffu, w, 0)) {
        ok = false;
        if (lane == 0) wait_failed(201);
        break;
      }
      float* st = stat + s * 128;
      st[lane] = cur[0];
      st[lane + 32] = cur[1];
      st[64 + lane] = cur[2];
      st[64 + lane + 32] = cur[3];
      __syncwarp();  // the warp's stores precede lane 0's arrive on the stage barrier
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(q_full(s), 2 * T64);
        load_tile<DP, 64>(base + L::Q + s * T64, &tq, q_full(s), ci * 64, g * a.share + ch, bb);
        load_tile<DP, 64>(base + L::DO + s * T64, &tdo, q_full(s), ci * 64, g * a.share + ch, bb);
      }
      nl = ii + 1;
#pragma unroll
      for (int x = 0; x < 4; ++x) cur[x] = nxt[x];
    }
    if (lane == 0 && n > 0) {
      // every load issued has landed before the CTA may exit
      bool dr = wait1(bar_kv, 0);
      for (int s = 0; s < QST && s < nl; ++s) dr = wait1(q_full(s), ((nl - 1 - s) / QST) & 1) && dr;
      if (!dr) wait_failed(202);
    }
  } else if (warp == 1) {
    if (lane == 0 && n > 0) {
      ok = wait1(bar_kv, 0);
      if (!ok) wait_failed(203);
      for (int ii = 0; ii < n && ok; ++ii) {  // S^T = K Q_i^T, dP^T = V dO_i^T into buffer ii % 2
        const int s = ii % QST, b = ii & 1;
        if (!wait1(q_full(s), (ii / QST) & 1) ||
            (ii >= 2 && !wait1(pd_empty(b), ((ii / 2) & 1) ^ 1))) {  // (block ii - 2 is done with)
          ok = false;
          wait_failed(204);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t qt = base + L::Q + s * T64, dt = base + L::DO + s * T64;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
          ptx::mma_bf16(t_st(b), kmajor_desc(base + L::K, kk), kmajor_desc(qt, kk, BOX64), IDESC_N64, kk > 0);
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
          ptx::mma_bf16(t_dpt(b), kmajor_desc(base + L::V, kk), kmajor_desc(dt, kk, BOX64), IDESC_N64, kk > 0);
        ptx::mma_commit(sdp_full(b));
      }
      ptx::mma_commit(sdp_drain);  // completes once every MMA this thread issued has
      if (!wait1(sdp_drain, 0)) {
        ok = false;
        wait_failed(207);
      }
    }
  } else if (warp == ACC_WARP) {
    if (lane == 0 && n > 0) {
      for (int ii = 0; ii < n && ok; ++ii) {  // dV += P^T dO_i, dK += dS^T Q_i
        const int s = ii % QST, b = ii & 1;
        if (!wait1(pd_full(b), (ii / 2) & 1)) {
          ok = false;
          wait_failed(206);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t qt = base + L::Q + s * T64, dt = base + L::DO + s * T64;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t accum = (ii > 0 || kk > 0) ? 1u : 0u;
          ptx::mma_bf16_ts(t_dv, t_st(b) + 16u * kk, mnmajor_desc(dt, kk, BOX64), IDESC_ACC, accum);
          ptx::mma_bf16_ts(t_dk, t_dpt(b) + 16u * kk, mnmajor_desc(qt, kk, BOX64), IDESC_ACC, accum);
        }
        // S^T, dP^T of block ii (which also read Q_i, dO_i) completed before P^T and
        // dS^T could be handed over: the stage is free once these MMAs are
        ptx::mma_commit(pd_empty(b));
        ptx::mma_commit(q_empty(s));
      }
      ptx::mma_commit(bar_fin);  // completes once every MMA this thread issued has
      if (!wait1(bar_fin, 0)) {
        ok = false;
        wait_failed(211);
      }
    }
  } else {
    const int qq = warp & 3, c = (warp - 2) >> 2;  // lane quarter; columns 16 c .. + 15
    const int row = qq * 32 + lane, kj = k0 + row, kw = k0 + qq * 32;
    const bool valid_k = kj < len;
    const uint32_t lane_off = (uint32_t)(qq * 32) << 16;
    int hh = 0, i = i0 - 1;
    float left = 0.f, right = 0.f, far_left = 0.f, far_right = 0.f;
    const bool grad = BIAS && a.bias_part != nullptr;
    float* bucket = reinterpret_cast<float*>(gbase + L::BUCKET) + (warp - 2) * MAX_BUCKETS;
    float* diag = reinterpret_cast<float*>(gbase + L::DIAG) + (warp - 2) * 48;
    if (grad) {
      for (int x = lane; x < a.bias.buckets; x += 32) bucket[x] = 0.f;
      __syncwarp();
    }
    auto flush = [&](int head) {  // the warp's buckets of a finished head, and 0 for the next
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        far_left += __shfl_xor_sync(~0u, far_left, o);
        far_right += __shfl_xor_sync(~0u, far_right, o);
      }
      if (lane == 0) {
        bucket[a.bias.left] += far_left;
        bucket[a.bias.right] += far_right;
      }
      __syncwarp();
      far_left = far_right = 0.f;
      float* out = a.bias_part + ((((int64_t)(g * a.share + head) * a.B + bb) * p.tiles + k0 / 128) * EW + (warp - 2)) *
                                     a.bias.buckets;
      for (int x = lane; x < a.bias.buckets; x += 32) {
        out[x] = bucket[x];
        bucket[x] = 0.f;
      }
      __syncwarp();
    };
    for (int ii = 0; ii < n && ok; ++ii) {
      const int s = ii % QST, b = ii & 1;
      if (++i == i0 + per_head) {
        if (grad) flush(hh);
        i = i0;
        ++hh;
      }
      if (BIAS && i == i0) {
        left = *a.bias.at(g * a.share + hh, -a.bias.R);
        right = *a.bias.at(g * a.share + hh, a.bias.R);
      }
      // this block's S^T, dP^T are in TMEM (which also means its stage, and the lse and
      // delta stored with it, have landed)
      if (!warp_wait(sdp_full(b), (ii / 2) & 1) || !warp_wait(q_full(s), (ii / QST) & 1)) {
        ok = false;
        if (lane == 0) wait_failed(208);
        break;
      }
      ptx::tc_fence_after();
      float v[16], w[16];
      ptx::tmem_ld16x2(t_st(b) + lane_off + c * 16, t_dpt(b) + lane_off + c * 16, v, w);
      const float* st = stat + s * 128 + c * 16;  // lse of these 16 queries; delta at + 64
      const int qb = i * 64 + c * 16;
      float mul = p.scale_log2, add = 0.f;
      const bool on_right = BIAS && kw - (p0 + qb + 15) >= a.bias.R;
      const bool on_left = BIAS && !on_right && kw + 31 - (p0 + qb) <= -a.bias.R;
      if (BIAS) {
        if (on_right) {
          add = right;
        } else if (on_left) {
          add = left;
        } else {
          const float* bv = a.bias.at(g * a.share + hh, kj - (p0 + qb));
#pragma unroll
          for (int x = 0; x < 16; ++x) v[x] = fmaf(v[x], p.scale_log2, __ldg(bv - x));
          mul = 1.f;
        }
      }
      uint32_t pp[8], pd[8];
      // scores wholly visible need no mask (warp-uniform)
      const bool full = kw + 32 <= len && qb + 16 <= a.Sq && (!a.causal || p0 + qb >= kw + 31);
      if (full) {
        const uint64_t sc = f2_splat(mul), ad = f2_splat(add);
#pragma unroll
        for (int x = 0; x < 16; x += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(st + x);
          const float4 d4 = *reinterpret_cast<const float4*>(st + 64 + x);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float l0 = e == 0 ? l4.x : l4.z, l1 = e == 0 ? l4.y : l4.w;
            const float d0 = e == 0 ? d4.x : d4.z, d1 = e == 0 ? d4.y : d4.w;
            uint64_t sh = f2_pack(-l0, -l1);
            if (BIAS) sh = f2_add(sh, ad);
            const uint64_t y = f2_fma(f2_pack(v[x + e], v[x + e + 1]), sc, sh);
            const uint64_t pr = f2_pack(fast_exp2(f2_lo(y)), fast_exp2(f2_hi(y)));
            const uint64_t ds = f2_mul(pr, f2_add(f2_pack(w[x + e], w[x + e + 1]), f2_pack(-d0, -d1)));
            pp[(x + e) / 2] = pack2(f2_lo(pr), f2_hi(pr));
            pd[(x + e) / 2] = pack2(f2_lo(ds), f2_hi(ds));
            if (BIAS) {
              w[x + e] = f2_lo(ds);
              w[x + e + 1] = f2_hi(ds);
            }
          }
        }
      } else {
        // queries qb + x with x < lo are before this key (causal), those with x >= hi past
        // the last; a key past the sequence's sees none
        const int lo = a.causal ? kj - p0 - qb : -(1 << 30), hi = valid_k ? a.Sq - qb : 0;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const bool in = x >= lo && x < hi;
          const float e = fast_exp2(fmaf(v[x], mul, add - st[x]));
          v[x] = in ? e : 0.f;
          w[x] = in ? e * (w[x] - st[64 + x]) : 0.f;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          pp[x] = pack2(v[2 * x], v[2 * x + 1]);
          pd[x] = pack2(w[2 * x], w[2 * x + 1]);
        }
      }
      ptx::tmem_st8_nowait(t_st(b) + lane_off + c * 16, pp);
      ptx::tmem_st8_nowait(t_dpt(b) + lane_off + c * 16, pd);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(pd_full(b));
      if (!grad) continue;
      if (!on_left && !on_right) {
        // sums along the diagonals, that of element (r, x) r - x + 15
        float run = 0.f;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          run = __shfl_up_sync(0xffffffffu, run, 1);
          run = (lane == 0 ? 0.f : run) + w[x];
          if (lane == 31) diag[46 - x] = run;
        }
        if (lane < 31) diag[lane] = run;
        __syncwarp();
        const int n0 = kw - (p0 + qb) - 15;  // the distance of diagonal 0
        for (int x = lane; x < a.bias.buckets; x += 32) {
          const int2 r = a.bias.range[x];
          float y = 0.f;
          for (int d = max(0, r.x - n0); d <= min(46, r.y - n0); ++d) y += diag[d];
          bucket[x] += y;
        }
        __syncwarp();
      } else {
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < 16; ++x) sum += w[x];
        if (on_left) far_left += sum;
        else far_right += sum;
      }
    }
    if (grad && ok) {  // (heads without blocks too: their partial sums are 0)
      flush(hh);
      for (int x = hh + 1; x < a.share; ++x) flush(x);
    }
    bool fin = true;
    if (n > 0) fin = warp_wait(bar_fin, 0);
    ptx::tc_fence_after();
#pragma unroll
    for (int part = 0; part < 2; ++part) {  // dK (scaled), then dV
      float v0[32];
      // tcgen05.ld is warp-collective: every lane loads (DP = 64: the last two column
      // groups' are not used)
      if (n > 0) ptx::tmem_ld32((part == 0 ? t_dk : t_dv) + lane_off + (c * 32 < DP ? c * 32 : 0), v0);
      const Strides& sd = part == 0 ? a.sdk : a.sdv;
      const float sc = part == 0 ? a.scale : 1.f;
      const bool store = ok && fin && kj < a.Sk && c * 32 < DP;
#pragma unroll
      for (int x = 0; x < 32; ++x)  // nothing of what stands behind the sequence's keys
        if (!valid_k || n == 0) v0[x] = 0.f;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(part == 0 ? a.dk : a.dv) + bb * sd.b + kj * sd.s + g * sd.h + c * 32;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (store && c * 32 + 8 * x < a.D)
          *reinterpret_cast<uint4*>(out + 8 * x) =
              make_uint4(pack2(v0[8 * x] * sc, v0[8 * x + 1] * sc), pack2(v0[8 * x + 2] * sc, v0[8 * x + 3] * sc),
                         pack2(v0[8 * x + 4] * sc, v0[8 * x + 5] * sc), pack2(v0[8 * x + 6] * sc, v0[8 * x + 7] * sc));
      __syncwarp();  // the next tcgen05.ld is warp-collective
    }
    if (!fin) {
      ok = false;
      if (lane == 0) wait_failed(212);
    }
  }
  if (!ok) atomicCAS(&g_xattn_bwd_error, 0, 5);
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int DP, bool BIAS>
cudaError_t launch(const Args& a, cudaStream_t st) {
  CUtensorMap tq128, tdo128, tq64, tdo64, tk, tv;
  OASES_TRY(map4d(&tq128, a.q, a.sq, a.D, a.Sq, a.H, a.B, 128));
  OASES_TRY(map4d(&tdo128, a.d_o, a.sdo, a.D, a.Sq, a.H, a.B, 128));
  OASES_TRY(map4d(&tq64, a.q, a.sq, a.D, a.Sq, a.H, a.B, 64));
  OASES_TRY(map4d(&tdo64, a.d_o, a.sdo, a.D, a.Sq, a.H, a.B, 64));
  OASES_TRY(map4d(&tk, a.k, a.sk, a.D, a.Sk, a.G, a.B, 128));
  OASES_TRY(map4d(&tv, a.v, a.sv, a.D, a.Sk, a.G, a.B, 128));
  using Dq = DqSmem<DP>;
  using Kv = KvSmem<DP, BIAS>;
  static DeviceOnce attr;
  OASES_TRY(attr.run([] {
    const cudaError_t e = cudaFuncSetAttribute(xattn_dq_kernel<DP, BIAS>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, Dq::BYTES);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(xattn_dkv_kernel<DP, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Kv::BYTES);
  }));
  const int64_t rows = (int64_t)a.B * a.Sq * a.H;
  if ((rows + 15) / 16 > INT32_MAX) return cudaErrorInvalidConfiguration;
  OASES_TRY(launch_pdl(xattn_delta_kernel, dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, st, a, rows));
  Plan p;
  p.a = a;
  p.scale_log2 = LOG2E * a.scale;
  p.tiles = (a.Sq + 127) / 128;
  const int64_t items = (int64_t)p.tiles * a.B * a.H;
  const int64_t ctas = (int64_t)((a.Sk + 127) / 128) * a.B * a.G;
  if (items > INT32_MAX / 2 || ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  p.items = (int)items;
  Plan pk = p;
  pk.tiles = (a.Sk + 127) / 128;
  OASES_TRY(launch_pdl(xattn_dq_kernel<DP, BIAS>, dim3((unsigned)std::min<int64_t>(items, sm_count())), dim3(NT),
                       Dq::BYTES, st, tq128, tdo128, tk, tv, p));
  return launch_pdl(xattn_dkv_kernel<DP, BIAS>, dim3((unsigned)ctas), dim3(NT), Kv::BYTES, st, tk, tv, tq64,
                    tdo64, pk);
}

}  // namespace

cudaError_t xattn_bwd_tc(const Args& a, cudaStream_t st) {
  if (a.D <= 64) return a.bias.buckets ? launch<64, true>(a, st) : launch<64, false>(a, st);
  return a.bias.buckets ? launch<128, true>(a, st) : launch<128, false>(a, st);
}

int xattn_bwd_read_and_clear_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_xattn_bwd_error, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_xattn_bwd_error, &z, sizeof(int));
  return v;
}

}  // namespace oases
