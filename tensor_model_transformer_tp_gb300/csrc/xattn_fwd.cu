// Attention over keys of another length, forward, on the 5th-generation tensor cores
// (bf16 in, fp32 softmax).
//
// A persistent kernel, one CTA per SM, 384 threads.  A work item is 256 queries of one
// (sequence, head), two tiles of 128 that share every block of 128 keys, over one share
// of the keys (all of them unless there are few items: then the shares' results are
// joined by join_splits()).  Items are numbered heaviest first and dealt in snake order.
//   warp 0      TMA loads in the order the MMAs consume them: Q_0, then K_j and V_j into
//               rings that run on across items, Q_1 after the first block;
//   warp 1      TMEM allocation (512 columns); one thread issues the MMAs;
//   warps 4..7  softmax of tile 0, warps 8..11 of tile 1: a thread owns one query's row.
// TMEM: S_t (then P_t) in columns 128 t .. + 127, O_t in 256 + 128 t ..
// Per tile t and block j:
//   S_t = Q_t K_j^T        A and B from shared memory
//   P_t = 2^(s - m)        written back over S_t's first 64 columns as packed bf16
//   O_t += P_t V_j         A = P_t from tensor memory
// issued PV_0(j), S_0(j+1), PV_1(j), S_1(j+1), so that one tile's softmax runs under the
// other's MMAs.  MMAs of one thread run in order: S_t(j) complete means PV_t(j-1) is, so
// a row of O may be rescaled in place before P_t(j) is published.  The reference maximum
// is raised only where the running one exceeds it by 2^8, so P <= 256 and O is rescaled
// rarely.  P is rounded to bf16, the operand type, its sum l is not.
//
// The position bias depends on j - p alone.  A warp's 32 rows x 128 keys that all lie
// R or more apart on one side have one value, which goes into the exponent's shift; only
// the blocks around the diagonal add a value per score, from the head's table by
// distance (a lane's 128 values are consecutive, neighbouring lanes' shifted by one).
//
// Keys that no query of the sequence sees (at and behind kv_lens; causal, behind the last
// query) count for nothing whatever they hold: their scores are replaced, not added to, and
// their rows of V are cleared in shared memory before the product (0 times an infinity would
// be NaN).
#include <math.h>

#include <algorithm>

#include "xattn_tc.cuh"

namespace oases {

__device__ int g_xattn_fwd_error;

namespace {
using namespace xattn;

// Registers move from the first warpgroup to the softmax warps: 128 x 120 + 256 x 192 =
// 384 x 168, what a block starts with.  (The thread that issues the MMAs is on every block's
// path: 72 registers make it spill, 226 against 206 us at 8 x 2048, 19 heads of 128.)
constexpr int NT = 384, REGS = 168, REGS_ISSUE = 120, REGS_SOFTMAX = 192;
static_assert(128 * REGS_ISSUE + 256 * REGS_SOFTMAX == NT * REGS, "registers of the warpgroups");
constexpr float RESCALE_LOG2 = 8.f;
constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(128, 128, false, false);

template <int DP>
struct Smem {
  static constexpr int TILE = tile_bytes<DP>();
  static constexpr int ST = DP == 128 ? 2 : 4;  // stages of K and of V
  static constexpr int Q = 0, K = 2 * TILE, V = K + ST * TILE, EPI = V + ST * TILE;
  static constexpr int ORDER = EPI + 8 * 4096;  // Order
  static constexpr int BAR = ORDER + ((int)sizeof(Order) + 15) / 16 * 16;
  // q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], drain, then the rings'
  static constexpr int NBAR = 13 + 4 * ST;
  static constexpr int USED = BAR + 8 * NBAR + 16;
  // the tiles need 1024-byte alignment: the window starts so aligned on this GPU, and
  // the kernel checks that what rounding takes is there
  static constexpr int BYTES = USED + 1024 <= 232448 ? USED + 1024 : 232448;
  static_assert(USED <= 232448, "more than 227 KB of shared memory");
};

struct Item {
  int h, b, q0, p0, len;  // head, sequence, first query, its position, the sequence's keys
  int split, j0;          // share of the keys, its first block
  int n0, n1;             // blocks of each tile (0 too where it lies past the queries)
};

struct Plan {
  Args a;
  int pairs, items;
  float scale_log2;
};

__device__ __forceinline__ Item item_at(const Plan& p, const Order* o, int i) {
  const Args& a = p.a;
  Item it;
  it.split = i % a.splits;
  i /= a.splits;
  it.h = i % a.H;
  int pair;
  query_item(a, o, i / a.H, p.pairs, &pair, &it.b);
  it.q0 = pair * 256;
  it.len = a.len(it.b);
  it.p0 = a.start(it.b) + it.q0;
  auto blocks = [&](int first, int t) {  // key blocks of tile t, whose first query is `first`
    if (first >= a.Sq) return 0;
    const int last = min(first + 128, a.Sq) - it.q0;  // queries of the item up to the tile's end
    const int vis = a.causal ? min(it.len, max(0, it.p0 + last)) : it.len;
    return (vis + 127) / 128;
  };
  const int n0 = blocks(it.q0, 0), n1 = blocks(it.q0 + 128, 1), n = max(n0, n1);
  const int share = (n + a.splits - 1) / a.splits;
  it.j0 = min(n, it.split * share);
  const int end = min(n, it.j0 + share);
  it.n0 = max(0, min(n0, end) - it.j0);
  it.n1 = max(0, min(n1, end) - it.j0);
  return it;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void wait_failed(int site) { atomicCAS(&g_xattn_fwd_error, 0, site); }

template <int DP, bool BIAS>
__global__ void __launch_bounds__(NT, 1)
xattn_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const __grid_constant__ Plan p) {
  using L = Smem<DP>;
  constexpr int TILE = L::TILE, ST = L::ST;
  constexpr uint32_t IDESC_PV = ptx::idesc_bf16_f32(128, DP, false, true);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  if (base - raw + L::USED > (uint32_t)L::BYTES) {  // (uniform: every thread leaves)
    if (threadIdx.x == 0) wait_failed(6);
    return;
  }
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::BAR;
  auto q_full = [&](int t) { return bars + 8u * t; };
  auto q_empty = [&](int t) { return bars + 8u * (2 + t); };
  auto s_full = [&](int t) { return bars + 8u * (4 + t); };
  auto p_full = [&](int t, int half) { return bars + 8u * (6 + 2 * half + t); };  // P of 64 keys
  auto o_full = [&](int t) { return bars + 8u * (10 + t); };
  const uint32_t bar_drain = bars + 8u * 12;
  auto k_full = [&](uint32_t s) { return bars + 8u * (13 + s); };
  auto k_empty = [&](uint32_t s) { return bars + 8u * (13 + ST + s); };
  auto v_full = [&](uint32_t s) { return bars + 8u * (13 + 2 * ST + s); };
  auto v_empty = [&](uint32_t s) { return bars + 8u * (13 + 3 * ST + s); };
  const uint32_t tslot = bars + 8u * L::NBAR;
  const Args& a = p.a;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int cta = blockIdx.x, G = gridDim.x;

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(q_full(t), 1);
      ptx::mbar_init(q_empty(t), 1);
      ptx::mbar_init(s_full(t), 1);
      for (int half = 0; half < 2; ++half) ptx::mbar_init(p_full(t, half), 4);  // one arrival per softmax warp of the tile
      ptx::mbar_init(o_full(t), 1);
    }
    ptx::mbar_init(bar_drain, 1);
    for (int s = 0; s < 4 * ST; ++s) ptx::mbar_init(k_full(s), 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tq);
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
  pdl_wait();
  pdl_trigger();
  Order* const order = reinterpret_cast<Order*>(gbase + L::ORDER);
  if (ragged(a)) order_sequences(a, reinterpret_cast<int*>(gbase), order, order->tiles);
  bool ok = true;

  if (warp < 4) {
    fewer_registers<REGS_ISSUE>();
    if (warp == 0) {
      if (ptx::elect_one()) {
        uint32_t ke = 0, qn[2] = {0u, 0u};  // ring entries loaded (entry e in stage e % ST), Q loads
        auto load_q = [&](const Item& it, int t) {
          if (qn[t] > 0 && !ptx::mbar_wait(q_empty(t), (qn[t] - 1) & 1)) return false;
          ptx::mbar_arrive_expect_tx(q_full(t), TILE);
          load_tile<DP, 128>(base + L::Q + t * TILE, &tq, q_full(t), it.q0 + 128 * t, it.h, it.b);
          ++qn[t];
          return true;
        };
        uint32_t ve = 0;
        for (int k = 0; ok; ++k) {
          const int i = persistent_item(k, cta, G);
          if (i >= p.items) break;
          const Item it = item_at(p, order, i);
          const int nmax = max(it.n0, it.n1), g = it.h / a.share;
          if (it.n0 > 0) ok = load_q(it, 0);
          for (int j = 0; j < nmax && ok; ++j) {
            const int r = (it.j0 + j) * 128;
            const uint32_t s = ke % ST, u = ke / ST;
            if (u > 0 && !ptx::mbar_wait(k_empty(s), (u - 1) & 1)) {
              ok = false;
              break;
            }
            ptx::mbar_arrive_expect_tx(k_full(s), TILE);
            load_tile<DP, 128>(base + L::K + s * TILE, &tk, k_full(s), r, g, it.b);
            ++ke;
            if (u > 0 && !ptx::mbar_wait(v_empty(s), (u - 1) & 1)) {
              ok = false;
              break;
            }
            ptx::mbar_arrive_expect_tx(v_full(s), TILE);
            load_tile<DP, 128>(base + L::V + s * TILE, &tv, v_full(s), r, g, it.b);
            ++ve;
            if (j == 0 && it.n1 > 0) ok = load_q(it, 1);
          }
        }
        if (!ok) wait_failed(11);
        // every load issued has landed before the CTA may exit: the last entry of each
        // stage, the last Q of each tile
        bool dr = true;
        for (uint32_t s = 0; s < ST; ++s) {
          if (ke > s) dr = ptx::mbar_wait(k_full(s), ((ke - 1 - s) / ST) & 1) && dr;
          if (ve > s) dr = ptx::mbar_wait(v_full(s), ((ve - 1 - s) / ST) & 1) && dr;
        }
        for (int t = 0; t < 2; ++t)
          if (qn[t] > 0) dr = ptx::mbar_wait(q_full(t), (qn[t] - 1) & 1) && dr;
        if (!dr) wait_failed(13);
      }
    } else if (warp == 1) {
      if (ptx::elect_one()) {
        uint32_t qc0 = 0u, qc1 = 0u, pc0 = 0u, pc1 = 0u;  // Q loads and hand-overs of P consumed
        // A ring entry is read by tile 0 first (it starts every item before tile 1 does
        // and its blocks are no more), so tile 1's MMA releases it, or tile 0's where tile
        // 1 does not read it (last).
        auto issue_s = [&](int t, uint32_t e, bool last) {  // S_t = Q_t K_e^T
          const uint32_t s = e % ST;
          if (!ptx::mbar_wait(k_full(s), (e / ST) & 1)) return false;
          ptx::tc_fence_after();
          const uint32_t qt = base + L::Q + t * TILE, kt = base + L::K + s * TILE;
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk)
            ptx::mma_bf16(tmem + 128u * t, kmajor_desc(qt, kk), kmajor_desc(kt, kk), IDESC_S, kk > 0);
          ptx::mma_commit(s_full(t));
          if (last) ptx::mma_commit(k_empty(s));
          return true;
        };
        auto issue_pv = [&](int t, uint32_t e, int j, bool last) {  // O_t += P_t V_e
          uint32_t& pc = t ? pc1 : pc0;
          const uint32_t s = e % ST;
          if (!ptx::mbar_wait(v_full(s), (e / ST) & 1)) return false;
          const uint32_t vt = base + L::V + s * TILE;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!ptx::mbar_wait(p_full(t, half), pc & 1)) return false;
            ptx::tc_fence_after();
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
              ptx::mma_bf16_ts(tmem + 256u + 128u * t, tmem + 128u * t + 8u * kk, mnmajor_desc(vt, kk), IDESC_PV,
                               (j > 0 || kk > 0) ? 1u : 0u);
          }
          ++pc;
          if (last) ptx::mma_commit(v_empty(s));
          return true;
        };
        // S_t(0) of an item whose block 0 is at ring entry e0 (nothing for an empty tile)
        auto start_tile = [&](const Item& it, int t, uint32_t e0) {
          const int n = t ? it.n1 : it.n0;
          if (n == 0) return true;
          uint32_t& qc = t ? qc1 : qc0;
          if (!ptx::mbar_wait(q_full(t), qc & 1)) return false;
          ++qc;
          if (!issue_s(t, e0, t == 1 || it.n1 == 0)) return false;
          if (n == 1) ptx::mma_commit(q_empty(t));  // the tile's last S of the item
          return true;
        };
        int k = 0, i = persistent_item(0, cta, G);
        uint32_t kb = 0;  // ring entry of the item's block 0
        Item it{};
        if (i < p.items) {
          it = item_at(p, order, i);
          ok = start_tile(it, 0, 0u) && start_tile(it, 1, 0u);
        }
        while (ok && i < p.items) {
          const int nmax = max(it.n0, it.n1);
          const int inext = persistent_item(k + 1, cta, G);
          const bool has_next = inext < p.items;
          Item nx{};
          if (has_next) nx = item_at(p, order, inext);
          const uint32_t kb_next = kb + (uint32_t)nmax;
          bool started0 = !has_next, started1 = !has_next;  // the next item's tiles
          for (int j = 0; j < nmax && ok; ++j) {
            bool done0 = false, done1 = false;  // the tile's last PV of the item issued in this round
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int n = t ? it.n1 : it.n0;
              if (!ok || j >= n) continue;
              ok = issue_pv(t, kb + j, j, t == 1 || it.n1 <= j);
              if (!ok) break;
              if (j + 1 < n) {
                ok = issue_s(t, kb + j + 1, t == 1 || it.n1 <= j + 1);
                if (!ok) break;
                if (j + 2 == n) ptx::mma_commit(q_empty(t));  // the tile's last S of the item
              } else {
                ptx::mma_commit(o_full(t));  // the tile's last PV of the item
                if (t) done1 = true; else done0 = true;
              }
            }
            // a tile whose item ended in this round starts the next one, tile 0 first
            if (ok && !started0 && (done0 || done1)) {
              ok = start_tile(nx, 0, kb_next);
              started0 = true;
            }
            if (ok && !started1 && done1) {
              ok = start_tile(nx, 1, kb_next);
              started1 = true;
            }
          }
          if (ok && !started0) ok = start_tile(nx, 0, kb_next);
          if (ok && !started1) ok = start_tile(nx, 1, kb_next);
          kb = kb_next;
          it = nx;
          i = inext;
          ++k;
        }
        if (!ok) wait_failed(14);
        ptx::mma_commit(bar_drain);  // completes once every MMA issued above has
        if (!ptx::mbar_wait(bar_drain, 0)) {
          ok = false;
          wait_failed(18);
        }
      }
    }
  } else {
    more_registers<REGS_SOFTMAX>();
    const int t = (warp - 4) >> 2, qq = warp & 3;
    const int row = qq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qq * 32) << 16;
    const uint32_t t_s = tmem + 128u * t + lane_off, t_o = tmem + 256u + 128u * t + lane_off;
    uint32_t sc = 0u, oc = 0u, kb = 0u;  // S_t blocks, finished items of this tile, ring entries so far
    for (int k = 0; ok; ++k) {
      const int i = persistent_item(k, cta, G);
      if (i >= p.items) break;
      const Item it = item_at(p, order, i);
      const int nt = t ? it.n1 : it.n0;
      const int qi = it.q0 + 128 * t + row;         // the thread's query
      const int pi = it.p0 + 128 * t + row;         // and its position
      if (it.q0 + 128 * t >= a.Sq) {                // (uniform per tile) no queries here
        kb += (uint32_t)max(it.n0, it.n1);
        continue;
      }
      float left = 0.f, right = 0.f;
      if (BIAS) {
        left = *a.bias.at(it.h, -a.bias.R);
        right = *a.bias.at(it.h, a.bias.R);
      }
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < nt && ok; ++j, ++sc) {
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(s_full(t), sc & 1))) {
          ok = false;
          if (lane == 0) wait_failed(19);
          break;
        }
        ptx::tc_fence_after();
        float sv[128];
        ptx::tmem_ld128(t_s, sv);
        const int kbase = (it.j0 + j) * 128;
        const int w0 = it.p0 + 128 * t + qq * 32;   // position of the warp's first query
        float mul = p.scale_log2, add = 0.f;        // s = sv mul + add in log2 units
        if (BIAS) {
          const int lo = kbase - (w0 + 31), hi = kbase + 127 - w0;
          if (lo >= a.bias.R) {
            add = right;
          } else if (hi <= -a.bias.R) {
            add = left;
          } else {
            const float* bv = a.bias.at(it.h, kbase - w0) - lane;
#pragma unroll
            for (int c = 0; c < 128; ++c) sv[c] = fmaf(sv[c], p.scale_log2, __ldg(bv + c));
            mul = 1.f;
          }
        }
        // a block that every row of the warp sees whole needs no mask (warp-uniform)
        const bool full = kbase + 128 <= it.len && (!a.causal || kbase + 127 <= w0);
        if (!full) {
          const int nvis = (a.causal ? min(pi + 1, it.len) : it.len) - kbase;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= nvis) sv[c] = -INFINITY;
        }
        // row maximum in eight independent chains, two scores a step (mul is positive)
        float pm[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) pm[c] = fmaxf(sv[2 * c], sv[2 * c + 1]);
#pragma unroll
        for (int c = 16; c < 128; c += 2) pm[c / 2 % 8] = max3(pm[c / 2 % 8], sv[c], sv[c + 1]);
        const float mx =
            fmaf(max3(max3(pm[0], pm[1], pm[2]), max3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7])), mul, add);
        const float m_new = fmaxf(m_ref, mx);
        // O_t is rescaled by f (below) where the reference maximum is raised
        float f = 1.f;
        bool rescale = false;
        if (j == 0) {
          m_ref = m_new;
        } else {
          const bool need = m_new > m_ref + RESCALE_LOG2;
          rescale = __any_sync(0xffffffffu, need);  // warp-uniform: tcgen05.ld/st are collective
          if (need) {
            f = exp2f(m_ref - m_new);
            l *= f;
            m_ref = m_new;
          }
        }
        if (rescale) {
#pragma unroll 1
          for (int c0 = 0; c0 < DP; c0 += 32) {
            float v[32];
            ptx::tmem_ld32(t_o + c0, v);
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) w[c] = __float_as_uint(v[c] * f);
            ptx::tmem_st32_nowait(t_o + c0, w);
          }
        }
        // the keys behind the sequence's, where the tensor goes on: rows of V cleared by
        // the first tile that reads them (tile 1's product follows tile 0's)
        if (kbase + 128 > it.len && it.len < a.Sk && (t == 0 || j >= it.n0)) {
          const uint32_t e = kb + j, s = e % ST;
          if (!__all_sync(0xffffffffu, ptx::mbar_wait(v_full(s), (e / ST) & 1))) {
            ok = false;
            if (lane == 0) wait_failed(21);
            break;
          }
          if (kbase + row >= it.len) {
            uint8_t* vr = gbase + L::V + s * TILE + row * 128;
#pragma unroll
            for (int c = 0; c < DP / 64; ++c)
#pragma unroll
              for (int x = 0; x < 8; ++x)
                *reinterpret_cast<uint4*>(vr + c * BOX + 16 * x) = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_async_smem();
          __syncwarp();
        }
        // P = 2^(s - m_ref): scale and shift in one fp32x2 FMA per pair, the row sum in
        // four fp32x2 accumulators; handed over 64 keys at a time
        // (no visible key so far: every weight 0, but a NaN stays one)
        const uint64_t sc2 = f2_splat(mul), nm2 = f2_splat(m_ref == -INFINITY ? -INFINITY : add - m_ref);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int at = 64 * half + 2 * c;
            const uint64_t x = f2_fma(f2_pack(sv[at], sv[at + 1]), sc2, nm2);
            const float p0 = fast_exp2(f2_lo(x)), p1 = fast_exp2(f2_hi(x));
            acc[c % 4] = f2_add(acc[c % 4], f2_pack(p0, p1));
            w[c] = pack2(p0, p1);
          }
          ptx::tmem_st32_nowait(t_s + 32u * half, w);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(p_full(t, half));
        }
        const uint64_t acc2 = f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3]));
        const float rs = f2_lo(acc2) + f2_hi(acc2);
        l += rs;
      }
      kb += (uint32_t)max(it.n0, it.n1);
      if (!ok) break;
      float v[DP];
      bool fin = true;
      if (nt > 0) {
        // the tile's last PV of the item is complete (or the MMA thread gave up)
        fin = __all_sync(0xffffffffu, ptx::mbar_wait(o_full(t), oc & 1));
        ++oc;
        if (!fin && lane == 0) wait_failed(20);
        ptx::tc_fence_after();
#pragma unroll
        for (int c0 = 0; c0 < DP; c0 += 32)
          ptx::tmem_ld32(t_o + c0, *reinterpret_cast<float(*)[32]>(v + c0));
      } else {
#pragma unroll
        for (int c = 0; c < DP; ++c) v[c] = 0.f;
      }
      if (!fin) {
        ok = false;
        break;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse = (m_ref + log2f(l)) * LN2;
      if (a.splits > 1) {
        if (qi < a.Sq) {
          a.part_lse[(int64_t)it.split * a.B * a.H * a.Sq + a.stat(it.b, it.h, qi)] = lse;
          float* out = a.part_o + ((((int64_t)it.split * a.B + it.b) * a.Sq + qi) * a.H + it.h) * a.D;
#pragma unroll
          for (int c = 0; c < DP; c += 4)
            if (c < a.D)
              *reinterpret_cast<float4*>(out + c) =
                  make_float4(v[c] * inv, v[c + 1] * inv, v[c + 2] * inv, v[c + 3] * inv);
        }
        continue;
      }
      // O rows through this warp's 4 KB of shared memory, 64 columns at a time: lane r
      // writes its row's 128 bytes as eight 16-byte chunks (chunk c at c ^ (r & 7), so
      // that eight lanes cover all banks), then a store writes 4 rows x 128 bytes
      uint8_t* stg = gbase + L::EPI + (warp - 4) * 4096;
      const int rw0 = it.q0 + 128 * t + qq * 32;  // the warp's first query
      __nv_bfloat16* ow = static_cast<__nv_bfloat16*>(a.o) + it.b * a.so.b + it.h * a.so.h + rw0 * a.so.s;
#pragma unroll
      for (int c0 = 0; c0 < DP; c0 += 64) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float* x = v + c0 + 8 * c;
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(pack2(x[0] * inv, x[1] * inv), pack2(x[2] * inv, x[3] * inv),
                         pack2(x[4] * inv, x[5] * inv), pack2(x[6] * inv, x[7] * inv));
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = 4 * u + (lane >> 3), c = lane & 7;
          const uint4 w = *reinterpret_cast<const uint4*>(stg + r * 128 + ((c ^ (r & 7)) << 4));
          if (rw0 + r < a.Sq && c0 + 8 * c < a.D)
            *reinterpret_cast<uint4*>(ow + (int64_t)r * a.so.s + c0 + 8 * c) = w;
        }
        __syncwarp();
      }
      if (qi < a.Sq) a.lse[a.stat(it.b, it.h, qi)] = lse;
    }
  }
  if (!ok) atomicCAS(&g_xattn_fwd_error, 0, 1);
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int DP, bool BIAS>
cudaError_t launch(const Args& a, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  OASES_TRY(map4d(&tq, a.q, a.sq, a.D, a.Sq, a.H, a.B, 128));
  OASES_TRY(map4d(&tk, a.k, a.sk, a.D, a.Sk, a.G, a.B, 128));
  OASES_TRY(map4d(&tv, a.v, a.sv, a.D, a.Sk, a.G, a.B, 128));
  static DeviceOnce attr;
  OASES_TRY(attr.run([] {
    cudaFuncAttributes at;
    OASES_TRY(cudaFuncGetAttributes(&at, xattn_fwd_kernel<DP, BIAS>));
    if (at.numRegs != REGS) return cudaErrorInvalidKernelImage;  // (the warpgroups' shares would not add up)
    return cudaFuncSetAttribute(xattn_fwd_kernel<DP, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<DP>::BYTES);
  }));
  Plan p;
  p.a = a;
  p.pairs = (a.Sq + 255) / 256;
  const int64_t items = (int64_t)p.pairs * a.B * a.H * a.splits;
  if (items > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
  p.items = (int)items;
  p.scale_log2 = LOG2E * a.scale;
  return launch_pdl(xattn_fwd_kernel<DP, BIAS>, dim3((unsigned)std::min<int64_t>(items, sm_count())), dim3(NT),
                    Smem<DP>::BYTES, st, tq, tk, tv, p);
}

}  // namespace

cudaError_t xattn_fwd_tc(const Args& a, cudaStream_t st) {
  if (a.D <= 64) return a.bias.buckets ? launch<64, true>(a, st) : launch<64, false>(a, st);
  return a.bias.buckets ? launch<128, true>(a, st) : launch<128, false>(a, st);
}

int xattn_fwd_read_and_clear_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_xattn_fwd_error, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_xattn_fwd_error, &z, sizeof(int));
  return v;
}

}  // namespace oases
