// Attention over keys of another length, backward, on the 5th-generation tensor cores
// (bf16 in, fp32 between the products).
//
//   P = e^(s - lse), delta = rowsum(dO * O), dP = dO V^T, dS = P (dP - delta),
//   dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO, and dS summed by bucket.
// Two kernels own disjoint outputs, so there are no atomics:
//   dq kernel   items of 128 queries, looped over blocks of 128 keys
//   dkv kernel  items of 128 keys of a key head, looped over its query heads and blocks
//               of 64 (DP = 128) or 128 queries (DP = 64)
// and dS is formed twice (9 products of the definition's 7).  Both are persistent
// pipelines of one TMA warp, two MMA-issuing threads (one for S and dP, one for the
// accumulations: a thread that issued both would wait at one's barrier while the other's
// operands are ready) and 16 element-wise warps, each on 32 rows x 32 columns of a block.
// P and dS, rounded to bf16, the operand type, are written packed over S (or dP) in tensor
// memory and read from there as the accumulations' A operand; the bias's gradient sums dS
// before the rounding.
//
// Items beyond whole rounds of the GPU's SMs are cut into pieces of their blocks, one for
// each SM; a piece writes fp32 sums of its own, which the join kernels add in order.
//
// delta.  From the rounded o it is off by up to 2^-8 of |dO||o|, which shows in rows of few
// keys (o as large as v) and in the bias's gradient (a row's error, summed over its keys).
// Its definition is sum P dP, and what dS sums to over a row is the difference: the dq
// kernel takes it from the first block of keys for the rows that see no other (an item of
// queries that begins behind a cache may hold such rows beside others), and corrects delta
// for the dkv kernel there and wherever there is a bias.
//
// The bias's gradient (dkv kernel).  A warp's 32 x 32 scores that lie R or more from the
// diagonal on one side belong to one bucket: every thread adds its own.  Nearer ones are
// summed along their 63 diagonals, by passing running sums from lane to lane as the
// column advances (lane r adds element (r, c) at step c, so a sum that moves one lane a
// step stays on its diagonal), and each bucket's run of diagonals is added to the warp's
// own buckets in shared memory: a fixed order throughout.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "xattn_tc.cuh"

namespace oases {

__device__ int g_xattn_bwd_error;

namespace {
using namespace xattn;

constexpr uint64_t WAIT = 1ull << 29;  // cycles before a wait gives up (~0.25 s)
// Warps 0..3 load and issue, 4..19 work element by element.  Registers move from the first
// warpgroup to the others: 128 x 64 + 512 x 104 = 640 x 96, what a block starts with.
constexpr int NT = 640, ACC_WARP = 2, EW = 16, EW0 = 4;
constexpr int REGS = 96, REGS_ISSUE = 64, REGS_EW = 104;
static_assert(128 * REGS_ISSUE + 32 * EW * REGS_EW == NT * REGS, "registers of the warpgroups");
constexpr int BOX64 = 64 * 64 * 2;  // one TMA box of 64 rows

__device__ __forceinline__ void wait_failed(int site) { atomicCAS(&g_xattn_bwd_error, 0, site); }
__device__ __forceinline__ bool wait1(uint32_t bar, uint32_t parity) { return ptx::mbar_wait(bar, parity, WAIT); }
// Warp-uniform bounded wait (every lane waits; the warp agrees on the outcome).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait1(bar, parity));
}
// A row's -lse in base 2, so that its weights are 2^(s - lse); a query without keys: every
// weight 0.
__device__ __forceinline__ float minus_lse2(float lse) { return beyond_weights(lse) ? -INFINITY : -lse * LOG2E; }

struct Plan {
  Args a;
  int tiles;          // dq: 128-query tiles; dkv: 128-key tiles
  Pieces cut;
  float scale_log2;
  float* part;        // the pieces' sums: dq [piece][128][D]; dkv [piece][dk, dv][128][D]
};

// Work k of CTA c of G: an item, and which of its pieces (-1: all of it).
struct Work {
  int item, piece;
  int part;  // the piece's place in p.part
};
__device__ __forceinline__ bool work_at(const Plan& p, int k, int c, int G, Work* w) {
  const int i = persistent_item(k, c, G);  // (whole rounds: cut.whole is a multiple of G, or 0)
  if (i < p.cut.whole) {
    *w = {i, -1, 0};
    return true;
  }
  const int r = k * G + c - p.cut.whole;
  if (r >= p.cut.rest * p.cut.pieces) return false;
  *w = {p.cut.whole + r / p.cut.pieces, p.cut.pieces > 1 ? r % p.cut.pieces : -1, r};
  return true;
}
// Blocks [first, end) of a piece, of the item's n.
__device__ __forceinline__ void cut_blocks(const Plan& p, int piece, int n, int* first, int* end) {
  *first = piece < 0 ? 0 : (int)((int64_t)n * piece / p.cut.pieces);
  *end = piece < 0 ? n : (int)((int64_t)n * (piece + 1) / p.cut.pieces);
}

// Every row's -lse (base 2) and -delta, [batch][heads][q_pitch] each, so that a block's are
// one copy: 16 lanes a row, 16 bytes each, four queries of a head at a time.  Rows behind
// the queries have no weights.
__global__ void __launch_bounds__(256)
xattn_stats_kernel(const __grid_constant__ Args a, int64_t fours) {
  pdl_wait();
  pdl_trigger();
  const int64_t r = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 16;  // (batch, four queries, head)
  const int lane = threadIdx.x % 16, c = lane * 8;
  const int64_t bq = r / a.H;
  const int h = (int)(r - bq * a.H), per = a.q_pitch / 4;
  const int64_t b = bq / per;
  const int q0 = (int)(bq - b * per) * 4;
  uint4 x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = y[i] = make_uint4(0, 0, 0, 0);
    if (r < fours && c < a.D && q0 + i < a.Sq) {
      x[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.o) + b * a.so.b + (q0 + i) * a.so.s +
                                             h * a.so.h + c);
      y[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.d_o) + b * a.sdo.b + (q0 + i) * a.sdo.s +
                                             h * a.sdo.h + c);
    }
  }
  float d[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      d[i] = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(w[e] << 16), d[i]);
      d[i] = fmaf(__uint_as_float(u[e] & 0xffff0000u), __uint_as_float(w[e] & 0xffff0000u), d[i]);
    }
  }
#pragma unroll
  for (int o = 8; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] += __shfl_xor_sync(~0u, d[i], o);
  if (r >= fours || lane > 0) return;
  const int64_t at = (b * a.H + h) * a.q_pitch + q0;
  float l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) l[i] = q0 + i < a.Sq ? minus_lse2(a.lse[a.stat((int)b, h, q0 + i)]) : -INFINITY;
  *reinterpret_cast<float4*>(a.neg_lse2 + at) = make_float4(l[0], l[1], l[2], l[3]);
  *reinterpret_cast<float4*>(a.delta + at) = make_float4(-d[0], -d[1], -d[2], -d[3]);
}

// 128 rows x DP columns through a map of 64-row boxes (two of a column group lie one
// behind the other, as one of 128 rows would).
template <int DP>
__device__ __forceinline__ void load_two(uint32_t dst, const void* tmap, uint32_t bar, int row, int head, int batch) {
#pragma unroll
  for (int c = 0; c < DP / 64; ++c)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      tma_load_4d(dst + c * BOX + r * BOX64, tmap, bar, 64 * c, row + 64 * r, head, batch);
}

// 32 columns of a row from tensor memory, times `scale`: in bf16 to the row `out` (columns
// from D on left out), or in fp32 to a piece's row.
__device__ __forceinline__ void store_row(__nv_bfloat16* out, const float (&v)[32], int columns, float scale) {
#pragma unroll
  for (int x = 0; x < 32; x += 8)
    if (x < columns)
      *reinterpret_cast<uint4*>(out + x) = make_uint4(pack2(v[x] * scale, v[x + 1] * scale), pack2(v[x + 2] * scale, v[x + 3] * scale),
                                                      pack2(v[x + 4] * scale, v[x + 5] * scale), pack2(v[x + 6] * scale, v[x + 7] * scale));
}
__device__ __forceinline__ void store_part(float* out, const float (&v)[32], int columns) {
#pragma unroll
  for (int x = 0; x < 32; x += 4)
    if (x < columns) *reinterpret_cast<float4*>(out + x) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
}

// ---- dq ---------------------------------------------------------------------------------
// Warp 0 TMA (per item K and V of its first block, then Q and dO, then the rings of K and
// V, which run on across items), warp 1 TMEM and the S and dP MMAs, warp 2 the dQ MMAs,
// warps 4..19 element-wise (lanes 32 (w % 4) .. of a block, columns 32 (w / 4 - 1) ..).  TMEM: S of even blocks 0..127, of odd blocks 128..255, dP 256..383, dQ 384..
// An element-wise warp forms its weights from S while dP is made, releases dP as soon as
// its columns are loaded, and writes dS packed over the first 16 of its own 32 columns of
// S: the tensor cores go from S, dP of block j + 1 to dQ of block j.
template <int DP>
struct DqSmem {
  static constexpr int TILE = tile_bytes<DP>();
  static constexpr int KST = DP == 64 ? 4 : 3, VST = DP == 64 ? 4 : 2;
  static constexpr int Q = 0, DO = TILE, K = 2 * TILE, V = K + KST * TILE;
  static constexpr int RED = V + VST * TILE;  // [column group][128] fp32: partial sums of the rows
  static constexpr int ORDER = RED + 4 * 128 * 4;  // the sequences in order
  static constexpr int BAR = ORDER + MAX_ORDER;
  static constexpr int NBAR = 14 + 2 * KST + 2 * VST;
  static constexpr int USED = BAR + 8 * NBAR + 16;
  // the tiles need 1024-byte alignment: the window starts so aligned on this GPU, and
  // the kernel checks that what rounding takes is there
  static constexpr int BYTES = USED + 1024 <= 232448 ? USED + 1024 : 232448;
  static_assert(USED <= 232448, "more than 227 KB of shared memory");
};

struct DqItem {
  int h, b, q0, p0, len;   // head, sequence, first query and its position, keys
  int j0, n, whole;        // key blocks: the first, how many, and how many without the cut
  bool few;                // some query sees the first block's keys and no others
  float* part;             // a piece's sums: dQ [128][D], then the rows' sums of dS
};
// The bytes of a piece of dq are 4 dq_piece(D).
__host__ __device__ __forceinline__ int64_t dq_piece(int D) { return 128 * (D + 1); }
__device__ __forceinline__ DqItem dq_item(const Plan& p, const Order* o, const Work& w) {
  const Args& a = p.a;
  DqItem it;
  it.h = w.item % a.H;
  int tile;
  query_item(a, o, w.item / a.H, p.tiles, &tile, &it.b);
  it.q0 = tile * 128;
  it.len = a.len(it.b);
  it.p0 = a.start(it.b) + it.q0;
  const int rows = min(128, a.Sq - it.q0);
  const int vis = a.causal ? min(it.len, max(0, it.p0 + rows)) : it.len;
  int end;
  it.whole = (vis + 127) / 128;
  it.few = it.whole == 1 || (it.whole > 1 && a.causal && it.p0 < 128);
  cut_blocks(p, w.piece, it.whole, &it.j0, &end);
  it.n = end - it.j0;
  it.part = w.piece < 0 ? nullptr : p.part + w.part * dq_piece(a.D);
  return it;
}

template <int DP, bool BIAS>
__global__ void __launch_bounds__(NT, 1)
xattn_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                const __grid_constant__ Plan p) {
  using L = DqSmem<DP>;
  constexpr int TILE = L::TILE, KST = L::KST, VST = L::VST;
  constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t IDESC_DQ = ptx::idesc_bf16_f32(128, DP, false, true);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  if (base - raw + L::USED > (uint32_t)L::BYTES) {  // (uniform: every thread leaves)
    if (threadIdx.x == 0) wait_failed(4);
    return;
  }
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::BAR;
  const uint32_t qdo_full = bars, qdo_empty = bars + 8u, dp_full = bars + 16u, dp_empty = bars + 24u;
  const uint32_t bar_fin = bars + 32u, drain = bars + 40u;
  auto s_full = [&](uint32_t b) { return bars + 8u * (6 + b); };
  auto ds_full = [&](uint32_t b) { return bars + 8u * (8 + b); };    // dS written over S
  auto ds_empty = [&](uint32_t b) { return bars + 8u * (10 + b); };  // and read
  const uint32_t red_full = bars + 96u, red_empty = bars + 104u;
  auto k_full = [&](uint32_t s) { return bars + 8u * (14 + s); };
  auto k_empty = [&](uint32_t s) { return bars + 8u * (14 + KST + s); };
  auto v_full = [&](uint32_t s) { return bars + 8u * (14 + 2 * KST + s); };
  auto v_empty = [&](uint32_t s) { return bars + 8u * (14 + 2 * KST + VST + s); };
  const uint32_t tslot = bars + 8u * L::NBAR;
  const Args& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
  const int cta = blockIdx.x, G = gridDim.x;

  if (tid == 0) {
    ptx::mbar_init(qdo_full, 1);
    ptx::mbar_init(qdo_empty, 1);
    ptx::mbar_init(dp_full, 1);
    ptx::mbar_init(dp_empty, EW);
    ptx::mbar_init(bar_fin, 1);
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(red_full, EW);
    ptx::mbar_init(red_empty, EW);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(s_full(b), 1);
      ptx::mbar_init(ds_full(b), EW);
      ptx::mbar_init(ds_empty(b), 1);
    }
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
  auto t_s = [&](uint32_t b) { return tmem + 128u * b; };
  const uint32_t t_dp = tmem + 256, t_dq = tmem + 384;
  pdl_wait();
  pdl_trigger();
  // (the items here need no counts of tiles: those stay in the scratch)
  Order* const order = reinterpret_cast<Order*>(gbase + L::ORDER);
  if (ragged(a)) order_sequences(a, reinterpret_cast<int*>(gbase), order, reinterpret_cast<int*>(gbase) + MAX_ORDER);
  bool ok = true;
  Work wk;

  if (warp < EW0) {
    fewer_registers<REGS_ISSUE>();
    if (warp == 0) {
      if (ptx::elect_one()) {
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
        for (int k = 0; ok && work_at(p, k, cta, G, &wk); ++k) {
          const DqItem it = dq_item(p, order, wk);
          if (it.n == 0) continue;
          const int g = it.h / a.share;
          ok = load_kv(it.j0 * 128, g, it.b);
          // Q and dO are free once the previous item's last S and dP are done
          if (ok && nq > 0 && !wait1(qdo_empty, (nq - 1) & 1)) ok = false;
          if (!ok) break;
          ptx::mbar_arrive_expect_tx(qdo_full, 2 * TILE);
          load_two<DP>(base + L::Q, &tq, qdo_full, it.q0, it.h, it.b);
          load_two<DP>(base + L::DO, &tdo, qdo_full, it.q0, it.h, it.b);
          ++nq;
          for (int j = 1; j < it.n && ok; ++j) ok = load_kv((it.j0 + j) * 128, g, it.b);
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
      if (ptx::elect_one()) {
        uint32_t g = 0, nq = 0;  // blocks (= ring entries) and items with blocks so far
        for (int k = 0; ok && work_at(p, k, cta, G, &wk); ++k) {
          const DqItem it = dq_item(p, order, wk);
          if (it.n == 0) continue;
          if (!wait1(qdo_full, nq & 1)) {
            ok = false;
            wait_failed(103);
            break;
          }
          ++nq;
          for (int j = 0; j < it.n; ++j, ++g) {  // S = Q K_j^T, dP = dO V_j^T
            const uint32_t sk = g % KST, sv = g % VST, b = g & 1;
            // (dQ of the block before the last, whose dS lay in this buffer, is done)
            if (!wait1(k_full(sk), (g / KST) & 1) || (g >= 2 && !wait1(ds_empty(b), ((g / 2) & 1) ^ 1))) {
              ok = false;
              wait_failed(104);
              break;
            }
            ptx::tc_fence_after();
            const uint32_t kt = base + L::K + sk * TILE, vt = base + L::V + sv * TILE;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
              ptx::mma_bf16(t_s(b), kmajor_desc(base + L::Q, kk), kmajor_desc(kt, kk), IDESC_S, kk > 0);
            ptx::mma_commit(s_full(b));
            // (the element-wise warps have loaded the previous block's dP)
            if (!wait1(v_full(sv), (g / VST) & 1) || (g >= 1 && !wait1(dp_empty, (g - 1) & 1))) {
              ok = false;
              wait_failed(105);
              break;
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
              ptx::mma_bf16(t_dp, kmajor_desc(base + L::DO, kk), kmajor_desc(vt, kk), IDESC_S, kk > 0);
            ptx::mma_commit(dp_full);
            ptx::mma_commit(v_empty(sv));
            if (j + 1 == it.n) ptx::mma_commit(qdo_empty);  // the item's last read of Q and dO
          }
        }
        ptx::mma_commit(drain);  // completes once every MMA this thread issued has
        if (!wait1(drain, 0)) {
          ok = false;
          wait_failed(107);
        }
      }
    } else if (warp == ACC_WARP) {
      if (ptx::elect_one()) {
        uint32_t g = 0, nk = 0;  // blocks, items with blocks finished
        for (int k = 0; ok && work_at(p, k, cta, G, &wk); ++k) {
          const DqItem it = dq_item(p, order, wk);
          if (it.n == 0) continue;
          for (int j = 0; j < it.n; ++j, ++g) {  // dQ += dS_j K_j
            const uint32_t sk = g % KST, b = g & 1;
            if (!wait1(ds_full(b), (g / 2) & 1)) {
              ok = false;
              wait_failed(106);
              break;
            }
            ptx::tc_fence_after();
            const uint32_t kt = base + L::K + sk * TILE;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              ptx::mma_bf16_ts(t_dq, t_s(b) + 32u * (kk >> 1) + 8u * (kk & 1), mnmajor_desc(kt, kk), IDESC_DQ,
                               (j > 0 || kk > 0) ? 1u : 0u);
            // S_j, which also read K_j, completed before dS_j could be handed over, so K_j is
            // free once these MMAs are
            ptx::mma_commit(ds_empty(b));
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
    }
  } else {
    more_registers<REGS_EW>();
    const int qq = warp & 3, sub = (warp - EW0) >> 2;  // lane quarter; columns 32 sub .. + 31
    const int row = qq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qq * 32) << 16;
    uint32_t g = 0, nf = 0;
    // this row's -lse (base 2) and -delta of an item, read one item ahead
    auto stats = [&](int k, float& nl, float& nd) {
      nl = -INFINITY;
      nd = 0.f;
      Work w;
      if (!work_at(p, k, cta, G, &w)) return;
      const DqItem it = dq_item(p, order, w);
      const int64_t at = ((int64_t)it.b * a.H + it.h) * a.q_pitch + it.q0 + row;
      nl = a.neg_lse2[at];
      nd = a.delta[at];
    };
    // a row's sum of the four column groups' x, by all 16 warps
    uint32_t nred = 0;
    const uint32_t red = base + L::RED + row * 4;
    auto row_sum = [&](float x, float& sum) {
      if (nred > 0 && !warp_wait(red_empty, (nred - 1) & 1)) return false;
      ptx::sts(red + sub * 512, x);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(red_full);
      if (!warp_wait(red_full, nred & 1)) return false;
      sum = (ptx::lds(red) + ptx::lds(red + 512)) + (ptx::lds(red + 1024) + ptx::lds(red + 1536));
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(red_empty);
      ++nred;
      return true;
    };
    float nl_next, nd_next;
    stats(0, nl_next, nd_next);
    for (int k = 0; ok && work_at(p, k, cta, G, &wk); ++k) {
      const DqItem it = dq_item(p, order, wk);
      const int qi = it.q0 + row;
      const bool valid_q = qi < a.Sq;
      const float nl = nl_next;
      float nd = nd_next;
      float off = 0.f;  // the row's sum of dS: how far delta is from sum P dP
      stats(k + 1, nl_next, nd_next);
      const int w0 = it.p0 + qq * 32;  // position of the warp's first query
      // the row's keys (none past the queries), and whether they all stand in the first block
      const int seen = valid_q ? (a.causal ? min(w0 + lane + 1, it.len) : it.len) : 0;
      const bool few_row = it.few && seen <= 128;
      float left = 0.f, right = 0.f;
      if (BIAS) {
        left = *a.bias.at(it.h, -a.bias.R);
        right = *a.bias.at(it.h, a.bias.R);
      }
      for (int j = 0; j < it.n; ++j, ++g) {
        const uint32_t b = g & 1, own = t_s(b) + lane_off + sub * 32;
        if (!warp_wait(s_full(b), (g / 2) & 1)) {
          ok = false;
          if (lane == 0) wait_failed(108);
          break;
        }
        ptx::tc_fence_after();
        float v[32];
        ptx::tmem_ld32(own, v);
        const int kb = (it.j0 + j) * 128 + sub * 32;
        // 32 x 32 scores wholly visible need no mask (warp-uniform)
        const bool full = it.q0 + qq * 32 + 32 <= a.Sq && kb + 32 <= it.len && (!a.causal || kb + 31 <= w0);
        const bool on_right = BIAS && kb - (w0 + 31) >= a.bias.R;
        const bool on_left = BIAS && !on_right && kb + 31 - w0 <= -a.bias.R;
        const float shift = (on_right ? right : on_left ? left : 0.f) + nl;
        float mul = p.scale_log2;
        if (BIAS && !on_left && !on_right) {
          const float* bv = a.bias.at(it.h, kb - w0) - lane;
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = fmaf(v[c], p.scale_log2, __ldg(bv + c));
          mul = 1.f;
        }
        const uint64_t sc = f2_splat(mul), sh = f2_splat(shift);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const uint64_t x = f2_fma(f2_pack(v[c], v[c + 1]), sc, sh);
          v[c] = fast_exp2(f2_lo(x));
          v[c + 1] = fast_exp2(f2_hi(x));
        }
        if (!warp_wait(dp_full, g & 1)) {
          ok = false;
          if (lane == 0) wait_failed(109);
          break;
        }
        ptx::tc_fence_after();
        float w[32];
        ptx::tmem_ld32(t_dp + lane_off + sub * 32, w);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(dp_empty);  // dP's buffer may be overwritten
        uint32_t pk[16];  // dS as packed bf16 pairs (keys 2i, 2i+1 of these 32)
        // keys kb + c with c >= nvis are past the diagonal or the sequence's keys (all of
        // them for a row past the queries); what dP holds there may be anything
        int nvis = seen - kb;
        if (it.few && it.j0 + j == 0) {
          float x = 0.f, sum = 0.f;
#pragma unroll
          for (int c = 0; c < 32; ++c) x += c < nvis ? v[c] * w[c] : 0.f;
          if (!row_sum(x, sum)) {
            ok = false;
            if (lane == 0) wait_failed(113);
            break;
          }
          if (few_row) {
            off = sum + nd;
            nd = -sum;
          }
          if (seen == 1) nvis = 0;  // one key, of weight 1: no gradient, not a rounding's
        }
        if (full && !it.few) {
          const uint64_t nd2 = f2_splat(nd);
          uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t ds = f2_mul(f2_pack(v[2 * i], v[2 * i + 1]), f2_add(f2_pack(w[2 * i], w[2 * i + 1]), nd2));
            pk[i] = pack2(f2_lo(ds), f2_hi(ds));
            if (BIAS) acc[i & 1] = f2_add(acc[i & 1], ds);
          }
          if (BIAS) {
            const uint64_t sum = f2_add(acc[0], acc[1]);
            off += f2_lo(sum) + f2_hi(sum);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = 2 * i < nvis ? v[2 * i] * (w[2 * i] + nd) : 0.f;
            const float y = 2 * i + 1 < nvis ? v[2 * i + 1] * (w[2 * i + 1] + nd) : 0.f;
            pk[i] = pack2(x, y);
            if (BIAS && !few_row) off += x + y;
          }
        }
        ptx::tmem_st16_nowait(own, pk);
        // the keys behind the sequence's, where the tensor goes on: their rows of K
        // cleared (S of this block, which also read the tile, is complete)
        if ((it.j0 + j) * 128 + 128 > it.len && it.len < a.Sk) {
          const int r = (warp - EW0) * 8 + lane / 4;
          if ((it.j0 + j) * 128 + r >= it.len) {
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
        if (lane == 0) ptx::mbar_arrive(ds_full(b));
      }
      if (!ok) break;
      // what follows takes delta as sum P dP
      if (it.few || BIAS) {
        if (BIAS && it.whole > 1) {
          // (a row of few keys has its whole sum in every column group)
          const float x = few_row && sub > 0 ? 0.f : off;
          if (!row_sum(x, off)) {
            ok = false;
            if (lane == 0) wait_failed(114);
            break;
          }
        }
        if (it.part) {
          if (sub == 0) it.part[128 * a.D + row] = it.n > 0 ? off : 0.f;
        } else if (sub == 0 && it.n > 0) {
          a.delta[((int64_t)it.b * a.H + it.h) * a.q_pitch + it.q0 + row] = few_row ? nd : nd - off;
        }
      }
      float v[32];
      if (it.n > 0) {
        // the item's last accumulation is complete (or the MMA thread gave up)
        if (!warp_wait(bar_fin, nf & 1)) {
          ok = false;
          if (lane == 0) wait_failed(112);
          break;
        }
        ++nf;
        ptx::tc_fence_after();
        // tcgen05.ld is warp-collective: every lane loads (DP = 64: what the last two
        // column groups load is not used)
        ptx::tmem_ld32(t_dq + lane_off + (sub * 32 < DP ? sub * 32 : 0), v);
      } else {
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = 0.f;
      }
      if (valid_q && sub * 32 < a.D) {
        if (it.part)
          store_part(it.part + row * a.D + sub * 32, v, a.D - sub * 32);
        else
          store_row(static_cast<__nv_bfloat16*>(a.dq) + it.b * a.sdq.b + qi * a.sdq.s + it.h * a.sdq.h + sub * 32, v,
                    a.D - sub * 32, a.scale);
      }
      __syncwarp();
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
// 128 keys of one key head.  Block x of the item's, from `first` on n of them: BQ queries
// from i0 + x % per_head on, of query head g share + x / per_head.
struct KvItem {
  int g, b, k0, len, p0, i0, per_head, first, n;
};
template <int BQ>
__device__ __forceinline__ KvItem kv_item(const Plan& p, const Order* o, const Work& w) {
  const Args& a = p.a;
  KvItem it;
  it.g = w.item % a.G;
  int tile;
  key_item(a, o, w.item / a.G, p.tiles, &tile, &it.b);
  it.k0 = tile * 128;
  it.len = a.len(it.b);
  it.p0 = a.start(it.b);
  it.i0 = a.causal ? max(0, it.k0 - it.p0) / BQ : 0;  // blocks before see none of these keys
  it.per_head = it.k0 < it.len ? max(0, (a.Sq + BQ - 1) / BQ - it.i0) : 0;
  int end;
  cut_blocks(p, w.piece, it.per_head * a.share, &it.first, &end);
  it.n = end - it.first;
  return it;
}

// Two pairs of floats from shared memory.  (In the order of the program: the compiler would
// fetch a block's all at once, and spill.)
__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t& x, uint64_t& y) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(addr));
}

// A warp's part of a block, 32 keys (rows) x 32 queries: where it lies, and the bias that
// all of its scores have.
template <bool BIAS>
struct KvTile {
  bool on_left, on_right;  // R or more from the diagonal
  float mul, add;

  // scores v of keys kw + lane, queries from position pq on
  __device__ __forceinline__ void start(const Plan& p, int h, int kw, int pq, int lane, float (&v)[32]) {
    mul = p.scale_log2;
    if (!BIAS) return;
    add = 0.f;
    on_right = kw - (pq + 31) >= p.a.bias.R;
    on_left = !on_right && kw + 31 - pq <= -p.a.bias.R;
    if (on_right) {
      add = __ldg(p.a.bias.at(h, p.a.bias.R));
    } else if (on_left) {
      add = __ldg(p.a.bias.at(h, -p.a.bias.R));
    } else {
      const float* bv = p.a.bias.at(h, kw - pq) + lane;
#pragma unroll
      for (int x = 0; x < 32; ++x) v[x] = fmaf(v[x], p.scale_log2, __ldg(bv - x));
      mul = 1.f;
    }
  }
  // Scores to weights, nl the shared address of the queries' -lse (base 2).
  __device__ __forceinline__ void weights(uint32_t nl, float (&v)[32]) const {
    const uint64_t sc = f2_splat(mul), ad = BIAS ? f2_splat(add) : 0ull;
#pragma unroll
    for (int x = 0; x < 32; x += 4) {
      uint64_t n[2];
      lds_pairs(nl + 4 * x, n[0], n[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (BIAS) n[e] = f2_add(n[e], ad);
        const uint64_t y = f2_fma(f2_pack(v[x + 2 * e], v[x + 2 * e + 1]), sc, n[e]);
        v[x + 2 * e] = fast_exp2(f2_lo(y));
        v[x + 2 * e + 1] = fast_exp2(f2_hi(y));
      }
    }
  }
};
// Weights v[FIRST ..] to dS, from 16 of dP and the shared address of the queries' -delta.
template <int FIRST>
__device__ __forceinline__ void gradients(uint32_t nd, const float (&w)[16], float (&v)[32]) {
#pragma unroll
  for (int x = 0; x < 16; x += 4) {
    uint64_t n[2];
    lds_pairs(nd + 4 * (FIRST + x), n[0], n[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int at = FIRST + x + 2 * e;
      const uint64_t ds = f2_mul(f2_pack(v[at], v[at + 1]), f2_add(f2_pack(w[x + 2 * e], w[x + 2 * e + 1]), n[e]));
      v[at] = f2_lo(ds);
      v[at + 1] = f2_hi(ds);
    }
  }
}

// A warp's share of the bias's gradient: sums by bucket in shared memory, those of scores
// far from the diagonal in registers.
struct KvBias {
  float far_left = 0.f, far_right = 0.f;
  uint32_t bucket, diag;  // shared addresses, the warp's own: [MAX_BUCKETS], [2][64] fp32

  __device__ __forceinline__ void init(const Args& a, uint32_t buckets, uint32_t diagonals, int lane) {
    bucket = buckets;
    diag = diagonals;
    for (int x = lane; x < a.bias.buckets; x += 32) ptx::sts(bucket + 4 * x, 0.f);
    __syncwarp();
  }
  // dS w of 32 keys, the first at distance n0 + 31 from query 0, summed by bucket.
  __device__ __forceinline__ void sum(const Args& a, bool on_left, bool on_right, int n0, int lane, const float (&w)[32]) {
    if (on_left || on_right) {
      uint64_t s[2] = {f2_pack(w[0], w[1]), f2_pack(w[2], w[3])};
#pragma unroll
      for (int x = 4; x < 32; x += 2) s[x / 2 & 1] = f2_add(s[x / 2 & 1], f2_pack(w[x], w[x + 1]));
      s[0] = f2_add(s[0], s[1]);
      const float t = f2_lo(s[0]) + f2_hi(s[0]);
      if (on_left) far_left += t;
      else far_right += t;
      return;
    }
    // along the diagonals, that of element (r, x) r - x + 31, of distance n0 + the same; two
    // chains, of columns 0 .. 15 (diagonals 16 .. 62) and 16 .. 31 (0 .. 46)
    float run0 = 0.f, run1 = 0.f;
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      run0 = __shfl_up_sync(0xffffffffu, run0, 1);
      run1 = __shfl_up_sync(0xffffffffu, run1, 1);
      run0 = (lane == 0 ? 0.f : run0) + w[x];
      run1 = (lane == 0 ? 0.f : run1) + w[16 + x];
      if (lane == 31) {
        ptx::sts(diag + 4 * (62 - x), run0);
        ptx::sts(diag + 256 + 4 * (46 - x), run1);
      }
    }
    if (lane < 31) {
      ptx::sts(diag + 4 * (16 + lane), run0);
      ptx::sts(diag + 256 + 4 * lane, run1);
    }
    __syncwarp();
    // a bucket's diagonals stand side by side: sums within runs of equal buckets, added by
    // each run's last lane
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int n = n0 + 32 * half + lane;
      const int u = a.bias.index[max(-a.bias.R, min(a.bias.R, n)) + a.bias.R];
      const int before = __shfl_up_sync(0xffffffffu, u, 1);
      const uint32_t heads = __ballot_sync(0xffffffffu, lane == 0 || u != before);
      const int first = 31 - __clz(heads & (0xffffffffu >> (31 - lane)));  // of this lane's run
      const int d = 32 * half + lane;  // (63: none)
      float t = 0.f;
      if (d >= 16 && d < 63) t = ptx::lds(diag + 4 * d);
      if (d < 47) t += ptx::lds(diag + 256 + 4 * d);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float below = __shfl_up_sync(0xffffffffu, t, o);
        if (lane - o >= first) t += below;
      }
      if (lane == 31 || (heads >> (lane + 1) & 1)) ptx::sts(bucket + 4 * u, ptx::lds(bucket + 4 * u) + t);
      __syncwarp();
    }
  }
  // The buckets of a finished head as one of its item's DKV_WARPS partial rows, and 0 for
  // the next.
  __device__ __forceinline__ void flush(const Plan& p, Work w, int h, int warp_row, int lane) {
    const Args& a = p.a;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      far_left += __shfl_xor_sync(~0u, far_left, o);
      far_right += __shfl_xor_sync(~0u, far_right, o);
    }
    if (lane == 0) {
      ptx::sts(bucket + 4 * a.bias.left, ptx::lds(bucket + 4 * a.bias.left) + far_left);
      ptx::sts(bucket + 4 * a.bias.right, ptx::lds(bucket + 4 * a.bias.right) + far_right);
    }
    __syncwarp();
    far_left = far_right = 0.f;
    // rows [0, batch tiles) are those of whole items and of first pieces, then the other
    // pieces' of the items from the first (sequence, tile) with a cut one on
    const int bt = w.item / a.G, cut0 = p.cut.whole / a.G, others = p.cut.pieces - 1;
    const int64_t beyond = (int64_t)a.B * p.tiles + (int64_t)(bt - cut0) * others;
    auto at = [&](int64_t row) {
      return a.bias_part + (h * a.bias_rows + row * DKV_WARPS + warp_row) * a.bias.buckets;
    };
    float* out = at(w.piece <= 0 ? bt : beyond + w.piece - 1);
    for (int x = lane; x < a.bias.buckets; x += 32) {
      out[x] = ptx::lds(bucket + 4 * x);
      ptx::sts(bucket + 4 * x, 0.f);
    }
    if (w.piece < 0 && bt >= cut0)  // (a whole item beside cut ones: it has no other pieces)
      for (int q = 0; q < others; ++q)
        for (int x = lane; x < a.bias.buckets; x += 32) at(beyond + q)[x] = 0.f;
    __syncwarp();
  }
};

// Warp 0 TMA (an item's K and V, then Q_i and dO_i into a ring, each stage with its queries'
// lse and delta), warp 1 TMEM and the S^T and dP^T MMAs, warp 2 the dV and dK MMAs, warps
// 4..19 element-wise (lanes 32 (w % 4) .., one key row each, 32 columns).  An
// element-wise warp starts on S^T while dP^T is formed.
//
// DP = 64: blocks of 128 queries, all 16 warps on each.  TMEM: S^T of even blocks 0..127, of
// odd ones 128..255, dP^T 256..383 (released as soon as it is loaded), dV 384.., dK 448..;
// P^T and dS^T, packed, stand over a warp's own 32 columns of S^T.
//
// DP = 128: the accumulators leave room for 64 queries a block: S^T of buffer b at 128 b ..,
// dP^T at + 64 .., dV 256.., dK 384..; P^T over S^T, dS^T over dP^T.  Two groups of 8 warps
// take a buffer each, so that one works while the other waits for its block (all 16 on every
// block, 16 columns each, waited on every barrier twice as often: 629 us against 497 when
// both were built, 505 now, at 8 sequences of 2048, 19 heads).  The products read 64 queries' operands with the whole of K
// and V: bound by shared memory's 128 bytes a clock, 1280 clocks a block against 1024 of the
// tensor cores'.
template <int DP_, bool BIAS>
struct Kv {
  static constexpr int DP = DP_, BQ = DP == 64 ? 128 : 64;
  static constexpr int GROUPS = DP == 64 ? 1 : 2;               // of element-wise warps, a block each
  static constexpr int NDP = DP == 64 ? 1 : 2, NSET = DP == 64 ? 2 : 1;  // buffers of dP^T; of K and V
  static constexpr int QST = 4;
  static constexpr int TILE = tile_bytes<DP>(), QTILE = TILE / 128 * BQ;
  static constexpr int KV = 0, Q = NSET * 2 * TILE, DO = Q + QST * QTILE;  // [set][K | V]
  static constexpr int STAT = DO + QST * QTILE;                            // [stage][-lse2[BQ] | -delta[BQ]] fp32
  static constexpr int BUCKET = STAT + QST * 2 * BQ * 4;                   // [16][MAX_BUCKETS] fp32
  static constexpr int DIAG = BUCKET + (BIAS ? EW * MAX_BUCKETS * 4 : 0);  // [16][2][64] fp32
  static constexpr int ORDER = DIAG + (BIAS ? EW * 128 * 4 : 0);  // Order
  static constexpr int BAR = ORDER + ((int)sizeof(Order) + 15) / 16 * 16;
  static constexpr int NBAR = 4 + 8 + NDP + 2 * NSET + 2 * QST;
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
  using L = Kv<DP, BIAS>;
  constexpr int TILE = L::TILE, QTILE = L::QTILE, QST = L::QST, NSET = L::NSET, NDP = L::NDP, BQ = L::BQ;
  constexpr int GROUPS = L::GROUPS, QBOX = BQ * 128;
  constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(128, BQ, false, false);
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
  const uint32_t bar_fin = bars, drain = bars + 8u, acc_empty = bars + 16u, dp_empty = bars + 24u;
  auto s_full = [&](uint32_t b) { return bars + 8u * (4 + b); };    // S^T formed
  auto p_full = [&](uint32_t b) { return bars + 8u * (6 + b); };    // P^T written
  auto ds_full = [&](uint32_t b) { return bars + 8u * (8 + b); };   // dS^T written
  auto pd_empty = [&](uint32_t b) { return bars + 8u * (10 + b); };  // and both read
  auto dp_full = [&](uint32_t b) { return bars + 8u * (12 + b); };  // dP^T formed
  auto kv_full = [&](uint32_t e) { return bars + 8u * (12 + NDP + e); };
  auto kv_empty = [&](uint32_t e) { return bars + 8u * (12 + NDP + NSET + e); };
  auto q_full = [&](uint32_t s) { return bars + 8u * (12 + NDP + 2 * NSET + s); };
  auto q_empty = [&](uint32_t s) { return bars + 8u * (12 + NDP + 2 * NSET + QST + s); };
  const uint32_t tslot = bars + 8u * L::NBAR;
  const Args& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
  const int cta = blockIdx.x, G = gridDim.x;

  if (tid == 0) {
    ptx::mbar_init(bar_fin, 1);
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(acc_empty, EW);
    ptx::mbar_init(dp_empty, EW);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(s_full(b), 1);
      ptx::mbar_init(p_full(b), EW / GROUPS);
      ptx::mbar_init(ds_full(b), EW / GROUPS);
      ptx::mbar_init(pd_empty(b), 1);
    }
    for (int x = 0; x < NDP + 2 * NSET + 2 * QST; ++x) ptx::mbar_init(dp_full(x), 1);
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
  auto t_s = [&](uint32_t b) { return tmem + 128u * b; };
  auto t_dp = [&](uint32_t b) { return NDP == 1 ? tmem + 256u : tmem + 128u * b + 64u; };
  // where a warp's packed words of its columns 32 c .. stand: P^T at t_s + 32 c
  auto t_ds = [&](uint32_t b) { return NDP == 1 ? t_s(b) + 16u : t_dp(b); };
  const uint32_t t_dv = tmem + (DP == 64 ? 384 : 256), t_dk = t_dv + DP;
  pdl_wait();
  pdl_trigger();
  Order* const order = reinterpret_cast<Order*>(gbase + L::ORDER);
  if (ragged(a)) order_sequences(a, reinterpret_cast<int*>(gbase), order, order->tiles);
  bool ok = true;
  Work wk;

  if (warp < EW0) {
    fewer_registers<REGS_ISSUE>();
    if (warp == 0) {
      if (ptx::elect_one()) {
        uint32_t ii = 0, nk = 0;  // blocks and items with blocks so far
        for (int k = 0; ok && work_at(p, k, cta, G, &wk); ++k) {
          const KvItem it = kv_item<BQ>(p, order, wk);
          if (it.n == 0) continue;
          const uint32_t e = nk % NSET;
          if (nk >= NSET && !wait1(kv_empty(e), ((nk / NSET) & 1) ^ 1)) {
            ok = false;
            break;
          }
          ptx::mbar_arrive_expect_tx(kv_full(e), 2 * TILE);
          load_tile<DP, 128>(base + L::KV + 2 * e * TILE, &tk, kv_full(e), it.k0, it.g, it.b);
          load_tile<DP, 128>(base + L::KV + (2 * e + 1) * TILE, &tv, kv_full(e), it.k0, it.g, it.b);
          ++nk;
          int head = it.g * a.share + it.first / it.per_head, i = it.i0 + it.first % it.per_head;
          for (int j = 0; j < it.n; ++j, ++ii) {
            const uint32_t s = ii % QST;
            if (ii >= QST && !wait1(q_empty(s), ((ii / QST) & 1) ^ 1)) {
              ok = false;
              break;
            }
            ptx::mbar_arrive_expect_tx(q_full(s), 2 * QTILE + 2 * BQ * 4);
            if (BQ == 64) {
              load_tile<DP, 64>(base + L::Q + s * QTILE, &tq, q_full(s), i * 64, head, it.b);
              load_tile<DP, 64>(base + L::DO + s * QTILE, &tdo, q_full(s), i * 64, head, it.b);
            } else {
              load_two<DP>(base + L::Q + s * QTILE, &tq, q_full(s), i * 128, head, it.b);
              load_two<DP>(base + L::DO + s * QTILE, &tdo, q_full(s), i * 128, head, it.b);
            }
            const int64_t at = ((int64_t)it.b * a.H + head) * a.q_pitch + i * BQ;
            const uint32_t st = base + L::STAT + s * (2 * BQ * 4);
            ptx::bulk_load(st, a.neg_lse2 + at, BQ * 4, q_full(s));
            ptx::bulk_load(st + BQ * 4, a.delta + at, BQ * 4, q_full(s));
            if (++i == it.i0 + it.per_head) {
              i = it.i0;
              ++head;
            }
          }
        }
        if (!ok) wait_failed(201);
        // every load issued has landed before the CTA may exit
        bool dr = true;
        for (uint32_t e = 0; e < NSET; ++e)
          if (nk > e) dr = wait1(kv_full(e), ((nk - 1 - e) / NSET) & 1) && dr;
        for (uint32_t s = 0; s < QST; ++s)
          if (ii > s) dr = wait1(q_full(s), ((ii - 1 - s) / QST) & 1) && dr;
        if (!dr) wait_failed(202);
      }
    } else if (warp == 1) {
      if (ptx::elect_one()) {
        uint32_t ii = 0, nk = 0;
        for (int k = 0; ok && work_at(p, k, cta, G, &wk); ++k) {
          const KvItem it = kv_item<BQ>(p, order, wk);
          if (it.n == 0) continue;
          const uint32_t e = nk % NSET;
          if (!wait1(kv_full(e), (nk / NSET) & 1)) {
            ok = false;
            wait_failed(203);
            break;
          }
          ++nk;
          const uint32_t kt = base + L::KV + 2 * e * TILE, vt = kt + TILE;
          for (int j = 0; j < it.n; ++j, ++ii) {  // S^T = K Q_i^T, dP^T = V dO_i^T
            const uint32_t s = ii % QST, b = ii & 1;
            // (the accumulations of the block before the last, whose operands lay in this
            // buffer, are done)
            if (!wait1(q_full(s), (ii / QST) & 1) || (ii >= 2 && !wait1(pd_empty(b), ((ii / 2) & 1) ^ 1))) {
              ok = false;
              wait_failed(204);
              break;
            }
            ptx::tc_fence_after();
            const uint32_t qt = base + L::Q + s * QTILE, dt = base + L::DO + s * QTILE;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
              ptx::mma_bf16(t_s(b), kmajor_desc(kt, kk), kmajor_desc(qt, kk, QBOX), IDESC_S, kk > 0);
            ptx::mma_commit(s_full(b));
            if (NDP == 1) {  // (the element-wise warps have loaded the previous block's dP^T)
              if (ii >= 1 && !wait1(dp_empty, (ii - 1) & 1)) {
                ok = false;
                wait_failed(205);
                break;
              }
              ptx::tc_fence_after();
            }
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
              ptx::mma_bf16(t_dp(b), kmajor_desc(vt, kk), kmajor_desc(dt, kk, QBOX), IDESC_S, kk > 0);
            ptx::mma_commit(dp_full(NDP == 1 ? 0 : b));
          }
          if (ok) ptx::mma_commit(kv_empty(e));  // the item's last read of K and V
        }
        ptx::mma_commit(drain);  // completes once every MMA this thread issued has
        if (!wait1(drain, 0)) {
          ok = false;
          wait_failed(207);
        }
      }
    } else if (warp == ACC_WARP) {
      if (ptx::elect_one()) {
        uint32_t ii = 0, nk = 0;
        for (int k = 0; ok && work_at(p, k, cta, G, &wk); ++k) {
          const KvItem it = kv_item<BQ>(p, order, wk);
          if (it.n == 0) continue;
          // (the element-wise warps have read the item before's dV and dK)
          if (nk > 0 && !wait1(acc_empty, (nk - 1) & 1)) {
            ok = false;
            wait_failed(210);
            break;
          }
          for (int j = 0; j < it.n; ++j, ++ii) {  // dV += P^T dO_i, dK += dS^T Q_i
            const uint32_t s = ii % QST, b = ii & 1;
            const uint32_t qt = base + L::Q + s * QTILE, dt = base + L::DO + s * QTILE;
            if (!wait1(p_full(b), (ii / 2) & 1)) {
              ok = false;
              wait_failed(206);
              break;
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < BQ / 16; ++kk)
              ptx::mma_bf16_ts(t_dv, t_s(b) + 32u * (kk >> 1) + 8u * (kk & 1), mnmajor_desc(dt, kk, QBOX), IDESC_ACC,
                               (j > 0 || kk > 0) ? 1u : 0u);
            if (!wait1(ds_full(b), (ii / 2) & 1)) {
              ok = false;
              wait_failed(213);
              break;
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < BQ / 16; ++kk)
              ptx::mma_bf16_ts(t_dk, t_ds(b) + 32u * (kk >> 1) + 8u * (kk & 1), mnmajor_desc(qt, kk, QBOX), IDESC_ACC,
                               (j > 0 || kk > 0) ? 1u : 0u);
            // S^T, dP^T of block ii (which also read Q_i, dO_i) completed before P^T and
            // dS^T could be handed over: the stage is free once these MMAs are
            ptx::mma_commit(pd_empty(b));
            ptx::mma_commit(q_empty(s));
          }
          if (!ok) break;
          ptx::mma_commit(bar_fin);  // the item's dV and dK are complete once this is
          ++nk;
        }
        // every MMA this thread issued is complete before the CTA may exit
        if (nk > 0 && !wait1(bar_fin, (nk - 1) & 1)) {
          ok = false;
          wait_failed(211);
        }
        if (!ok) {  // one more commit drains whatever was issued after the last finished item
          ptx::mma_commit(bar_fin);
          (void)wait1(bar_fin, nk & 1);
        }
      }
    }
  } else {
    more_registers<REGS_EW>();
    const int qq = warp & 3, part = (warp - EW0) >> 2;  // lane quarter
    const int group = GROUPS == 2 ? part >> 1 : 0, c = GROUPS == 2 ? part & 1 : part;  // columns 32 c ..
    const uint32_t lane_off = (uint32_t)(qq * 32) << 16;
    const bool grad = BIAS && a.bias_part != nullptr;
    KvBias kb;
    if (grad)
      kb.init(a, base + L::BUCKET + (warp - EW0) * MAX_BUCKETS * 4, base + L::DIAG + (warp - EW0) * 512, lane);
    // Block ii of the warp, queries from qi on: weights and dS (masked where !FULL).
    auto block = [&](auto FULL, uint32_t ii, int h, int kw, int len, int p0, int qi) {
      const uint32_t b = ii & 1, own = lane_off + c * 32;
      const uint32_t st = base + L::STAT + ii % QST * (2 * BQ * 4) + c * 128;
      const int pq = p0 + qi;
      // queries qi + x with x < lo are before this key (causal), those with x >= hi past the
      // last; a key past the sequence's sees none
      int lo = 0, hi = 0;
      if (!FULL) {
        lo = a.causal ? kw + lane - pq : -(1 << 30);
        hi = kw + lane < len ? a.Sq - qi : 0;
      }
      float v[32];
      ptx::tmem_ld32(t_s(b) + own, v);
      KvTile<BIAS> tile;
      tile.start(p, h, kw, pq, lane, v);
      tile.weights(st, v);
      if (!FULL) {
#pragma unroll
        for (int x = 0; x < 32; ++x)
          if (x < lo || x >= hi) v[x] = 0.f;
      }
      {
        uint32_t pk[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) pk[x] = pack2(v[2 * x], v[2 * x + 1]);
        ptx::tmem_st16_nowait(t_s(b) + own, pk);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full(b));
      }
      if (!warp_wait(dp_full(NDP == 1 ? 0 : b), (NDP == 1 ? ii : ii / 2) & 1)) {
        if (lane == 0) wait_failed(209);
        return false;
      }
      ptx::tc_fence_after();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float w[16];
        ptx::tmem_ld16(t_dp(b) + own + 16 * half, w);
        if (NDP == 1 && half == 1) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(dp_empty);  // dP^T's buffer may be overwritten
        }
        if (half == 0) gradients<0>(st + 4 * BQ, w, v);
        else gradients<16>(st + 4 * BQ, w, v);
        if (!FULL) {
          // 0 times what a hidden key holds; and a query that sees one key, of weight 1, gives
          // no gradient, not a rounding's: any of a sequence of one key, causal the one at key 0
          const int first = a.causal && kw + lane == 0 ? lo + 1 : lo, end = len == 1 ? 0 : hi;
#pragma unroll
          for (int x = 16 * half; x < 16 * half + 16; ++x)
            if (x < first || x >= end) v[x] = 0.f;
        }
        uint32_t pk[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) pk[x] = pack2(v[16 * half + 2 * x], v[16 * half + 2 * x + 1]);
        ptx::tmem_st8_nowait(t_ds(b) + own + 8 * half, pk);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ds_full(b));
      if (BIAS && grad) kb.sum(a, tile.on_left, tile.on_right, kw - pq - 31, lane, v);
      return true;
    };
    uint32_t ii0 = 0, nk = 0;
    for (int k = 0; ok && work_at(p, k, cta, G, &wk); ++k) {
      int n;
      {
        const KvItem it = kv_item<BQ>(p, order, wk);
        n = it.n;
        const int kw = it.k0 + qq * 32, end = (it.g + 1) * a.share;
        int h = it.g * a.share;  // the head whose buckets are being summed
        int j = 0;
        if (GROUPS == 2) j = (int)((ii0 + (uint32_t)group) & 1);  // the group's first block
        int i = it.first + j;
        for (; j < n; j += GROUPS, i += GROUPS) {
          const uint32_t ii = ii0 + (uint32_t)j;
          while (i >= it.per_head) {  // (i: the block's place among its head's)
            if (grad) kb.flush(p, wk, h, warp - EW0, lane);
            i -= it.per_head;
            ++h;
          }
          // this block's lse and delta have landed, and its S^T is in TMEM
          if (!warp_wait(q_full(ii % QST), (ii / QST) & 1) || !warp_wait(s_full(ii & 1), (ii / 2) & 1)) {
            ok = false;
            if (lane == 0) wait_failed(208);
            break;
          }
          ptx::tc_fence_after();
          // scores wholly visible need no mask (warp-uniform)
          const int qi = (it.i0 + i) * BQ + c * 32;
          const bool full = kw + 32 <= it.len && qi + 32 <= a.Sq && (!a.causal || it.p0 + qi >= kw + 31);
          ok = full ? block(std::true_type{}, ii, h, kw, it.len, it.p0, qi)
                    : block(std::false_type{}, ii, h, kw, it.len, it.p0, qi);
          if (!ok) break;
        }
        if (!ok) break;
        ii0 += (uint32_t)n;
        if (grad)  // (heads without blocks too: their partial sums are 0)
          for (; h < end; ++h) kb.flush(p, wk, h, warp - EW0, lane);
      }
      if (n > 0) {
        if (!warp_wait(bar_fin, nk & 1)) {
          ok = false;
          if (lane == 0) wait_failed(212);
          break;
        }
        ++nk;
        ptx::tc_fence_after();
      }
      // (the item once more: what is not needed among its blocks holds no registers there)
      asm volatile("" : "+r"(wk.item));
      const KvItem it = kv_item<BQ>(p, order, wk);
      float* const sums = wk.piece < 0 ? nullptr : p.part + (int64_t)wk.part * 2 * 128 * a.D;
      const int kw = it.k0 + qq * 32;
      // 2 DP columns of dK and dV: DP / 2 of them to each of the four column groups
      const int key = kw + lane;
      const bool in = key < it.len && it.n > 0;
#pragma unroll
      for (int x = 0; x < DP / 64; ++x) {
        const bool dk = DP == 64 ? part < 2 : x == 0;
        const int col = DP == 64 ? (part & 1) * 32 : part * 32;
        float v[32];
        if (it.n > 0) {
          ptx::tmem_ld32((dk ? t_dk : t_dv) + lane_off + col, v);  // every lane loads
          if (x == DP / 64 - 1) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(acc_empty);
          }
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) v[y] = in ? v[y] : 0.f;  // (0 behind the sequence's keys)
        if (key < a.Sk && col < a.D) {
          const Strides& sd = dk ? a.sdk : a.sdv;
          if (sums)
            store_part(sums + ((dk ? 0 : 128) + key - it.k0) * a.D + col, v, a.D - col);
          else
            store_row(static_cast<__nv_bfloat16*>(dk ? a.dk : a.dv) + it.b * sd.b + key * sd.s + it.g * sd.h + col, v,
                      a.D - col, dk ? a.scale : 1.f);
        }
        __syncwarp();  // the next tcgen05.ld is warp-collective
      }
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

// ---- pieces joined ------------------------------------------------------------------------
// A cut item's 32 rows a CTA, 8 lanes a row: dq, and -delta of rows whose sums of dS were
// taken (of the first block's keys alone, or `sums`).
__global__ void __launch_bounds__(256)
xattn_dq_join_kernel(const __grid_constant__ Plan p, int sums) {
  pdl_wait();
  pdl_trigger();
  const Args& a = p.a;
  __shared__ Order order;
  __shared__ int lens[MAX_ORDER];
  if (ragged(a)) order_sequences(a, lens, &order, order.tiles);
  const int row = blockIdx.x * 32 + threadIdx.x / 8, lane = threadIdx.x % 8;
  const Work w = {p.cut.whole + (int)blockIdx.y, 0, (int)blockIdx.y * p.cut.pieces};
  const DqItem it = dq_item(p, &order, w);
  const int qi = it.q0 + row;
  if (qi >= a.Sq) return;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.dq) + it.b * a.sdq.b + qi * a.sdq.s + it.h * a.sdq.h;
  const int64_t step = dq_piece(a.D);
  for (int c = 4 * lane; c < a.D; c += 32) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int q = 0; q < p.cut.pieces; ++q) {
      const float4 x = *reinterpret_cast<const float4*>(it.part + q * step + row * a.D + c);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    *reinterpret_cast<uint2*>(out + c) = make_uint2(pack2(s.x * a.scale, s.y * a.scale), pack2(s.z * a.scale, s.w * a.scale));
  }
  if (lane == 0 && (sums || it.few)) {
    float off = 0.f;
    for (int q = 0; q < p.cut.pieces; ++q) off += it.part[q * step + 128 * a.D + row];
    a.delta[((int64_t)it.b * a.H + it.h) * a.q_pitch + qi] -= off;
  }
}
// dk (even blockIdx.y) and dv of a cut item.
__global__ void __launch_bounds__(256)
xattn_dkv_join_kernel(const __grid_constant__ Plan p) {
  pdl_wait();
  pdl_trigger();
  const Args& a = p.a;
  __shared__ Order order;
  __shared__ int lens[MAX_ORDER];
  if (ragged(a)) order_sequences(a, lens, &order, order.tiles);
  const int row = blockIdx.x * 32 + threadIdx.x / 8, lane = threadIdx.x % 8;
  const int y = blockIdx.y / 2, item = p.cut.whole + y;
  int tile, b;
  key_item(a, &order, item / a.G, p.tiles, &tile, &b);
  const int key = tile * 128 + row;
  const bool dk = blockIdx.y % 2 == 0;
  if (key >= a.Sk) return;
  const Strides& sd = dk ? a.sdk : a.sdv;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(dk ? a.dk : a.dv) + b * sd.b + key * sd.s + item % a.G * sd.h;
  const int64_t step = (int64_t)2 * 128 * a.D;
  const float* part = p.part + y * p.cut.pieces * step + ((dk ? 0 : 128) + row) * a.D;
  const float scale = dk ? a.scale : 1.f;
  for (int c = 4 * lane; c < a.D; c += 32) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int q = 0; q < p.cut.pieces; ++q) {
      const float4 x = *reinterpret_cast<const float4*>(part + q * step + c);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    *reinterpret_cast<uint2*>(out + c) = make_uint2(pack2(s.x * scale, s.y * scale), pack2(s.z * scale, s.w * scale));
  }
}

template <int DP, bool BIAS>
cudaError_t launch(const Args& a, const BwdCut& cut, cudaStream_t st) {
  CUtensorMap tq, tdo, tk, tv;
  OASES_TRY(map4d(&tq, a.q, a.sq, a.D, a.Sq, a.H, a.B, 64));
  OASES_TRY(map4d(&tdo, a.d_o, a.sdo, a.D, a.Sq, a.H, a.B, 64));
  OASES_TRY(map4d(&tk, a.k, a.sk, a.D, a.Sk, a.G, a.B, 128));
  OASES_TRY(map4d(&tv, a.v, a.sv, a.D, a.Sk, a.G, a.B, 128));
  constexpr int DQ_BYTES = DqSmem<DP>::BYTES, DKV_BYTES = Kv<DP, BIAS>::BYTES;
  static DeviceOnce attr;
  OASES_TRY(attr.run([&] {
    for (const void* f : {(const void*)xattn_dq_kernel<DP, BIAS>, (const void*)xattn_dkv_kernel<DP, BIAS>}) {
      cudaFuncAttributes at;
      const cudaError_t e = cudaFuncGetAttributes(&at, f);
      if (e != cudaSuccess) return e;
      if (at.numRegs != REGS) return cudaErrorInvalidKernelImage;  // (the warpgroups' shares would not add up)
    }
    const cudaError_t e =
        cudaFuncSetAttribute(xattn_dq_kernel<DP, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, DQ_BYTES);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(xattn_dkv_kernel<DP, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, DKV_BYTES);
  }));
  const int64_t rows = (int64_t)a.B * (a.q_pitch / 4) * a.H;
  if ((rows + 15) / 16 > INT32_MAX) return cudaErrorInvalidConfiguration;
  OASES_TRY(launch_pdl(xattn_stats_kernel, dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, st, a, rows));
  Plan pq;
  pq.a = a;
  pq.scale_log2 = LOG2E * a.scale;
  Plan pk = pq;
  pq.tiles = (a.Sq + 127) / 128;
  pq.cut = cut.dq;
  pq.part = a.piece_dq;
  pk.tiles = (a.Sk + 127) / 128;
  pk.cut = cut.dkv;
  pk.part = a.piece_dkv;
  auto grid = [](const Pieces& c) { return dim3((unsigned)(c.whole ? sm_count() : c.rest * c.pieces)); };
  OASES_TRY(launch_pdl(xattn_dq_kernel<DP, BIAS>, grid(pq.cut), dim3(NT), DQ_BYTES, st, tq, tdo, tk, tv, pq));
  if (pq.cut.pieces > 1)
    OASES_TRY(launch_pdl(xattn_dq_join_kernel, dim3(4, (unsigned)pq.cut.rest), dim3(256), 0, st, pq, (int)BIAS));
  OASES_TRY(launch_pdl(xattn_dkv_kernel<DP, BIAS>, grid(pk.cut), dim3(NT), DKV_BYTES, st, tk, tv, tq, tdo, pk));
  if (pk.cut.pieces == 1) return cudaSuccess;
  return launch_pdl(xattn_dkv_join_kernel, dim3(4, 2 * (unsigned)pk.cut.rest), dim3(256), 0, st, pk);
}

// Items in whole rounds of the SMs, and the rest in as many pieces as fill one more round,
// `least` of an item's `blocks` to a piece at least.
Pieces pieces(int64_t items, int blocks, int least) {
  const int sms = sm_count();
  Pieces c;
  c.rest = (int)(items % sms);
  c.whole = (int)(items - c.rest);
  c.pieces = c.rest ? std::max(1, std::min(sms / c.rest, blocks / least)) : 1;
  return c;
}

}  // namespace

size_t xattn_dq_piece_bytes(int D) { return 4 * (size_t)dq_piece(D); }
bool xattn_bwd_cut(const Args& a, BwdCut* cut) {
  const int64_t nq = (int64_t)((a.Sq + 127) / 128) * a.B * a.H, nk = (int64_t)((a.Sk + 127) / 128) * a.B * a.G;
  if (std::max(nq, nk) > INT32_MAX / 2) return false;
  const int bq = a.D <= 64 ? 128 : 64;
  // (a piece's sums cost 64 or 128 KB written and read again, the time of about two blocks)
  cut->dq = pieces(nq, (a.Sk + 127) / 128, 4);
  cut->dkv = pieces(nk, (int)std::min<int64_t>((int64_t)((a.Sq + bq - 1) / bq) * a.share, INT32_MAX / 2), a.D <= 64 ? 4 : 8);
  return true;
}

cudaError_t xattn_bwd_tc(const Args& a, cudaStream_t st) {
  BwdCut cut;
  if (!xattn_bwd_cut(a, &cut)) return cudaErrorInvalidConfiguration;
  if (a.D <= 64) return a.bias.buckets ? launch<64, true>(a, cut, st) : launch<64, false>(a, cut, st);
  return a.bias.buckets ? launch<128, true>(a, cut, st) : launch<128, false>(a, cut, st);
}

int xattn_bwd_read_and_clear_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_xattn_bwd_error, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_xattn_bwd_error, &z, sizeof(int));
  return v;
}

}  // namespace oases
