// Persistent tcgen05 main loop with an epilogue given as a type, for the
// operators whose epilogues differ from the block's (gated feed-forward,
// cross entropy):
//   D[m, n] = sum_k A(m, k) B(n, k), bf16 operands, fp32 accumulation in TMEM.
//
// One CTA (CL = 1) per 128 x BN tile or a CTA pair (CL = 2) per 256 x BN tile,
// one CTA per SM, 320 threads: warp 0 loads K-slices of 64 elements with TMA
// into a ring of shared-memory stages, warp 1 issues the MMAs, warps 2..9 read
// the double-buffered accumulator and run Epi::tile while the next tile's main
// loop is on.  A pair shares each MMA (M = 256): CTA r holds A rows 128 r ..
// and half of the B tile.  In a DUAL tile the B rows are BN / 2 rows from n0
// and the BN / 2 rows b_off further down, so columns c and BN / 2 + c of the
// accumulator are two products of one output column (gate and up).
//
// A contraction that leaves SMs idle is split: split z of `splits` takes
// K-slices [z kbs, (z + 1) kbs) and its epilogue sees z.
//
// Several products can share a launch (a backward's dx and weight gradients):
// their tiles, of different lengths, are dealt to the CTAs longest first so that
// the CTAs finish together, instead of every product leaving its last round of
// tiles partly idle.
//
// Every mbarrier wait is bounded (2 s); on expiry the thread records an error,
// drains what it has in flight and leaves, so the kernel always terminates.
#pragma once
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "sm100_ptx.cuh"

namespace oases {
namespace core {

// Error word of this translation unit's kernels (0: none).
static __device__ int g_core_error;

constexpr int BM = 128;
constexpr int BKE = 64;                    // K elements per stage (128 bytes)
constexpr int NTHREADS = 320;              // 2 control warps + 8 epilogue warps
constexpr int64_t A_L2_BYTES = 48ll << 20;  // A up to this size stays in L2 across tile rounds
constexpr int GROUP_M = 8;                 // row blocks per group of the tile order beyond it

template <int BN, int CL, int STG, int WBARS>  // STG, WBARS: staging bytes and barriers per epilogue warp
struct Cfg {
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = BN / CL * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int EPI_BYTES = 8 * STG;
  static constexpr int STAGES = (226 * 1024 - EPI_BYTES - 1536) / STAGE;
  static constexpr int EPI_OFF = STAGES * STAGE;
  static constexpr int BAR_BYTES = 8 * (2 * STAGES + 5 + 8 * WBARS) + 8;
  static constexpr int SMEM = STAGES * STAGE + EPI_BYTES + BAR_BYTES + 1024;
  static constexpr int TMEM_COLS = 2 * BN > 256 ? 512 : 2 * BN;  // a power of two
  static_assert(STAGE % 1024 == 0 && STG % 1024 == 0, "swizzled tiles keep 1024-byte alignment");
  static_assert(SMEM <= 227 * 1024 && STAGES >= 3 && STAGES <= 31, "shared memory");
};

struct Problem {
  int M, N, K;         // N: output columns (of the two products each, DUAL)
  int a_rows;          // rows of A's box: 128, fewer (a multiple of 8) when M is smaller
  int b_off;           // DUAL: row offset of the second product's B
  int num_mp, num_n;   // tiles along M (CL * 128 rows) and N
  int group;           // row blocks per group of the tile order
  int splits, kbs;     // splits of the contraction, K-slices per split
};

constexpr int MAX_SLOTS = 160;  // CTAs or CTA pairs of a launch of several products

template <class Epi>
struct Item {
  CUtensorMap a, b;
  typename Epi::Params ep;
  Problem p;
  int a_k;  // A is K-major
};
// The products of a launch.  One: its tiles go round the CTAs.  Several: slot s
// (CTA or pair) takes tiles [first[i][s], first[i][s + 1]) of product i, in turn.
template <class Epi, int ITEMS>
struct Work {
  Item<Epi> item[ITEMS];
  uint16_t first[ITEMS][MAX_SLOTS + 1];
};
template <class Epi>
struct Work<Epi, 1> {
  Item<Epi> item[1];
};

// Walks the tiles of a slot.
template <class Epi, int ITEMS>
struct Walk {
  const Work<Epi, ITEMS>& w;
  const int slot, slots;
  int i, t, end;
  __device__ __forceinline__ Walk(const Work<Epi, ITEMS>& w_, int slot_, int slots_)
      : w(w_), slot(slot_), slots(slots_), i(0) {
    if constexpr (ITEMS == 1) {
      t = slot;
      end = w.item[0].p.num_mp * w.item[0].p.num_n * w.item[0].p.splits;
    } else {
      t = w.first[0][slot];
      end = w.first[0][slot + 1];
      skip();
    }
  }
  __device__ __forceinline__ void skip() {
    if constexpr (ITEMS > 1)
      while (t >= end && ++i < ITEMS) {
        t = w.first[i][slot];
        end = w.first[i][slot + 1];
      }
  }
  __device__ __forceinline__ bool more() const { return ITEMS == 1 ? t < end : i < ITEMS; }
  __device__ __forceinline__ void next() {
    if constexpr (ITEMS == 1) {
      t += slots;
    } else {
      ++t;
      skip();
    }
  }
  __device__ __forceinline__ const Item<Epi>& item() const { return w.item[ITEMS == 1 ? 0 : i]; }
};

// A_MODE: 1 A is K-major, 0 it is not, 2 as each item says.
template <class Epi, int BN, int A_MODE, bool B_K, int CL, int ITEMS>
__global__ void __launch_bounds__(NTHREADS, 1)
gemm_core_kernel(const __grid_constant__ Work<Epi, ITEMS> work) {
  using C = Cfg<BN, CL, Epi::STG, Epi::WBARS>;
  constexpr int BNH = BN / CL;                    // B rows held by this CTA
  constexpr int TN = Epi::DUAL ? BN / 2 : BN;     // output columns per tile
  static_assert(!Epi::DUAL || (CL == 2 && B_K), "DUAL tiles are CTA pairs over K-major weights");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::EPI_OFF + C::EPI_BYTES;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (C::STAGES + s); };
  auto tfull = [&](int b) { return bars + 8u * (2 * C::STAGES + b); };
  auto tempty = [&](int b) { return bars + 8u * (2 * C::STAGES + 2 + b); };
  const uint32_t drain = bars + 8u * (2 * C::STAGES + 4);
  const uint32_t wbars = drain + 8, tslot = wbars + 8u * (8 * Epi::WBARS);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = CL > 1 ? (int)ptx::cluster_rank() : 0;
  const int slot = blockIdx.x / CL, slots = gridDim.x / CL;
  // Tile order within a split: groups of `group` row blocks, the row block
  // fastest inside a group (the operands of the tiles in flight stay in L2).
  struct Tile {
    int m0, n0, z, kb0, kb1;
  };
  auto tile_of = [&](const Problem& p, int t) {
    Tile q;
    const int tiles1 = p.num_mp * p.num_n, nkb = (p.K + BKE - 1) / BKE;
    q.z = t / tiles1;
    const int r = t - q.z * tiles1, g = r / (p.group * p.num_n);
    const int gm = min(p.group, p.num_mp - g * p.group), i = r - g * p.group * p.num_n;
    q.n0 = i / gm * TN;
    q.m0 = ((g * p.group + i % gm) * CL + rank) * BM;
    q.kb0 = q.z * p.kbs;
    q.kb1 = min(nkb, q.kb0 + p.kbs);
    return q;
  };
  auto a_kmajor = [&](const Item<Epi>& it) { return A_MODE == 2 ? it.a_k != 0 : A_MODE == 1; };
  constexpr uint16_t MASK = (1u << CL) - 1u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(full(s), 1);
      ptx::mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(tfull(b), 1);
      ptx::mbar_init(tempty(b), 8 * CL);  // one arrival per epilogue warp of the pair
    }
    ptx::mbar_init(drain, 1);
    for (int i = 0; i < 8 * Epi::WBARS; ++i) ptx::mbar_init(wbars + 8u * i, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    if (CL > 1) {
      ptx::tmem_alloc_pair(tslot, C::TMEM_COLS);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(tslot, C::TMEM_COLS);
      ptx::tmem_relinquish();
    }
  }
  if (warp == 0 && lane < ITEMS) {
    ptx::prefetch_tmap(&work.item[lane].a);
    ptx::prefetch_tmap(&work.item[lane].b);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + (tslot - base));
  if (CL > 1) ptx::cluster_sync();  // the partner's barriers are initialised
  // global memory from here on (everything above overlapped the previous kernel)
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, iphase = 0;  // bit s: stage s loaded, parity of its last load
      bool ok = true;
      for (Walk<Epi, ITEMS> k(work, slot, slots); k.more() && ok; k.next()) {
        const Item<Epi>& it = k.item();
        const Problem& p = it.p;
        const bool ak = a_kmajor(it);
        const uint32_t bytes = (uint32_t)(CL * (p.a_rows * 128 + C::B_BYTES));
        const Tile q = tile_of(p, k.t);
        for (int kb = q.kb0; kb < q.kb1; ++kb) {
          if (!ptx::mbar_wait(empty(stage), phase ^ 1u)) { ok = false; break; }
          // a pair's loads complete on the even CTA's barrier, which expects both
          const uint32_t fb = CL > 1 ? ptx::mapa(full(stage), 0) : full(stage);
          if (rank == 0) ptx::mbar_arrive_expect_tx(full(stage), bytes);
          auto load = [&](uint32_t dst, const CUtensorMap* tm, int x, int y) {
            if (CL > 1)
              ptx::tma_load_2d_pair(dst, tm, fb, x, y);
            else
              ptx::tma_load_2d(dst, tm, fb, x, y);
          };
          const uint32_t sa = base + stage * C::STAGE, sb = sa + C::A_BYTES;
          const int k0 = kb * BKE;
          if (ak) {
            load(sa, &it.a, k0, q.m0);
          } else {
            load(sa, &it.a, q.m0, k0);
            load(sa + 8192, &it.a, q.m0 + 64, k0);
          }
          const int nb = Epi::DUAL ? q.n0 + rank * p.b_off : q.n0 + rank * BNH;
          if (B_K) {
            load(sb, &it.b, k0, nb);
          } else {
#pragma unroll
            for (int c = 0; c < BNH / 64; ++c) load(sb + c * 8192, &it.b, nb + 64 * c, k0);
          }
          issued |= 1u << stage;
          iphase = (iphase & ~(1u << stage)) | (phase << stage);
          if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // every load this thread issued has landed before the CTA leaves (the odd
      // CTA of a pair sees that through the release of each stage)
      for (int s = 0; s < C::STAGES; ++s)
        if ((issued >> s) & 1u)
          if (!ptx::mbar_wait(rank == 0 ? full(s) : empty(s), (iphase >> s) & 1u)) ok = false;
      if (!ok) atomicExch(&g_core_error, 1);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {  // the even CTA issues the pair's MMAs
      int stage = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (Walk<Epi, ITEMS> k(work, slot, slots); k.more() && ok; k.next(), ++n) {
        const int buf = n & 1;
        const bool ak = a_kmajor(k.item());
        const uint32_t idesc = ak ? ptx::idesc_bf16_f32(BM * CL, BN, false, !B_K)
                                  : ptx::idesc_bf16_f32(BM * CL, BN, true, !B_K);
        const Tile q = tile_of(k.item().p, k.t);
        if (!ptx::mbar_wait(tempty(buf), (((uint32_t)n >> 1) & 1u) ^ 1u)) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t dt = tmem + (uint32_t)(buf * BN);
        for (int kb = q.kb0; kb < q.kb1; ++kb) {
          if (!ptx::mbar_wait(full(stage), phase)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t sa = base + stage * C::STAGE, sb = sa + C::A_BYTES;
          const uint64_t ad0 = ak ? ptx::smem_desc_sw128(sa, 16, 1024) : ptx::smem_desc_sw128(sa, 8192, 1024);
          const uint64_t bd0 = B_K ? ptx::smem_desc_sw128(sb, 16, 1024) : ptx::smem_desc_sw128(sb, 8192, 1024);
#pragma unroll
          for (int kk = 0; kk < BKE / 16; ++kk) {
            const uint64_t ad = ad0 + (uint64_t)(ak ? 2 * kk : 128 * kk);
            const uint64_t bd = bd0 + (uint64_t)(B_K ? 2 * kk : 128 * kk);
            const uint32_t acc = (kb > q.kb0 || kk != 0) ? 1u : 0u;
            if (CL > 1)
              ptx::mma_bf16_pair(dt, ad, bd, idesc, acc);
            else
              ptx::mma_bf16(dt, ad, bd, idesc, acc);
          }
          if (CL > 1)
            ptx::mma_commit_pair_mc(empty(stage), MASK);
          else
            ptx::mma_commit(empty(stage));
          if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (CL > 1)
          ptx::mma_commit_pair_mc(tfull(buf), MASK);
        else
          ptx::mma_commit(tfull(buf));
      }
      // all MMAs issued by this thread are complete before TMEM is freed
      if (CL > 1)
        ptx::mma_commit_pair(drain);
      else
        ptx::mma_commit(drain);
      if (!ptx::mbar_wait(drain, 0)) ok = false;
      if (!ok) atomicExch(&g_core_error, 2);
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;  // of the lanes, of the columns
    typename Epi::Warp w;
    w.stg = gbase + C::EPI_OFF + (warp - 2) * Epi::STG;
    w.stg_s = base + C::EPI_OFF + (warp - 2) * Epi::STG;
    w.lane = lane;
    w.bars = wbars + 8u * (warp - 2) * Epi::WBARS;
    w.init();
    int n = 0;
    for (Walk<Epi, ITEMS> k(work, slot, slots); k.more(); k.next(), ++n) {
      const int buf = n & 1;
      const Problem& p = k.item().p;
      const typename Epi::Params& ep = k.item().ep;
      const Tile tl = tile_of(p, k.t);
      const int mw = tl.m0 + quarter * 32;
      w.template before<BN>(ep, p, mw, tl.n0, half);  // loads that do not wait for the accumulator
      // the decision is warp-uniform: tcgen05.ld is warp-collective
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(tfull(buf), ((uint32_t)n >> 1) & 1u))) {
        if (lane == 0) atomicExch(&g_core_error, 3);
        break;
      }
      ptx::tc_fence_after();
      const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * BN);
      if (mw < (Epi::PAD_ROWS ? (p.M + BM - 1) / BM * BM : p.M))
        w.template tile<BN>(ep, p, mw, tl.n0, half, tl.z, trow);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CL > 1)
          ptx::mbar_arrive_cluster(ptx::mapa(tempty(buf), 0));
        else
          ptx::mbar_arrive(tempty(buf));
      }
    }
    w.finish();
    if (lane == 0) ptx::bulk_wait0();  // stores performed before the CTA retires
  }
  ptx::tc_fence_before();
  __syncthreads();
  // the pair's MMAs and every cross-CTA arrival are complete before either CTA
  // frees TMEM or leaves
  if (CL > 1) ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    if (CL > 1)
      ptx::tmem_dealloc_pair(tmem, C::TMEM_COLS);
    else
      ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (CL > 1) ptx::cluster_sync();
}

// ---- epilogue helpers --------------------------------------------------------
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}

// Common state of an epilogue warp: its staging buffer and the store through it.
struct WarpBase {
  uint8_t* stg;
  uint32_t stg_s, bars;
  int lane;
  // hooks of an epilogue: set up; what a tile can do before its accumulator is
  // there; whatever it has in flight is waited for before the CTA leaves
  __device__ __forceinline__ void init() {}
  template <int BN, class Params>
  __device__ __forceinline__ void before(const Params&, const Problem&, int, int, int) {}
  __device__ __forceinline__ void finish() {}
  // One row of 128 bytes per lane (32 words w) goes to the swizzled staging
  // buffer at stg + off, then lane 0 stores the box at (x, y); the TMA unit
  // clips rows and columns beyond the matrix.
  __device__ __forceinline__ void stage_row(const uint32_t (&w)[32], int off = 0) {
    uint8_t* row = stg + off + lane * 128;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      *reinterpret_cast<uint4*>(row + ((u ^ (lane & 7)) << 4)) =
          make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
  }
  __device__ __forceinline__ void wait_free() {  // earlier stores have read the buffer
    if (lane == 0) ptx::bulk_wait_read0();
    __syncwarp();
  }
  __device__ __forceinline__ void store_box(const CUtensorMap* tm, int x, int y, int off = 0) {
    ptx::fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      ptx::tma_store_2d(tm, stg_s + off, x, y);
      ptx::bulk_commit();
    }
  }
  __device__ __forceinline__ void reduce_box(const CUtensorMap* tm, int x, int y) {
    ptx::fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      ptx::tma_reduce_add_2d(tm, stg_s, x, y);
      ptx::bulk_commit();
    }
  }
};

// ---- host side ---------------------------------------------------------------
// 2-D tensor map over a row-major [outer, inner] matrix with leading dimension
// ld (elements), box rows of 128 bytes with 128-byte swizzle or of 64 bytes with
// 64-byte swizzle, zero fill; false if it cannot be encoded.
inline bool tensor_map(CUtensorMap* out, const void* ptr, bool f32, uint64_t inner, uint64_t outer,
                       uint64_t ld, uint32_t box_inner, uint32_t box_outer) {
  typedef CUresult (*Fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                         const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                         CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                         CUtensorMapFloatOOBfill);
  static Fn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<Fn>(p);
  });
  if (!fn) return false;
  const cuuint64_t dims[2] = {inner, outer}, strides[1] = {ld * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {box_inner, box_outer}, estr[2] = {1, 1};
  return fn(out, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_inner * (f32 ? 4 : 2) == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int sm_count() {
  static std::atomic<int> cache[64];
  const int dev = current_device();
  int n = dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      return 2;  // no device: sizes can still be asked for
    if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}
inline int pair_count() { return std::max(1, sm_count() / 2); }

// Operands of one product.  A(m, k): A_K ? a[m * lda + k] : a[k * lda + m]; B
// likewise over N (DUAL: over b_off + N rows).
struct Operands {
  int M, N, K;
  const void* a;
  int64_t lda;
  const void* b;
  int64_t ldb;
  int b_off = 0;
  int splits = 1;
};

// K-slices per split, and the number of splits that leaves none empty.
inline int slices_per_split(int K, int* splits) {
  const int nkb = (K + BKE - 1) / BKE, kbs = (nkb + *splits - 1) / *splits;
  *splits = (nkb + kbs - 1) / kbs;
  return kbs;
}

// One product of a launch with BN-column tiles of CL CTAs.
template <class Epi, int BN, bool B_K, int CL>
bool make_item(Item<Epi>* it, const Operands& o, bool a_k, const typename Epi::Params& ep) {
  constexpr int TN = Epi::DUAL ? BN / 2 : BN;
  Problem& p = it->p;
  p.M = o.M;
  p.N = o.N;
  p.K = o.K;
  p.b_off = o.b_off;
  p.a_rows = a_k && CL == 1 ? std::min(BM, (o.M + 7) / 8 * 8) : BM;
  p.num_mp = ((o.M + BM - 1) / BM + CL - 1) / CL;
  p.num_n = (o.N + TN - 1) / TN;
  p.group = (int64_t)o.M * o.K * 2 > A_L2_BYTES ? std::min(GROUP_M, p.num_mp) : p.num_mp;
  p.splits = o.splits;
  p.kbs = slices_per_split(o.K, &p.splits);
  it->ep = ep;
  it->a_k = a_k;
  const uint64_t rows_b = (uint64_t)o.N + o.b_off;
  return (a_k ? tensor_map(&it->a, o.a, false, o.K, o.M, o.lda, BKE, p.a_rows)
              : tensor_map(&it->a, o.a, false, o.M, o.K, o.lda, 64, BKE)) &&
         (B_K ? tensor_map(&it->b, o.b, false, o.K, rows_b, o.ldb, BKE, BN / CL)
              : tensor_map(&it->b, o.b, false, rows_b, o.K, o.ldb, 64, BKE));
}

// A kernel's launch configuration and the CTAs (CL = 1) or CTA pairs of it that
// can be resident at once on the current device (per kernel: the statics belong to this one).
template <int BN, int CL, class Epi, auto kern>
cudaError_t prepare(cudaStream_t st, cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attrs,
                    int* slots) {
  using C = Cfg<BN, CL, Epi::STG, Epi::WBARS>;
  static DeviceOnce attr;
  const cudaError_t ea = attr.run([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (ea != cudaSuccess) return ea;
  *cfg = {};
  cfg->blockDim = dim3(NTHREADS);
  cfg->dynamicSmemBytes = C::SMEM;
  cfg->stream = st;
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = CL;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg->attrs = attrs;
  cfg->numAttrs = CL > 1 ? 2 : 1;
  static std::atomic<int> by_dev[64];
  const int dev = current_device();
  int n = dev < 64 ? by_dev[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    n = std::max(1, sm_count() / CL);
    if (CL > 1) {
      cudaLaunchConfig_t q = *cfg;
      q.gridDim = dim3(n * CL);
      q.attrs = attrs + 1;
      q.numAttrs = 1;
      int c = 0;
      if (cudaOccupancyMaxActiveClusters(&c, kern, &q) == cudaSuccess && c > 0 && c < n) n = c;
      cudaGetLastError();
    }
    if (dev < 64) by_dev[dev].store(n, std::memory_order_relaxed);
  }
  *slots = n;
  return cudaSuccess;
}

template <class Epi, int BN, bool A_K, bool B_K, int CL>
cudaError_t launch(const Operands& o, const typename Epi::Params& ep, cudaStream_t st) {
  Work<Epi, 1> w;
  if (!make_item<Epi, BN, B_K, CL>(&w.item[0], o, A_K, ep)) return cudaErrorInvalidValue;
  constexpr auto kern = gemm_core_kernel<Epi, BN, A_K ? 1 : 0, B_K, CL, 1>;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attrs[2];
  int slots;
  const cudaError_t e = prepare<BN, CL, Epi, kern>(st, &cfg, attrs, &slots);
  if (e != cudaSuccess) return e;
  const Problem& p = w.item[0].p;
  const int64_t tiles = (int64_t)p.num_mp * p.num_n * p.splits;
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  // no more CTAs than finish in the same number of tile rounds
  const int rounds = (int)((tiles + slots - 1) / slots);
  cfg.gridDim = dim3((unsigned)((tiles + rounds - 1) / rounds) * CL);
  ++g_launch_count;
  return cudaLaunchKernelEx(&cfg, kern, w);
}

// Several products with N-major B (BN = 256 CTA-pair tiles) in one launch.
struct Product {
  Operands o;
  bool a_k;
};
constexpr int64_t GROUP_BYTES = 256ll << 20;  // operands of the products, counted for each
constexpr int TILE_COST = 4;  // a tile's fixed cost in K-slices (fill, hand-over)

inline int64_t tiles256(int64_t M, int64_t N) {
  return (M + 2 * BM - 1) / (2 * BM) * ((N + 255) / 256);
}
inline int64_t operand_bytes(int64_t M, int64_t N, int64_t K) { return 2 * K * (M + N); }

// Splits of a long contraction of `tiles` tiles that shares a launch with other
// work (K-slices of tiles), so that none of its tiles is longer than the slots'
// even share.  (A quarter longer is cheaper than the partial sums.)
inline int even_splits(int64_t tiles, int K, int64_t other, int slots) {
  const int64_t slices = (K + BKE - 1) / BKE;
  const int64_t share = std::max<int64_t>(8, (tiles * slices + other) / slots);
  int splits = slices * 4 > share * 5 ? (int)std::min<int64_t>(16, (slices + share - 1) / share) : 1;
  slices_per_split(K, &splits);
  return splits;
}

// Deals `tiles` tiles of length `len` to the slots, least loaded first, and adds
// them to `load`; first[s] .. first[s + 1] are slot s's tiles.
inline void deal(int tiles, int len, int slots, int* load, uint16_t* first) {
  // the highest level (in K-slices) to which the slots can be filled
  int lo = *std::min_element(load, load + slots);
  int hi = *std::max_element(load, load + slots) + (tiles / slots + 1) * len;
  auto fits = [&](int level) {
    int n = 0;
    for (int s = 0; s < slots; ++s) n += std::max(0, level - load[s]) / len;
    return n;
  };
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (fits(mid) <= tiles)
      lo = mid;
    else
      hi = mid - 1;
  }
  int count[MAX_SLOTS], left = tiles - fits(lo);
  for (int s = 0; s < slots; ++s) {
    count[s] = std::max(0, lo - load[s]) / len;
    load[s] += count[s] * len;
  }
  while (left-- > 0) {
    int best = 0;
    for (int s = 1; s < slots; ++s)
      if (load[s] < load[best]) best = s;
    ++count[best];
    load[best] += len;
  }
  int at = 0;
  for (int s = 0; s < slots; ++s) {
    first[s] = (uint16_t)at;
    at += count[s];
  }
  first[slots] = (uint16_t)at;
}

// K-slices on the longest path of a product launched alone.
inline int64_t rounds_cost(int64_t tiles, int len, int slots) {
  return (tiles + slots - 1) / slots * len;
}

// One launch of the N products, their tiles dealt out, where that is better than one
// launch after the other by the K-slices on the longest path (*taken, else nothing is
// launched).
template <class Epi, int N>
cudaError_t launch_group(const Product* prod, const typename Epi::Params* ep, bool* taken,
                         cudaStream_t st) {
  constexpr auto kern = gemm_core_kernel<Epi, 256, 2, false, 2, N>;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attrs[2];
  int slots;
  *taken = false;
  const cudaError_t e = prepare<256, 2, Epi, kern>(st, &cfg, attrs, &slots);
  if (e != cudaSuccess) return e;
  if (slots > MAX_SLOTS) return cudaSuccess;
  // A slot's tiles of a product are neighbours, so the tiles in flight are spread
  // over the whole product: right while the operands stay in L2, else each is
  // streamed more than once.  Measured apart and together, operands counted for
  // each product: 192 MB 126 and 98 us, 134 MB 142 and 98, 493 MB 245 and 249,
  // 980 MB 4% slower together.
  int64_t bytes = 0;
  for (int i = 0; i < N; ++i)
    bytes += operand_bytes(prod[i].o.M, prod[i].o.N, prod[i].o.K);
  if (bytes > GROUP_BYTES) return cudaSuccess;
  // longest tiles first
  int order[N], len[N];
  int64_t tiles[N], apart = 0;
  for (int i = 0; i < N; ++i) {
    const Operands& o = prod[i].o;
    int splits = o.splits;
    len[i] = slices_per_split(o.K, &splits) + TILE_COST;
    tiles[i] = tiles256(o.M, o.N) * splits;
    if (tiles[i] > UINT16_MAX || tiles[i] * len[i] > INT32_MAX / 8) return cudaSuccess;
    apart += rounds_cost(tiles[i], len[i], slots) + 2 * TILE_COST;  // a launch more
    order[i] = i;
  }
  std::sort(order, order + N, [&](int a, int b) { return len[a] > len[b]; });
  Work<Epi, N> w;
  int load[MAX_SLOTS] = {};
  for (int k = 0; k < N; ++k) deal((int)tiles[order[k]], len[order[k]], slots, load, w.first[k]);
  const int together = *std::max_element(load, load + slots);
  if (together * 100ll > apart * 97ll) return cudaSuccess;
  for (int k = 0; k < N; ++k)
    if (!make_item<Epi, 256, false, 2>(&w.item[k], prod[order[k]].o, prod[order[k]].a_k, ep[order[k]]))
      return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)slots * 2);
  ++g_launch_count;
  *taken = true;
  return cudaLaunchKernelEx(&cfg, kern, w);
}

// Reads and clears this translation unit's error word (-1: unreadable).
static inline int read_and_clear_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_core_error, sizeof(int)) != cudaSuccess) return -1;
  if (v) cudaMemcpyToSymbol(g_core_error, &z, sizeof(int));
  return v;
}

}  // namespace core
}  // namespace oases
