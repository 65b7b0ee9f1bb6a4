// Attention over keys of another length on the 5th-generation tensor cores: what the
// forward and the backward kernels share.  Head sizes up to 64 run with DP = 64 columns
// per tile, larger ones with DP = 128; TMA fills the columns behind the head size and
// the rows behind a sequence with zeros.
#pragma once

#include <cuda.h>

#include <mutex>

#include "sm100_ptx.cuh"
#include "xattn.cuh"

namespace oases {
namespace xattn {

constexpr int BOX = 128 * 64 * 2;  // one TMA box: 128 rows x 64 bf16
template <int DP>
constexpr int tile_bytes() { return DP / 64 * BOX; }  // 128 rows x DP

// 2^x on the hardware unit (relative error ~2^-22); results below the normal range,
// including 2^-inf for hidden keys, are flushed to 0.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Shared-memory descriptors, formed once per tile and stepped in 16-byte units (every
// shared address is below 2^18, so a step cannot carry out of the address field).
__device__ __forceinline__ uint64_t desc_step(uint64_t base_desc, uint32_t byte_off) {
  return base_desc + (uint64_t)(byte_off >> 4);
}
// K-major operand [rows][DP], 64 columns per box of `box` bytes, k-step kk of DP / 16.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t tile, int kk, uint32_t box = BOX) {
  return desc_step(ptx::smem_desc_sw128(tile, 16, 1024), (uint32_t)(kk >> 2) * box + (uint32_t)(kk & 3) * 32);
}
// MN-major operand [k rows][DP columns], k-step kk of 16 rows.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t tile, int kk, uint32_t box = BOX) {
  return desc_step(ptx::smem_desc_sw128(tile, box, 1024), (uint32_t)kk * 2048);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int x, int row,
                                            int head, int batch) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(row), "r"(head), "r"(batch)
      : "memory");
}
// ROWS rows of a head, DP columns, into consecutive boxes of 64 columns.
template <int DP, int ROWS>
__device__ __forceinline__ void load_tile(uint32_t dst, const void* tmap, uint32_t bar, int row, int head,
                                          int batch) {
#pragma unroll
  for (int c = 0; c < DP / 64; ++c) tma_load_4d(dst + c * ROWS * 128, tmap, bar, 64 * c, row, head, batch);
}

// Registers of a warpgroup's threads, given up or taken over from those that gave up theirs.
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Item k of CTA c (of G) in a persistent kernel whose items are numbered heaviest
// first: rounds of G items, in snake order.
__device__ __forceinline__ int persistent_item(int k, int c, int G) {
  return k * G + ((k & 1) ? G - 1 - c : c);
}

// Ragged sequences (up to MAX_ORDER of them) by falling number of keys, so that items of
// falling size are dealt out and those without keys come last: order[place] is the
// sequence, tiles[place] how many tiles of 128 keys the sequences before it have
// (tiles[batch]: all).  By all of a CTA's threads, MAX_ORDER at least, before it loads
// anything to shared memory; `lens` is scratch, `tiles` o->tiles or scratch too.  8 sequences of up to 1531 keys, 16 heads of
// 64, forward and backward: 149 -> 142 us.
constexpr int MAX_ORDER = 256;
struct Order {
  uint8_t order[MAX_ORDER];
  int tiles[MAX_ORDER + 4];
};
__device__ __forceinline__ bool ragged(const Args& a) { return a.kv_lens != nullptr && a.B > 1 && a.B <= MAX_ORDER; }
__device__ __forceinline__ void order_sequences(const Args& a, int* lens, Order* o, int* tiles) {
  const int t = threadIdx.x;
  if (t < a.B) lens[t] = a.len(t);
  __syncthreads();
  if (t < a.B) {
    const int mine = lens[t];
    int place = 0, before = 0, all = 0;
    for (int x = 0; x < a.B; ++x) {
      const int n = (lens[x] + 127) / 128;
      const bool first = lens[x] > mine || (lens[x] == mine && x < t);
      place += first;
      before += first ? n : 0;
      all += n;
    }
    o->order[place] = (uint8_t)t;
    tiles[place] = before;
    if (place == 0) tiles[a.B] = all;
  }
  ptx::fence_async_smem();  // (TMA writes over `lens` next)
  __syncthreads();
}
// Item r of batch x tiles in the order of their work: causal by falling tile (the last
// queries see the most keys), otherwise sequence by sequence.
__device__ __forceinline__ void query_item(const Args& a, const Order* o, int r, int tiles, int* tile, int* b) {
  const int place = a.causal ? r % a.B : r / tiles;
  *tile = a.causal ? tiles - 1 - r / a.B : r % tiles;
  *b = ragged(a) ? o->order[place] : place;
}
// ... of key tiles: causal by rising tile (the first keys are seen by the most queries),
// otherwise the tiles that hold keys, sequence by sequence, then the others.
__device__ __forceinline__ void key_item(const Args& a, const Order* o, int r, int tiles, int* tile, int* b) {
  if (a.causal || !ragged(a)) {
    const int place = r % a.B;
    *tile = r / a.B;
    *b = ragged(a) ? o->order[place] : place;
    return;
  }
  const int full = o->tiles[a.B];
  const bool held = r < full;
  const int x = held ? r : r - full;
  int lo = 0, hi = a.B;  // the last place whose tiles begin at or before x
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2, first = held ? o->tiles[mid] : mid * tiles - o->tiles[mid];
    if (first <= x) lo = mid;
    else hi = mid;
  }
  const int first = held ? o->tiles[lo] : lo * tiles - o->tiles[lo];
  *tile = (held ? 0 : o->tiles[lo + 1] - o->tiles[lo]) + x - first;
  *b = o->order[lo];
}

// ---- host ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}
// Tensor map over [batch, tokens, heads, D] bf16 with strides of its own: boxes of `rows`
// tokens x 64 values of one head, 128-byte swizzle, zero fill outside.
inline cudaError_t map4d(CUtensorMap* m, const void* p, const Strides& s, int D, int tokens, int heads,
                         int batch, int rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)tokens, (cuuint64_t)heads, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {(cuuint64_t)s.s * 2, (cuuint64_t)s.h * 2, (cuuint64_t)s.b * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}
}  // namespace xattn
}  // namespace oases
