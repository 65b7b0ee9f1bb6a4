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

// Item k of CTA c (of G) in a persistent kernel whose items are numbered heaviest
// first: rounds of G items, in snake order.
__device__ __forceinline__ int persistent_item(int k, int c, int G) {
  return k * G + ((k & 1) ? G - 1 - c : c);
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
