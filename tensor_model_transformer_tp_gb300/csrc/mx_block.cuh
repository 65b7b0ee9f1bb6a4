// One block of the MX-FP8 format: scale exponent, E4M3 conversion and the place
// of its scale byte in the 512-byte tiles (128 rows x 4 blocks).
#pragma once
#include <stdint.h>

#include "common.cuh"

namespace oases {

constexpr int MXB = 32;  // elements per scale block

// floor(log2(m)) of a finite m > 0, subnormals included.
__device__ __forceinline__ int floor_log2(float m) {
  const uint32_t b = __float_as_uint(m);
  const int ex = (int)(b >> 23);
  if (ex > 0) return ex - 127;
  return (31 - __clz((int)(b & 0x7FFFFFu))) - 149;
}

// Scale exponent of a block with maximum magnitude amax (0 for amax = 0).
__device__ __forceinline__ int block_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  return max(-127, min(127, floor_log2(amax) - 8));
}

// 2^-xe as an fp32 (xe in [-127, 126]: always a normal number).
__device__ __forceinline__ float pow2_neg(int xe) { return __int_as_float((127 - xe) << 23); }

// 2^(s - 127) of a scale byte s < 255 (s = 0: the subnormal 2^-127).
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s ? s << 23 : 0x00400000u);
}

// Two E4M3 codes, a at the lower address.
__device__ __forceinline__ uint16_t e4m3x2(float a, float b) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
  return d;
}

// The values of two E4M3 codes (exact), the lower address first.
__device__ __forceinline__ float2 e4m3x2_values(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  float2 f;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Byte of the scale of row r, block j in tiles of `kgroups` groups per row block.
__device__ __forceinline__ int64_t sf_offset(int r, int j, int kgroups) {
  return ((int64_t)(r / 128) * kgroups + j / 4) * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4 + (j % 4);
}

}  // namespace oases
