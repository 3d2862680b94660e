// Numbers of the 8-bit cache: e4m3 (4 exponent and 3 fraction bits, no
// infinities, the largest 448) times a power of two 2^e for each block of rows,
// kept as e8m0 (the byte e + 127; 255 is NaN).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace blkattn {

// 2^i, i in [-127, 127] (others: the nearer end); 2^-127 is subnormal.
__device__ __forceinline__ float pow2(int i) {
  i = min(max(i, -127), 127);
  return __uint_as_float(i > -127 ? (uint32_t)(i + 127) << 23 : 0x00400000u);
}
// The scale that a byte stands for.
__device__ __forceinline__ float scale_of(int byte) {
  return byte == 255 ? __uint_as_float(0x7fc00000u) : pow2(byte - 127);
}

// The least e with amax <= 448 2^e (448 = 1.75 2^8), at least -127.  A power of
// two, not amax / 448: a number's relative error does not change by it, and a
// block whose scale rises is rounded again exactly but for its smallest
// numbers, so rows do not wear out as neighbours are appended.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);  // finite, not negative
  return max((int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0), -127);
}

// Two floats as e4m3 (rounded to nearest, ties to even; lo in the low byte).
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 as f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}
// Four e4m3 of a word as f16: the lower two, the upper two.
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float2 e4m3x2_to_f2(uint32_t w) {
  const uint32_t h = e4m3x2_to_h2(w);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace blkattn
