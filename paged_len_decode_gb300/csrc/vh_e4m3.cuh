// vh_e4m3.cuh -- 8-bit values with a scale: what the append writes and the
// attention and the read-back take.
#pragma once

#include "vh_common.cuh"

namespace vh {

constexpr float kE4m3Max = 448.f;               // the largest e4m3 value
constexpr float kScaleMin = 1.17549435e-38f;    // 2^-126: the least scale, so that 1 / s is finite

// Two values rounded to nearest even, the first in the low byte; beyond 448 they become 448 (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 values (the low byte first) as two fp16 ones, which hold them exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
// The same of the upper two bytes.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

}  // namespace vh
