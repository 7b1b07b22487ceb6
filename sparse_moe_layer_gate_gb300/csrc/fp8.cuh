// e4m3 conversions and block scales shared by the FP8 kernels.
#pragma once

#include "common.cuh"

namespace epoch {

constexpr int kFp8Block = 128;  // columns (and, for weights, rows) that share a scale

// Scale of a block whose largest |x| has bit pattern m: max(|x| / 448, 2^-126).
// NaN patterns pass through (the comparison is false for them).
__device__ __forceinline__ float fp8_scale(unsigned m) {
  const float s = __uint_as_float(m) / 448.0f;
  return s < 1.17549435e-38f ? 1.17549435e-38f : s;
}

// Four values to e4m3 (round to nearest even, out of range to the largest
// finite value, NaN to NaN), the first in the lowest byte.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

}  // namespace epoch
