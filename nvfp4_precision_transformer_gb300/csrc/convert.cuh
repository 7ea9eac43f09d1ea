// Conversions shared by the kernels that write 8-bit outputs: the hardware casts to FP8
// (round-to-nearest-even, satfinite) and the shared exponent of an MXFP8 block.
#pragma once

#include <stdint.h>

namespace te {
namespace {

[[maybe_unused]] __device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
[[maybe_unused]] __device__ __forceinline__ uint32_t cvt_e5m2x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// Shared exponent of an MXFP8 block: clamp(floor(log2 amax) - 8, -127, 127); -127 for a zero block.
[[maybe_unused]] __device__ __forceinline__ int mx_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0) return -127;
  const uint32_t ef = b >> 23;
  int e = (ef == 0) ? (31 - __clz(static_cast<int>(b))) - 149 : static_cast<int>(ef) - 127;
  e -= 8;
  return max(-127, min(127, e));
}
[[maybe_unused]] __device__ __forceinline__ float mx_mult(int E) {
  return __uint_as_float(static_cast<uint32_t>(127 - E) << 23);
}

}  // namespace
}  // namespace te
