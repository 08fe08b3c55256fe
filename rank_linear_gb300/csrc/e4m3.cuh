// e4m3.cuh -- e4m3 with power-of-two scales, as the fp8 layers take it.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

namespace lora {
namespace {

// The scale of a block with absolute maximum a > 0 is 2^e, e the smallest
// integer with a <= 448 * 2^e (448 = 0.875 * 2^9, the largest e4m3 value);
// a = 0 gives 2^0.  Dividing by it is exact, so the one rounding is the
// conversion to e4m3 (nearest, ties to even, saturating).
__device__ __forceinline__ int pow2_exponent(float a) {
  if (!(a > 0.f)) return 0;
  int k;
  const float m = frexpf(a, &k);  // a = m 2^k, m in [0.5, 1)
  return m <= 0.875f ? k - 9 : k - 8;
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}
// Two at once: f.x in the low byte, f.y in the high byte (one conversion
// instruction, the same rounding as to_e4m3).
__device__ __forceinline__ uint32_t to_e4m3x2(float2 f) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3));
}

}  // namespace
}  // namespace lora
