// Conversions of the 8-bit cache (e4m3: 4 significant bits, exponents -6 to 8, subnormals, NaN,
// no infinity), two elements at a time.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <stdint.h>

namespace gdn {

// Two elements (low byte first), rounded to nearest even; infinities and NaN become NaN. The
// scale keeps finite values within 448.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  a = fabsf(a) <= 3.402823466e38f ? a : NAN;
  b = fabsf(b) <= 3.402823466e38f ? b : NAN;
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// The two low bytes as fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)x, __NV_E4M3);
  return (uint32_t)h.x | (uint32_t)h.y << 16;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t x) {
  const uint32_t h = e4m3x2_to_f16x2(x);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace gdn
