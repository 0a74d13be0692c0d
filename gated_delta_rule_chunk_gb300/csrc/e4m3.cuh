// Conversions of the 8-bit cache (e4m3: 4 significant bits, exponents -6 to 8, subnormals, NaN,
// no infinity), two elements at a time.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <stdint.h>

namespace gdn {

// Two finite elements of at most 448 in size (low byte first), rounded to nearest even.
__device__ __forceinline__ uint32_t finite_to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// The same for any elements: infinities and NaN become NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  a = fabsf(a) <= 3.402823466e38f ? a : NAN;
  b = fabsf(b) <= 3.402823466e38f ? b : NAN;
  return finite_to_e4m3x2(a, b);
}

// Four bytes as two pairs of fp16 values (exact). (Through cuda_fp8.h's types the halves of a
// pair were taken apart and put together again, an instruction or two each.)
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
// The two low bytes.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t x) {
  uint32_t lo, hi;
  e4m3x4_to_f16x4(x & 0xFFFFu, lo, hi);
  return __half22float2(*reinterpret_cast<const __half2*>(&lo));
}

}  // namespace gdn
