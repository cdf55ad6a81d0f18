// pfa_q4.cuh -- device helpers of the operators around the 4-bit cache: e2m1 and e4m3
// conversions, the quantisation of 16 channels.
#pragma once
#include "pfa_q8.cuh"

namespace pfa {

// Two e2m1 codes, byte I of a word -> a half pair (exact).
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_half(uint32_t w) {
  uint32_t h;
  if constexpr (I == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
        : "=r"(h) : "r"(w));
  else if constexpr (I == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
        : "=r"(h) : "r"(w));
  else if constexpr (I == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}"
        : "=r"(h) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}"
        : "=r"(h) : "r"(w));
  return h;
}

// Two e4m3 values, the low half of a word -> a half pair (exact, NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_half(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ float e4m3_to_float(uint8_t c) {
  const uint32_t h = e4m3x2_to_half(c);
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// The nearest e4m3 of x >= 0, ties to even, 448 beyond it.
__device__ __forceinline__ uint8_t float_to_e4m3(float x) {
  uint16_t w;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w) : "f"(0.f), "f"(x));
  return (uint8_t)w;
}

// Eight floats -> eight e2m1 codes, nearest with ties to even, +-6 beyond them.
__device__ __forceinline__ uint32_t float_to_e2m1x8(const float* f) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}

__device__ __forceinline__ float pow2(int e) {   // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

}  // namespace pfa
