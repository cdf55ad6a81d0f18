// pfa_q8.cuh -- device helpers of the operators around the 8-bit cache: e4m3
// conversions, the block scale, division by numbers that the host knows.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace pfa {

// Division of 0 <= n < 2^31 by a number that the host knows: a 64-bit product and a
// shift, where / takes some thirty instructions (the kernels' code is mostly run
// once a launch, and fetching it is a good part of their start).
struct Divisor {
  uint32_t by, m;
  int shift;
};
inline Divisor divisor(uint32_t by) {
  int s = 0;
  while ((1u << s) < by) ++s;
  return Divisor{by, (uint32_t)(((uint64_t)1 << (31 + s)) / by + 1), 31 + s};
}
__device__ __forceinline__ int operator/(int n, const Divisor& d) {
  return (int)(((uint64_t)(uint32_t)n * d.m) >> d.shift);
}

// Four e4m3 codes of a word -> two half pairs; every e4m3 value (NaN among
// them) is exact in half.
__device__ __forceinline__ void e4m3x4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float* f) {
  uint32_t lo, hi;
  e4m3x4_to_half(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// Four floats -> four e4m3 codes, nearest with ties to even.  e4m3 has no
// infinity: the conversion would turn one into 448, so it becomes NaN first.
__device__ __forceinline__ uint32_t float_to_e4m3x4(float a, float b, float c, float d) {
  auto f = [](float x) { return fabsf(x) <= 3.402823466e38f ? x : __int_as_float(0x7fffffff); };
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w) : "f"(f(a)), "f"(f(b)), "f"(f(c)), "f"(f(d)));
  return w;
}

// The scale of a block whose largest finite magnitude is amax: the smallest
// power of two s >= 2^-126 with amax / s <= 448 = 1.75 * 2^8; 0 for amax 0.
// A power of two costs e4m3 no precision (its values are floating) and makes a
// later, larger scale re-express the codes that are there without another
// rounding, but for those that fall below the smallest normal value.
__device__ __forceinline__ float pow2_scale(float amax) {
  if (amax == 0.f) return 0.f;
  const uint32_t bits = __float_as_uint(amax);
  int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < 1 ? 1 : e;
  return __uint_as_float((uint32_t)e << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;  // NaN and infinity take no part in a scale
}

// Eight floats -> eight consecutive bf16 (16-byte aligned).
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace pfa
