// e4m3 codes with a scale per block of 128: shared device helpers.
#pragma once

#include <float.h>

#include <type_traits>

#include "common.cuh"

namespace moe {
namespace fp8 {

constexpr int kBlock = 128;             // elements per scale
constexpr float kMaxCode = 448.0f;      // the largest e4m3 value
// Groups whose largest magnitude is below 2^-100 take that magnitude's scale,
// so that neither the scale nor its reciprocal leaves the normal fp32 range
// (an all-zero group gets zero codes).
constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100

// |v| where v is finite, else 0: infinities and NaN take no part in a scale
__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= FLT_MAX ? a : 0.f;
}

// scale = amax / 448, and the factor its codes are made with, 448 / amax
// (both IEEE divisions: one pair per 128 elements)
__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax, kTiny) / kMaxCode; }
__device__ __forceinline__ float rscale_of(float amax) { return kMaxCode / fmaxf(amax, kTiny); }

// what is rounded to a code: v times the group's factor, NaN for a value
// that is not finite (its code is NaN, so it shows in every product)
__device__ __forceinline__ float code_arg(float v, float r) {
  return fabsf(v) <= FLT_MAX ? v * r : __int_as_float(0x7fffffff);
}

// four floats to four e4m3 codes, the first in the low byte; round to
// nearest even. The arguments are at most 448 (1 + 2^-23) in magnitude.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ uint8_t e4m3x1(float a) { return (uint8_t)e4m3x4(a, 0.f, 0.f, 0.f); }

}  // namespace fp8
}  // namespace moe
