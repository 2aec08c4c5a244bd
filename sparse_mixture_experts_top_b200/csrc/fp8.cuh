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

// act(g) * u of the gate|up products. The tanh form of GELU as
//   0.5 g (1 + tanh z) = g / (1 + exp(-2z)),  z = sqrt(2/pi) (g + 0.044715 g^3),
// since 1 + tanh z cancels for a negative gate: in fp32 it is off by up to 2e-5 at
// g = -3, 1.5e-3 at -4 and half at -5, and zero from -5.5 down. A 16-bit h hides
// that below its own last place; a block of codes does not, whose scale follows
// its largest magnitude down to 2^-100. (It is also the shorter one: gate|up of
// 20,480 rows over 512 experts 210 against 222 us on one B200.) The error relative
// to the result is below (8 + 3.2 |2z|) 2^-23: the argument's roundings (4 |2z| of
// 2^-24) and the fast exponential's 2 + 1.16 |2z|. Past 2z = -87 (g below -9.4) the
// result is zero.
__device__ __forceinline__ float glu_codes(int act, float g, float u) {
  if (act == MOE_ACT_GEGLU_TANH) {
    const float m2z = -1.5957691216057308f * fmaf(0.044715f * g, g * g, g);
    return __fdividef(g, 1.0f + __expf(m2z)) * u;
  }
  return swiglu(g, u);
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
