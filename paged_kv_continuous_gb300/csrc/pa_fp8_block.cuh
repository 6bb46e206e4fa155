// The block-scaled FP8 cache: E4M3 codes with one power-of-two scale for each
// (16-token block, kv head), K and V apart, held as a biased exponent in one
// byte: value = code * 2^(byte - 127).  A power of two, because E4M3 is a
// floating-point format: its relative precision does not depend on where a
// block's scale sits, while a power of two makes the scaling exact, lets a
// block be re-coded to a larger scale without error (subnormals aside), and
// lets the readers fold it into an exponent or an accumulator exactly.
#pragma once

#include "pa_common.cuh"

namespace pa {

constexpr int kScaleBias = 127;
// Exponents a scale may take, -40 .. 40.  The span bounds how far the scales
// of two blocks of one sequence can lie apart (2^80), so the attention
// kernels can keep one running reference per row for weight times V scale
// without losing a weight to underflow: a weight 2^-46 of the largest still
// counts in the softmax sum when its block's V scale is the smallest and
// another's the largest.  Values stay representable from 2^-49 to 448 * 2^40.
constexpr int kScaleMin = kScaleBias - 40, kScaleMax = kScaleBias + 40;

// The readers clamp the scale bytes of four heads at once to that span, so
// that a byte never stored by the library cannot overflow their arithmetic.
__device__ __forceinline__ uint32_t clamp_scales4(uint32_t w) {
  constexpr uint32_t lo = 0x01010101u * kScaleMin, hi = 0x01010101u * kScaleMax;
  return __vminu4(__vmaxu4(w, lo), hi);
}

__device__ __forceinline__ float scale_of(int byte) {  // 2^(byte - 127), 1 <= byte <= 254
  return __uint_as_float((uint32_t)byte << 23);
}
__device__ __forceinline__ float inv_scale_of(int byte) {  // 2^(127 - byte)
  return __uint_as_float((uint32_t)(2 * kScaleBias - byte) << 23);
}

// Smallest exponent e with a <= 448 * 2^e, as a clamped byte; a >= 0 and
// finite (0: the smallest scale).  448 = 1.75 * 2^8, so with a = m * 2^x,
// 1 <= m < 2, e = x - 8, or one more when m > 1.75.
__device__ __forceinline__ int scale_for(float a) {
  const uint32_t u = __float_as_uint(a);
  const int byte = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(byte, kScaleMin), kScaleMax);
}

// Two floats to two E4M3 codes (lo in the low byte): nearest even, magnitudes
// past the largest finite value (448) saturated to it, NaN to the NaN code.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes times a power of two f <= 1, coded again.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float f) {
  uint32_t out = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p;  // two f16 values, exact
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p) : "h"((unsigned short)(w >> (16 * h))));
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\t"
        "cvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(p));
    out |= e4m3x2_of(lo * f, hi * f) << (16 * h);
  }
  return out;
}

}  // namespace pa
