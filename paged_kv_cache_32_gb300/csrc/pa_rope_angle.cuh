// pa_rope_angle.cuh - angles of rotary positions, reduced to a fraction of a turn in fixed point (see pa_rope.cu).
#pragma once

#include <stdint.h>

namespace pa {

// f / 2 pi as a fraction of a turn in units of 2^-64 (whole turns per position drop out)
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  const double t = f * 0.15915494309189533577;  // 1 / 2 pi
  const double frac = t - floor(t);             // [0, 1]
  const unsigned long long hi = (unsigned long long)(frac * 4294967296.0);  // < 2^33: wraps below
  const double rest = frac * 4294967296.0 - (double)hi;
  return (hi << 32) + (unsigned long long)(rest * 4294967296.0);
}

// (cos, sin) of position times that fraction, times magnitude
__device__ __forceinline__ float2 turn_of(unsigned long long fraction, long long position, float magnitude) {
  const long long turns = (long long)(fraction * (unsigned long long)position);
  float s, c;
  sincospif(__ll2float_rn(turns) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns in [-1, 1]
  return make_float2(c * magnitude, s * magnitude);
}

// A pair turned by c = (cos, sin).  Which products are rounded is written out: left to the compiler, kernels differ in
// the last place of some elements, and rows held in 4 bits from the same rows turned over a 16-bit cache.
__device__ __forceinline__ void turn_pair(float2 c, float& x0, float& x1) {
  const float y0 = fmaf(c.x, x0, -__fmul_rn(c.y, x1)), y1 = fmaf(c.x, x1, __fmul_rn(c.y, x0));
  x0 = y0, x1 = y1;
}

}  // namespace pa
