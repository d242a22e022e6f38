// pa_fp4.cuh - rows held in 4 bits: 16 neighbouring elements share an E4M3 scale, each is an E2M1 code.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "pa_fp4.h"

namespace pa {

// eight E2M1 codes (nibbles of x from the lowest on) -> four f16x2, in order, exact
__device__ __forceinline__ void fp4_to_half(uint32_t x, uint32_t& h0, uint32_t& h1, uint32_t& h2, uint32_t& h3) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
      : "r"(x));
}
// two E4M3 codes (the low 16 bits) -> f16x2, exact
__device__ __forceinline__ uint32_t fp4_scales_to_half(uint32_t x) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(x));
  return h;
}
__device__ __forceinline__ uint32_t half_dup_lo(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t half_dup_hi(uint32_t x) { return __byte_perm(x, x, 0x3232); }
// An E2M1 number (2 significant bits) times an E4M3 one (4) is exact in fp16: 6 bits, multiples of 2^-10 up to 2688.
__device__ __forceinline__ uint32_t half_mul(uint32_t a, uint32_t b) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// The scale's code of a group whose largest magnitude is amax (unit6 = 6 unit, rounded to fp32): amax / unit6 to the
// nearest E4M3 number, ties to even, at most 448.
__device__ __forceinline__ uint32_t fp4_scale_code(float amax, float unit6) {
  return __nv_cvt_float_to_fp8(__fdiv_rn(amax, unit6), __NV_SATFINITE, __NV_E4M3);
}
// What the group's elements are multiplied with before they are rounded to E2M1: 1 / (scale unit), or 0 for a scale of 0.
__device__ __forceinline__ float fp4_inverse(uint32_t code, float unit) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
  const float t = __fmul_rn(__half2float(__half(h)), unit);
  return t > 0.f ? __fdiv_rn(1.f, t) : 0.f;
}
// The codes of eight elements times inv, the first in the lowest nibble; ties to even, magnitudes past 6 (infinities
// too) become 6.
__device__ __forceinline__ uint32_t fp4_codes8(const float (&x)[8], float inv) {
  uint32_t y;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(y)
      : "f"(__fmul_rn(x[0], inv)), "f"(__fmul_rn(x[1], inv)), "f"(__fmul_rn(x[2], inv)), "f"(__fmul_rn(x[3], inv)),
        "f"(__fmul_rn(x[4], inv)), "f"(__fmul_rn(x[5], inv)), "f"(__fmul_rn(x[6], inv)), "f"(__fmul_rn(x[7], inv)));
  return y;
}

// Softmax weights over these caches enter the value product as one fp16 number each, off by at most 2^-11 of itself
// (2^-12 on average, in either direction): less than what the output's rounding takes (fp16 2^-11, bf16 2^-8), where a
// second term would double the product's MMAs.  Their range is what has to be looked after: against a reference maximum
// that no score exceeds by more than 2^8, plain weights reach down to 2^-25 only, and a long context's many small ones
// would vanish beside one large (a first token that takes nearly everything: of 2^20 tokens of 2^-25.5 each 2 %).  So they
// are 2^(7 + s - m), at most 2^15, and what vanishes lies below 2^-32 of the largest; the factor drops out with the sum.
constexpr float kFp4WeightShift = 7.f;

// A bf16 query row whose largest magnitude is mx becomes fp16 after a multiplication by `down`, a power of two that brings
// mx into [1, 2) (mx subnormal: below); `up` is its inverse.  1 for a row with an infinity.  (Callers' fmaxf
// passes over NaNs: they do not choose the power, and stay NaN whatever it is.)
__device__ __forceinline__ void row_power(float mx, float& up, float& down) {
  const int e = mx < INFINITY ? max((int)(__float_as_uint(mx) >> 23), 1) : 127;
  up = __uint_as_float((uint32_t)e << 23);
  // 2^(127 - e); 2^-127, for an element past 2^127, has no normal fp32 form
  down = e < 254 ? __uint_as_float((uint32_t)(254 - e) << 23) : 5.877471754111438e-39f;
}

// A row's place in a cache: its 64 bytes of codes, and its 8 bytes of scales `kFp4CodeBytes` and so on behind the tile.
__host__ __device__ __forceinline__ size_t fp4_tile(int64_t block, int num_kv_heads, int head, int block_size, int off) {
  return (((size_t)block * num_kv_heads + head) * (block_size / kFp4Tokens) + off / kFp4Tokens) * kFp4TileBytes;
}

}  // namespace pa
