// pa_fp8.cuh - E4M3 codes as fp16 values.
#pragma once

#include <stdint.h>

namespace pa {

// four E4M3 codes (bytes 0..3 of r) -> two f16x2, exact: lo = (byte 0, byte 1), hi = (byte 2, byte 3)
__device__ __forceinline__ void codes_to_half(uint32_t r, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(r));
}

}  // namespace pa
