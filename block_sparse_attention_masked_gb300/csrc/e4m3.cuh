// Eight-bit rows of a paged cache: e4m3 codes with one power of two for each row
// (token, key/value head), kept as a byte e: the row's values are code * 2^(e - 127).
// A power of two loses nothing where a code is formed or read back: the only rounding
// is the code's own (2^-4 of a value at most, or 2^-10 of the row's power), and the row
// read back as bf16 is exact.  It is the least one that leaves no value above e4m3's
// 448 = 1.75 * 2^8, e >= 0.  A row with an infinite or NaN value is NaN throughout:
// byte 255, codes 0x7f.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mattn {
namespace e4m3 {

// A row's exponent byte from the bits of its largest |value| in bf16.
__host__ __device__ constexpr int row_exponent(uint32_t top) {
  const int e = (int)(top >> 7), m = (int)(top & 127u);
  if (e == 255) return 255;
  const int x = e - 8 + (m > 96 ? 1 : 0);  // (96 / 128: the fraction of 1.75)
  return x > 0 ? x : 0;
}

// 2^(e - 127); 255: NaN.
__device__ __forceinline__ float power(int e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7fffffffu : (uint32_t)e << 23);
}
// 2^(127 - e), the factor that takes a row's values to its codes (e <= 248); 255: NaN.
__device__ __forceinline__ float inverse(int e) {
  return __uint_as_float(e == 255 ? 0x7fffffffu : (uint32_t)(254 - e) << 23);
}

// Two values, rounded to nearest even (none is above 448; NaN gives 0x7f).
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes as f16, exactly.
__device__ __forceinline__ uint32_t to_half2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(r)
      : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t to_half2_hi(uint32_t four) {  // codes 2 and 3 of four
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(four));
  return r;
}

}  // namespace e4m3
}  // namespace mattn
