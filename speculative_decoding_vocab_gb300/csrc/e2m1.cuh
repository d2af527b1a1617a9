// e2m1.cuh -- the 4-bit cache's number format: e2m1 codes (sign, two exponent
// bits, one fraction bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) and the scale
// bytes, 2^(b - 127) per 32 elements of a token and head, 255 for NaN.
#pragma once

#include "common.cuh"

namespace ssd {

constexpr int kQ4Group = 32;
// Scale bytes that the append writes: 2^-100 .. 2^125.  Above, 6 scale passes fp32's range;
// below, v counts as 0 in the attention (its sums reach 2^108 a key where all of a
// row's v scales are this small).
constexpr int kMinScaleByte = 27, kMaxScaleByte = 252, kNanScaleByte = 255;

// eight fp32 -> eight codes (nearest even, clamped to +-6): f[2 j] in the low half of byte j
SSD_DEV uint32_t e2m1_pack8(const float *f) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
// eight codes -> four pairs of halves (exact), byte j -> h[j], its low code in the low half
SSD_DEV void e2m1_halves8(uint32_t w, uint32_t *h) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// scale byte -> its value (2^-127 is subnormal, 255 NaN)
SSD_DEV float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : (b == 255 ? 0x7fc00000u : b << 23));
}
// the scale byte of a group whose largest magnitude has these bf16 bits: 6 * 2^e = 1.5 * 2^(e + 2), so the exponent - 2,
// one more where the fraction is above a half (0x40)
SSD_DEV uint32_t e8m0_of(uint32_t bits) {
  return static_cast<uint32_t>(min(max(static_cast<int>((bits + 0x3Fu) >> 7) - 2, kMinScaleByte), kMaxScaleByte));
}

}  // namespace ssd
