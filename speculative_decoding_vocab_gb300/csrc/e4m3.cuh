// e4m3.cuh -- the 8-bit cache's number format: e4m3 codes (largest value 448,
// no infinities, 0x7F / 0xFF NaN) and the block scales.
#pragma once

#include "common.cuh"

namespace ssd {

constexpr float kE4m3Max = 448.f;
// Block scales below this are not written, and count as 0 in values: where all of
// a row's v scales are this small the attention's sums reach 2^108 a key, which
// leaves 2^19 keys of room in fp32's range.
constexpr float kMinBlockScale = 0x1p-100f;

// two fp32 -> two codes (nearest even, clamped to +-448; NaN -> 0x7F): lo in the low byte
SSD_DEV uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two codes -> two halves (exact)
SSD_DEV uint32_t e4m3_to_half2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
SSD_DEV void half2_to_float(uint32_t h, float &lo, float &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}
SSD_DEV void e4m3_unpack4(uint32_t w, float *f) {
  half2_to_float(e4m3_to_half2(static_cast<uint16_t>(w & 0xFFFFu)), f[0], f[1]);
  half2_to_float(e4m3_to_half2(static_cast<uint16_t>(w >> 16)), f[2], f[3]);
}
// a block scale a cache may hold: finite and not negative
SSD_DEV bool good_scale(float s) { return s >= 0.f && s <= 3.402823466e38f; }

}  // namespace ssd
