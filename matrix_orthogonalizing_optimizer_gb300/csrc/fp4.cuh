// Device-side helpers for microscaled 4-bit floating point: the codes' and scales' conversions and
// the scales' place in memory.
#pragma once

#include "common.cuh"
#include "fp4.h"

namespace gns {

// Byte of row r, block k in its 512-byte tile of 128 rows x 4 blocks. The four scales of a row
// are one word, and the words of rows 32 apart lie side by side: the order in which
// tcgen05.cp takes 32 rows of 16 bytes to the 32 lanes x 4 columns that the block-scaled MMA
// reads them from.
GNS_DEV int fp4_scale_at(int r, int k) { return ((r & 31) << 4) | (((r >> 5) & 3) << 2) | (k & 3); }

// 2^(e - 127) for a byte e (0: 2^-127, a subnormal), NaN for 255.
GNS_DEV float e8m0_to_f(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : e == 255u ? 0x7FC00000u : e << 23);
}

// Two e4m3 values, low byte first (every e4m3 value is an fp16 one).
GNS_DEV float2 e4m3x2_to_f2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
GNS_DEV float e4m3_to_f(uint8_t v) { return e4m3x2_to_f2(v).x; }

// Nearest e4m3, ties to even, at most 448; NaN stays NaN (0x7F).
GNS_DEV uint8_t f_to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return static_cast<uint8_t>(r);
}

// Four bytes of two codes each, from eight values: nearest, ties to even, at most 6.
GNS_DEV uint32_t f8_to_e2m1(float a, float b, float c, float d, float e, float f, float g, float h) {
  uint32_t r;
  asm("{\n\t.reg .b8 p0, p1, p2, p3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p3, %8, %7;\n\t"
      "mov.b32 %0, {p0, p1, p2, p3};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d), "f"(e), "f"(f), "f"(g), "f"(h));
  return r;
}

// The two values of one byte (every code's value is an fp16 one), as two halves.
GNS_DEV uint32_t e2m1x2_to_h2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 p0, p1, p2, p3;\n\t"
      "mov.b32 {p0, p1, p2, p3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p0;\n\t}"
      : "=r"(h)
      : "r"(byte));
  return h;
}
GNS_DEV float2 e2m1x2_to_f2(uint32_t byte) {
  const uint32_t h = e2m1x2_to_h2(byte);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <int FMT>
GNS_DEV float fp4_scale_to_f(uint8_t s) {
  return FMT == GNS_NVFP4 ? e4m3_to_f(s) : e8m0_to_f(s);
}

// The smallest power of two g with amax <= 6 * 448 * g (6 * 448 = 1.3125 * 2^11), at least
// 2^-126, from the bits of a finite amax >= 0; 0 for 0.
GNS_DEV uint32_t fp4_tensor_scale_bits(uint32_t amax_bits) {
  if (amax_bits == 0u) return 0u;
  const int e = (int)(amax_bits >> 23) - 11 + ((amax_bits & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e) << 23;
}

// 1 / g of a power of two 2^-126 <= g <= 2^126.
GNS_DEV float pow2_inverse(float g) { return __uint_as_float((254u << 23) - __float_as_uint(g)); }

}  // namespace gns
