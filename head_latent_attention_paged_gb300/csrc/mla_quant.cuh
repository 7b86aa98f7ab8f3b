// The quantisers of the FP8 and FP4 rows (e4m3 with one e8m0 scale per 32
// values, e2m1 with one per 16), shared by the cache appends and the norm.
#pragma once

#include <cstdint>

namespace mla {

__device__ __forceinline__ float bf16_bits_to_f32(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}

// ceil(log2(a / 448)) for a > 0 finite, exactly: a = m 2^E with m in [1, 2),
// 448 = 1.75 2^8, so a / 448 = (m / 1.75) 2^(E - 8) and m / 1.75 lies in
// (0.5, 1] unless m > 1.75.  Subnormal a gives a value below -127.
__device__ __forceinline__ int ceil_log2_over_448(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int ef = static_cast<int>((bits >> 23) & 0xFFu);
  if (ef == 0) return -200;
  const uint32_t man = bits & 0x7FFFFFu;
  return (ef - 127) - 8 + (man > 0x600000u ? 1 : 0);
}

// ceil(log2(a / 6)) for a > 0 finite, exactly: 6 = 1.5 2^2, so a / 6 =
// (m / 1.5) 2^(E - 2) with m / 1.5 in [2/3, 1] unless m > 1.5.
__device__ __forceinline__ int ceil_log2_over_6(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int ef = static_cast<int>((bits >> 23) & 0xFFu);
  if (ef == 0) return -200;
  const uint32_t man = bits & 0x7FFFFFu;
  return (ef - 127) - 2 + (man > 0x400000u ? 1 : 0);
}

// Nearest e2m1 code of v (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), ties to
// the even code, saturating at 6; the sign bit of v becomes bit 3.  Each
// comparison moves past one midpoint of the grid: a midpoint between an
// even and the next odd code counts only when exceeded, one between an odd
// and the next even code already when reached.
__device__ __forceinline__ uint32_t f32_to_e2m1(float v) {
  const float a = fabsf(v);
  const uint32_t mag = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) +
                       (a >= 3.5f) + (a > 5.0f);
  return mag | ((__float_as_uint(v) >> 28) & 8u);
}

// 2^-e as a float for e in [-127, 127] (2^-127 is the subnormal 0x00400000).
__device__ __forceinline__ float pow2_neg(int e) {
  return e == 127 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// The scale bytes e + 127 of the two quantisers, e = ceil(log2(amax / 448)) or
// ceil(log2(amax / 6)) clamped to -127 from below (0 for a zero amax): adding
// the mantissa's distance from 1.75 (1.5) to the next power of two carries
// into the exponent exactly where the ceiling does.  Bytes stay below 254, so
// the reciprocal 2^-e is a normal number.
__device__ __forceinline__ uint32_t e4m3_scale_byte(float amax) {
  return max((__float_as_uint(amax) + 0x1FFFFFu) >> 23, 8u) - 8u;
}
__device__ __forceinline__ uint32_t e2m1_scale_byte(float amax) {
  return max((__float_as_uint(amax) + 0x3FFFFFu) >> 23, 2u) - 2u;
}
__device__ __forceinline__ float scale_byte_reciprocal(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// e4m3 codes of two values, the first in the low byte: nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(hi), "f"(lo));
  return two;
}

__device__ __forceinline__ uint32_t f32_to_e4m3(float v) { return e4m3x2(v, v) & 0xFFu; }

// e2m1 codes of two values, the first in the low nibble, and of eight: as
// f32_to_e2m1.
__device__ __forceinline__ uint32_t pack_e2m1(float2 v) {
  uint32_t two;
  asm("{\n .reg .b8 c;\n cvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n cvt.u32.u8 %0, c;\n}"
      : "=r"(two)
      : "f"(v.y), "f"(v.x));
  return two;
}
__device__ __forceinline__ uint32_t pack_e2m1(const float2 (&v)[4]) {   // eight, in order from the low nibble
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(w)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return w;
}

}  // namespace mla
