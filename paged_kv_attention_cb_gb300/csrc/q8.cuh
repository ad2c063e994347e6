// The 8-bit cache format (device side): e4m3 values with one power-of-two scale per row.
//
// A row is the K (or V) of one token and KV head, D values x. Its scale is 2^e with the
// least e >= -126 for which max |x| <= 448 * 2^e (448: the largest e4m3 value), stored as
// the byte e + 127 (e8m0); the values are x / 2^e rounded to nearest even. Powers of two
// because e4m3 is a floating format: its 3 fraction bits bound the relative error by 2^-4
// wherever the row's largest value lies below 448 scales, so a finer scale would buy nothing
// but the last binade's headroom, while with a power of two both x / 2^e and the value read
// back are exact in fp32 (and in bf16), the one rounding is the conversion to e4m3, and a
// scale takes one byte per row (1/128 of the stream at D 128).
#pragma once
#include "common.cuh"

namespace cb {

constexpr int kE8m0Bias = 127;

// Bits of |x|, 0 where x is infinite or NaN (they take no part in the choice of the scale).
// The bits of non-negative floats order as the floats do, so maxima are taken on them.
CB_DEV uint32_t finite_magnitude(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// The scale code of a row from the bits of its largest finite magnitude a = 1.m * 2^k:
// a <= 1.75 * 2^(8 + e) holds from e = k - 8 on if 1.m <= 1.75, else from k - 7.
CB_DEV int e8m0_of_magnitude(uint32_t a) {
  if (a == 0u) return kE8m0Bias;
  const int k = (int)(a >> 23) - 127;  // -127 for subnormals: below the clamp either way
  const int e = k - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -126) + kE8m0Bias;
}

// 2^-(code - 127) for a code e8m0_of_magnitude returns (1 .. 247): exact, normal.
CB_DEV float e8m0_inverse(int code) { return __uint_as_float((uint32_t)(254 - code) << 23); }

// 2^(code - 127); code 0 is 2^-127 (subnormal) and code 255 NaN, as in the e8m0 format.
CB_DEV float e8m0_value(int code) {
  uint32_t b = (uint32_t)code << 23;
  if (code == 0) b = 0x00400000u;
  if (code == 255) b = 0x7fc00000u;
  return __uint_as_float(b);
}

// Two fp32 values to e4m3, round to nearest even, magnitudes past 448 (infinities too) to
// 448, NaN to NaN: `lo` in the low byte.
CB_DEV uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 values (16 bits) as a pair of fp16: exact.
CB_DEV uint32_t f16x2_of_e4m3x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}

CB_DEV float2 float2_of_f16x2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

}  // namespace cb
