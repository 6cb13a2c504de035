// The 8-bit cache format and its conversions.
//
// A value is code * scale: code an e4m3 number, scale a power of two, one for the keys
// and one for the values of each block of 16 tokens of one KV head.  Such a scale only
// moves exponents: codes are divided by it and multiplied by it exactly, a code times
// its scale is a bf16 number, and when a block that fills token by token needs a larger
// one, the codes already there keep their value but for those that fall below 2^-6 of it.
//
// One block of one KV head is one span of 32 d + 32 bytes, so that a single bulk copy
// brings everything the attention needs of it:
//   [0, 16 d)      key codes, [16 tokens][d], each row's d/16 chunks of 16 bytes in an
//                  order of its own: chunk c of token n is the (c ^ fp8_turn(n))-th
//   [16 d, 32 d)   value codes, the same
//   32 d, 32 d + 4 the scales of the keys and the values, fp32; 24 bytes are unused (a
//                  span is a whole number of sectors)
// The order of the chunks is that of shared memory's banks: eight lanes that read a
// chunk each of two rows (keys) or of four (values) meet all 32 of them, with the span
// copied as it lies.
#pragma once
#include <cstddef>
#include <cstdint>

#include "fp4.cuh"

namespace exattn {

constexpr int kFp8LowExponent = -117;   // of a scale: its smallest code stays a normal number
constexpr int kFp8HighExponent = 119;   // 448 of them stay finite

template <int D>
struct Fp8Span {
  static constexpr int kKeyCodes = 0;
  static constexpr int kValueCodes = 16 * D;
  static constexpr int kScales = 32 * D;
  static constexpr int kBytes = 32 * D + 32;
  static constexpr int kRow = D;  // bytes of one token's codes
};

// What the numbers of token n's chunks are turned by.
template <int D>
__host__ __device__ constexpr int fp8_turn(int n) {
  return D == 128 ? n & 7 : (n >> 1) & 3;
}

// Biased exponent of the scale for a largest magnitude: the smallest with which it is at
// most 448 = 1.75 * 2^8.
__device__ __forceinline__ int fp8_scale_exponent(float most) {
  const uint32_t u = __float_as_uint(most);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(127 + kFp8LowExponent, min(127 + kFp8HighExponent, e));
}

// Four e4m3 numbers as two fp16 pairs, exactly; 0x7F and 0xFF are NaN.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Four fp32 values to e4m3 (nearest, ties to even, saturating at 448; NaN stays NaN).
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 l, u;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 u, %4, %3;\n\t"
      "mov.b32 %0, {l, u};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

}  // namespace exattn
