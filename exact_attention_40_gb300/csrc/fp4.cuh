// The 4-bit cache format and its conversions.
//
// A value is code * scale * g: code an e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4,
// 6 and their negatives), scale an e4m3 number shared by 16 neighbouring
// columns, g the tensor's fp32 scale.  code * scale has at most 6 significant
// bits and lies in [2^-10, 2688], so fp16 holds it exactly.
//
// One block of 16 tokens of one KV head is one span of 18 d bytes, so that a
// single bulk copy brings everything the attention needs of it:
//   [0, 8 d)      key codes   [16 tokens][d/2]: column 2c in the low, 2c + 1 in
//                 the high four bits of byte c
//   [8 d, 16 d)   value codes [16][d/2]
//   [16 d, 17 d)  key scales  [16][d/16]
//   [17 d, 18 d)  value scales [16][d/16]
#pragma once
#include <cstddef>
#include <cstdint>

namespace exattn {

constexpr int kFp4Group = 16;  // columns that share a scale

template <int D>
struct Fp4Span {
  static constexpr int kKeyCodes = 0;
  static constexpr int kValueCodes = 8 * D;
  static constexpr int kKeyScales = 16 * D;
  static constexpr int kValueScales = 17 * D;
  static constexpr int kBytes = 18 * D;
  static constexpr int kCodeRow = D / 2;           // bytes of one token's codes
  static constexpr int kScaleRow = D / kFp4Group;  // ... and scales
};

// Eight e2m1 codes (low four bits first) as four fp16 pairs, exactly.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight fp32 values to e2m1 (nearest, ties to even, saturating at 6).
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float* x) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

// Two e4m3 numbers (low 16 bits) as an fp16 pair, exactly; 0x7F is NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t b) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(b));
  return h;
}

// One fp32 value to e4m3 (nearest, ties to even, saturating at 448).
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(x));
  return h & 0xFFu;
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float f16_lo(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

__device__ __forceinline__ float f16_hi(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, u;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Maximum that returns NaN when an operand is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace exattn
