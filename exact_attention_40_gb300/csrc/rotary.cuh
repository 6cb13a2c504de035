// Rotary angles of several position axes and their cosines and sines.
//
// Pair i of d/2 turns by position[axis(i)] * theta_i.  u_i = theta_i / (2 pi)
// is held as a 64-bit fixed-point fraction of a turn (formed on the host in
// fp64), so the angle in turns is one integer product modulo 2^64: exact for
// any position, negative ones too.  The angle is brought to |x| <= pi/4 and the
// sine and cosine are Taylor sums whose two largest terms are kept with their
// rounding errors, so both come out within 2^-29 of the exact value before
// the last rounding: the nearest fp32 number but for a few in a hundred.  The
// 4-bit cache needs that: a key next to the border of two codes must fall to
// the side that the exact rotation says, and one unit in the last place of a
// cosine moves every key of its pair.
#pragma once
#include <cstdint>

#include "launch.h"

namespace exattn {

// cos and sin of `turn` / 2^64 turns.
__device__ __forceinline__ float2 turn_cos_sin(unsigned long long turn) {
  const unsigned int quadrant = static_cast<unsigned int>((turn + (1ull << 61)) >> 62);
  const long long rem = static_cast<long long>(turn - (static_cast<unsigned long long>(quadrant) << 62));
  // |rem| <= 2^61 as two exact fp32 integers: rem / 2^14 = r1 * 2^24 + r0
  const float r1 = static_cast<float>(static_cast<int>(rem >> 38));
  const float r0 = static_cast<float>(static_cast<int>((rem >> 14) & 0xFFFFFF));
  // x = xh + xl = 2 pi rem / 2^64; 2 pi = 6.28318548202514648 - 1.7484556e-7
  constexpr float kC1h = 6.28318548202514648f * 1.4901161193847656e-8f;   // 2 pi * 2^-26, leading part
  constexpr float kC1l = -1.7484556e-7f * 1.4901161193847656e-8f;     // ... the rest
  constexpr float kC0 = 6.28318548202514648f * 8.8817841970012523e-16f;   // 2 pi * 2^-50
  const float xh = __fmul_rn(r1, kC1h);
  const float xl = __fmaf_rn(r1, kC1h, -xh) + __fmaf_rn(r1, kC1l, __fmul_rn(r0, kC0));
  const float z = __fmul_rn(xh, xh);
  const float zl = __fmaf_rn(xh, xh, -z) + 2.f * xh * xl;
  // cos x = 1 - z/2 + z^2/24 - ...; 1 - z/2 with its rounding error
  const float h = 0.5f * z;
  const float a = __fsub_rn(1.f, h);
  const float ae = __fsub_rn(__fsub_rn(1.f, a), h);
  const float pc =
      z * z * fmaf(z, fmaf(z, fmaf(z, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f), 4.1666667e-2f);
  const float c = __fadd_rn(a, ae + fmaf(-0.5f, zl, pc));
  // sin x = x - x^3/6 + x^5/120 - ...; x - x^3/6 with its rounding errors
  const float p = __fmul_rn(xh, z);
  const float pl = __fmaf_rn(xh, z, -p) + fmaf(xh, zl, xl * z);
  constexpr float kS3h = -0.16666667163372039795f, kS3l = 4.9670537e-9f;  // -1/6
  const float u = __fmul_rn(kS3h, p);
  const float ul = __fmaf_rn(kS3h, p, -u) + fmaf(kS3h, pl, kS3l * p);
  const float ps =
      p * z * fmaf(z, fmaf(z, fmaf(z, -2.5052108e-8f, 2.7557319e-6f), -1.9841270e-4f), 8.3333333e-3f);
  const float b = __fadd_rn(xh, u);
  const float be = __fadd_rn(__fsub_rn(xh, b), u);
  const float s = __fadd_rn(b, be + (ul + (xl + ps)));
  const float cq = (quadrant & 1u) ? s : c;
  const float sq = (quadrant & 1u) ? c : s;
  return make_float2((quadrant == 1u || quadrant == 2u) ? -cq : cq, quadrant >= 2u ? -sq : sq);
}

}  // namespace exattn
