// Rotary angles of several position axes and their cosines and sines.
//
// Pair i of d/2 turns by position[axis(i)] * theta_i.  u_i = theta_i / (2 pi)
// is held as a 64-bit fixed-point fraction of a turn (formed on the host in
// fp64), so the angle in turns is one integer product modulo 2^64, for negative
// positions too, and its reduction loses nothing.  What is left is u's own rounding,
// some 1e-15 relative and 2^-65 absolute: beyond 10^7 radians it moves an angle by
// about half an fp32 unit.  The angle is brought to |x| <= pi/4 and the
// sine and cosine are Taylor sums whose three largest terms are kept with their
// rounding errors, so that the last rounding gives the nearest fp32 number but for
// 3 in 10,000 (14 in 1,000 with two such terms).  The 4-bit cache needs that: a key
// next to the border of two codes must fall to the side that the exact rotation
// says, and one unit in the last place of a cosine moves every key of its pair.
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
  // cos x = 1 - z/2 + z^2/24 - z^3/720 + ...
  const float h = 0.5f * z;
  const float a = __fsub_rn(1.f, h);
  const float ae = __fsub_rn(__fsub_rn(1.f, a), h);
  const float zz = __fmul_rn(z, z);
  const float zzl = __fmaf_rn(z, z, -zz) + 2.f * z * zl;
  constexpr float kC4h = 0.0416666679084301f, kC4l = -1.2417634e-9f;  // 1/24
  const float w = __fmul_rn(kC4h, zz);
  const float wl = __fmaf_rn(kC4h, zz, -w) + fmaf(kC4h, zzl, kC4l * zz);
  const float d = __fadd_rn(a, w);
  const float de = __fadd_rn(__fsub_rn(a, d), w);
  const float rc = zz * z * fmaf(z, fmaf(z, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f);
  const float c = __fadd_rn(d, (de + ae) + fmaf(-0.5f, zl, wl) + rc);
  // sin x = x - x^3/6 + x^5/120 - x^7/5040 + ...
  const float p = __fmul_rn(xh, z);
  const float pl = __fmaf_rn(xh, z, -p) + fmaf(xh, zl, xl * z);
  constexpr float kS3h = -0.16666667163372039795f, kS3l = 4.9670537e-9f;  // -1/6
  const float u = __fmul_rn(kS3h, p);
  const float ul = __fmaf_rn(kS3h, p, -u) + fmaf(kS3h, pl, kS3l * p);
  const float q = __fmul_rn(p, z);
  const float ql = __fmaf_rn(p, z, -q) + fmaf(p, zl, pl * z);
  constexpr float kS5h = 0.008333333767950535f, kS5l = -4.3461720e-10f;  // 1/120
  const float v = __fmul_rn(kS5h, q);
  const float vl = __fmaf_rn(kS5h, q, -v) + fmaf(kS5h, ql, kS5l * q);
  const float b = __fadd_rn(xh, u);
  const float be = __fadd_rn(__fsub_rn(xh, b), u);
  const float e = __fadd_rn(b, v);
  const float ee = __fadd_rn(__fsub_rn(b, e), v);
  const float rs = q * z * fmaf(z, fmaf(z, -2.5052108e-8f, 2.7557319e-6f), -1.9841270e-4f);
  const float s = __fadd_rn(e, ((ee + be) + ((ul + vl) + xl)) + rs);
  const float cq = (quadrant & 1u) ? s : c;
  const float sq = (quadrant & 1u) ? c : s;
  return make_float2((quadrant == 1u || quadrant == 2u) ? -cq : cq, quadrant >= 2u ? -sq : sq);
}

}  // namespace exattn
