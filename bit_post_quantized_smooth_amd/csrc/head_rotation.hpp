// The rotation of a head's channels by a position (gfx950).
//
// Channel pairs (a, b) turn by position * freq radians. The angle is formed and
// reduced in fp64, in whole turns: position * (freq / 2 pi) is good to 3 * 2^-53 of
// itself, so at an angle of 2^20 radians it is good to 2^-31 of one, where an fp32 angle
// would be off by 2^-4. At 2^28 radians that is 2^-23.4, less than fp32's roundings
// behind it; at 2^31 it is 2^-20.4 and exceeds them. What is left, at most an eighth of a
// turn, goes through the Taylor polynomials of sine (to x^9) and cosine (to x^8),
// whose next terms are below 2e-9 and 3e-8, less than an fp32 rounding. Nine fp64
// instructions, three conversions and 20 fp32 ones per pair and token, shared by the
// token's heads: a table of cosines would cost a load of as many bytes as a head.
#pragma once

#include "block_common.hpp"

namespace svdq {

__device__ __forceinline__ void cos_sin(int32_t position, double freq, float& c, float& s) {
  const double turns = static_cast<double>(position) * (freq * 0.15915494309189535);
  const double part = turns - __builtin_rint(turns);             // -1/2 .. 1/2
  const double quarter = __builtin_rint(4.0 * part);
  const float x = static_cast<float>((part - 0.25 * quarter) * 6.283185307179586);
  const float t = x * x;
  const float sx =
      __builtin_fmaf(x * t, __builtin_fmaf(t, __builtin_fmaf(t, __builtin_fmaf(t, 1.f / 362880.f, -1.f / 5040.f),
                                                             1.f / 120.f), -1.f / 6.f), x);
  const float cx =
      __builtin_fmaf(t, __builtin_fmaf(t, __builtin_fmaf(t, __builtin_fmaf(t, 1.f / 40320.f, -1.f / 720.f),
                                                         1.f / 24.f), -0.5f), 1.f);
  const int q = static_cast<int>(quarter);
  c = (q & 1) ? sx : cx;
  s = (q & 1) ? cx : sx;
  if ((q + 1) & 2) c = -c;
  if (q & 2) s = -s;
}

}  // namespace svdq
