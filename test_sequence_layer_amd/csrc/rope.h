// The angle of a rotary position.
#pragma once
#include "args_attn.h"

namespace ttt {

// cos and sin of position * freq.  The product and its reduction to one turn are in
// 64 bits: at position 10^6 an fp32 product would be 0.03 radians off.  What is left, at
// most half a turn, goes to the fp32 functions rounded, and what that rounding took off (up
// to pi 2^-25, which near half a turn is many steps of the sine) is put back to first order.
__device__ __forceinline__ void rope_angle(int64_t pos, double freq, float& c, float& s) {
  const double turns = static_cast<double>(pos) * freq * 0.15915494309189533577;  // 1 / (2 pi)
  const double x = 2.0 * (turns - rint(turns));                                   // in units of pi
  const float near = static_cast<float>(x);
  const float rest = 3.14159265f * static_cast<float>(x - static_cast<double>(near));
  float c0, s0;
  sincospif(near, &s0, &c0);
  c = fmaf(-s0, rest, c0);
  s = fmaf(c0, rest, s0);
}

__device__ __forceinline__ int64_t rope_pos(const Rope& r, int b, int t) {
  if (!r.pos) return r.pos0 + t;
  return r.pos0 + (r.pos_t ? r.pos[b * r.pos_b + t * r.pos_t] : r.pos[b * r.pos_b] + t);
}

}  // namespace ttt
