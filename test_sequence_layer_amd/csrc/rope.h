// The angle of a rotary position.
#pragma once
#include "args_attn.h"

namespace ttt {

// cos and sin of position * freq.  The product and its reduction to one turn are
// in 64 bits: at position 10^6 an fp32 product would be 0.03 radians off.  What is
// left is at most half a turn, whose rounding to fp32 costs 2^-24 of it.
__device__ __forceinline__ void rope_angle(int64_t pos, double freq, float& c, float& s) {
  const double turns = static_cast<double>(pos) * freq * 0.15915494309189533577;  // 1 / (2 pi)
  sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
}

__device__ __forceinline__ int64_t rope_pos(const Rope& r, int b, int t) {
  if (!r.pos) return r.pos0 + t;
  return r.pos0 + (r.pos_t ? r.pos[b * r.pos_b + t * r.pos_t] : r.pos[b * r.pos_b] + t);
}

}  // namespace ttt
