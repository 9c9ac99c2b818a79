// Sums and maxima over a wave of 64 lanes by data-parallel moves: four steps within rows of 16 lanes, two across them, the result
// read from lane 63.  A step is an ordinary vector instruction (a shuffle goes through LDS and takes some 10 times as long).
#pragma once

#include <hip/hip_runtime.h>

namespace eff {

// v of the lane that CTRL names, `none` where there is no such lane or ROWS leaves this row of 16 out
template <int CTRL, int ROWS>
__device__ inline float lane_move(float none, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ inline float last_lane(float v) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63)); }

// all 64 lanes must be active
__device__ inline float wave_sum(float v) {
  v += lane_move<0x111, 0xF>(0.f, v);  // the lane 1, 2, 4, 8 below in its row
  v += lane_move<0x112, 0xF>(0.f, v);
  v += lane_move<0x114, 0xF>(0.f, v);
  v += lane_move<0x118, 0xF>(0.f, v);
  v += lane_move<0x142, 0xA>(0.f, v);  // the last lane of the row below, into rows 1 and 3
  v += lane_move<0x143, 0xC>(0.f, v);  // lane 31, into rows 2 and 3
  return last_lane(v);
}
__device__ inline float wave_max(float v) {
  const float none = -__builtin_inff();
  v = fmaxf(v, lane_move<0x111, 0xF>(none, v));
  v = fmaxf(v, lane_move<0x112, 0xF>(none, v));
  v = fmaxf(v, lane_move<0x114, 0xF>(none, v));
  v = fmaxf(v, lane_move<0x118, 0xF>(none, v));
  v = fmaxf(v, lane_move<0x142, 0xA>(none, v));
  v = fmaxf(v, lane_move<0x143, 0xC>(none, v));
  return last_lane(v);
}

}  // namespace eff
