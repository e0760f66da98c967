// Cross-lane sums and exchanges of a 64-wide wave.  Internal to libternary.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tern {

template <int CTRL>
__device__ inline float dpp_move(float x) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}

// x of the lower and of the upper half's lane, in the same order in both.
__device__ inline void halves(float x, float& lo, float& hi) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  // (An element of the pair is passed by value: a bit cast of the element
  // itself reads the first one.)
  lo = __uint_as_float(r[0]);
  hi = __uint_as_float(r[1]);
}

// The sum over the wave, in every lane: lanes 1 and 2 apart (quad permutes),
// the two quads of eight and the two eights of a row (mirrors), rows, halves.
__device__ inline float wave_sum(float x) {
  x += dpp_move<0xB1>(x);   // quad_perm [1, 0, 3, 2]
  x += dpp_move<0x4E>(x);   // quad_perm [2, 3, 0, 1]
  x += dpp_move<0x141>(x);  // row_half_mirror
  x += dpp_move<0x140>(x);  // row_mirror
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  float lo, hi;
  halves(x, lo, hi);
  return lo + hi;
}

// The sum over each aligned group of eight lanes, in every lane.
__device__ inline float eight_sum(float x) {
  x += dpp_move<0xB1>(x);
  x += dpp_move<0x4E>(x);
  return x + dpp_move<0x141>(x);
}

}  // namespace tern
