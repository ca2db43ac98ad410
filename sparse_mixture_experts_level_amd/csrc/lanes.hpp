// Reductions by lane moves, shared by the kernels that reduce rows held across lanes.
#pragma once

#include "common.hpp"

namespace moe {

// Reductions over groups of LPT neighbouring lanes, the result in every lane: lane moves
// within a row of 16 (lane ^ 1, lane ^ 2, then half-row and row mirrors, which pair equal
// values), then rows and halves of the wavefront exchanged.  T: a 32-bit type.
template <int CTRL, typename T>
__device__ __forceinline__ T lane_move(T v) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
template <int LPT, typename T, typename Op>
__device__ __forceinline__ T group_reduce(T v, Op op) {
  if constexpr (LPT >= 2) v = op(v, lane_move<0xb1>(v));
  if constexpr (LPT >= 4) v = op(v, lane_move<0x4e>(v));
  if constexpr (LPT >= 8) v = op(v, lane_move<0x141>(v));
  if constexpr (LPT >= 16) v = op(v, lane_move<0x140>(v));
  if constexpr (LPT >= 32) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = op(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
  }
  if constexpr (LPT >= 64) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = op(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
  }
  return v;
}

}  // namespace moe
