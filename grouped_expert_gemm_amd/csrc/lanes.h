// Reductions over 2^n neighbouring lanes of a wavefront, the result in every lane, on the
// vector ALU's own lane moves (DPP, and gfx950's row and half swaps): a butterfly step is a
// few cycles where a shuffle through LDS waits about a hundred.
#pragma once

#include "common.h"

namespace moe {

template <int CTRL>
__device__ __forceinline__ uint32_t lane_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// op over groups of L lanes (L = 1, 2, 4, ... 64). Steps 4 and 8 read the mirrored lane of a
// half row and of a row: the groups below already hold one value each, so any lane of the
// other group serves.
template <int L, typename F>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, F op) {
  if constexpr (L >= 2) v = op(v, lane_move<0xB1>(v));   // quad_perm 1, 0, 3, 2
  if constexpr (L >= 4) v = op(v, lane_move<0x4E>(v));   // quad_perm 2, 3, 0, 1
  if constexpr (L >= 8) v = op(v, lane_move<0x141>(v));  // row_half_mirror
  if constexpr (L >= 16) v = op(v, lane_move<0x140>(v)); // row_mirror
  if constexpr (L >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op((uint32_t)s[0], (uint32_t)s[1]);
  }
  if constexpr (L >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op((uint32_t)s[0], (uint32_t)s[1]);
  }
  return v;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(lanes_reduce<L>(
      __float_as_uint(v), [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); }));
}

template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  return __uint_as_float(lanes_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}

template <int L>
__device__ __forceinline__ uint32_t lanes_umax(uint32_t v) {
  return lanes_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

}  // namespace moe
