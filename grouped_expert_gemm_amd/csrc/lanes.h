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

// the sum of a float64 over the wavefront: both halves move, the additions are the ALU's own
__device__ __forceinline__ double wave_sum(double v) {
  auto add = [&](uint32_t lo, uint32_t hi) { v += __hiloint2double((int)hi, (int)lo); };
  auto step = [&](auto move) {
    const uint32_t lo = (uint32_t)__double2loint(v), hi = (uint32_t)__double2hiint(v);
    add(move(lo), move(hi));
  };
  step([](uint32_t x) { return lane_move<0xB1>(x); });
  step([](uint32_t x) { return lane_move<0x4E>(x); });
  step([](uint32_t x) { return lane_move<0x141>(x); });
  step([](uint32_t x) { return lane_move<0x140>(x); });
  const auto swapped = [&](auto a, auto b) { return __hiloint2double((int)b, (int)a); };
  {
    const uint32_t lo = (uint32_t)__double2loint(v), hi = (uint32_t)__double2hiint(v);
    const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false), h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    v = swapped(l[0], h[0]) + swapped(l[1], h[1]);
  }
  {
    const uint32_t lo = (uint32_t)__double2loint(v), hi = (uint32_t)__double2hiint(v);
    const auto l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false), h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    v = swapped(l[0], h[0]) + swapped(l[1], h[1]);
  }
  return v;
}

// The end of the last expert's rows as the grouped GEMMs, which take the offsets as their running
// maximum inside [0, R], have it: the largest of offsets[0..E], clamped. Every lane active.
__device__ __forceinline__ int64_t routed_end(const int32_t* __restrict__ offsets, int E, int64_t R) {
  const int lane = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  int top = 0;
  for (int e = lane; e <= E; e += 64) top = max(top, offsets[e]);
  top = (int)lanes_reduce<64>((uint32_t)top, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
  return top < R ? top : R;
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
