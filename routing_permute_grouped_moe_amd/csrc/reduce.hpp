// Sums over lanes on the vector ALU alone: a shuffle goes through LDS and takes
// some 60 cycles a step, a DPP or permlane step a few.
#pragma once

#include "common.hpp"

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf,
                                                               0xf, true));
}
// v of the lane 32 (16) away, added: the swap leaves a half's (row's) values in both.
__device__ __forceinline__ float add_swap32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_swap16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float max_swap32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_swap16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The sum over each N lanes in a row (8, 16, 32 or 64), in all of them.  From 16
// on the pairs are those of wave_sum, so the bits are the same.
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  static_assert(N == 8 || N == 16 || N == 32 || N == 64, "lanes");
  if constexpr (N == 8) {
    v += dpp<0x141>(v);               // row_half_mirror
    v += dpp<0x4e>(v);                // quad_perm 2 3 0 1
    v += dpp<0xb1>(v);                // quad_perm 1 0 3 2
  } else {
    if constexpr (N == 64) v = add_swap32(v);
    if constexpr (N >= 32) v = add_swap16(v);
    v += dpp<0x128>(v);               // row_ror 8, 4, 2, 1
    v += dpp<0x124>(v);
    v += dpp<0x122>(v);
    v += dpp<0x121>(v);
  }
  return v;
}
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
  static_assert(N == 16 || N == 32 || N == 64, "lanes");
  if constexpr (N == 64) v = max_swap32(v);
  if constexpr (N >= 32) v = max_swap16(v);
  v = fmaxf(v, dpp<0x128>(v));
  v = fmaxf(v, dpp<0x124>(v));
  v = fmaxf(v, dpp<0x122>(v));
  return fmaxf(v, dpp<0x121>(v));
}

// The same of a double: its halves move side by side.
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const unsigned long long u = __builtin_bit_cast(unsigned long long, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, ((unsigned long long)hi << 32) | lo);
}
__device__ __forceinline__ double lanes_sum64(double v) {
  auto join = [](uint32_t hi, uint32_t lo) {
    return __builtin_bit_cast(double, ((unsigned long long)hi << 32) | lo);
  };
  unsigned long long u = __builtin_bit_cast(unsigned long long, v);
  auto lo = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
  auto hi = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  v = join(hi[0], lo[0]) + join(hi[1], lo[1]);
  u = __builtin_bit_cast(unsigned long long, v);
  lo = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
  hi = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  v = join(hi[0], lo[0]) + join(hi[1], lo[1]);
  v += dpp64<0x128>(v);
  v += dpp64<0x124>(v);
  v += dpp64<0x122>(v);
  return v + dpp64<0x121>(v);
}
// A whole number's, over the 64 lanes.
__device__ __forceinline__ int lanes_sum_int(int v) {
  const auto a = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
  v = (int)(a[0] + a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
  v = (int)(b[0] + b[1]);
  v += __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x124, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x122, 0xf, 0xf, true);
  return v + __builtin_amdgcn_update_dpp(0, v, 0x121, 0xf, 0xf, true);
}
