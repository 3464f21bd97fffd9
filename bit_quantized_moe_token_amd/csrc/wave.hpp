// Exchanges and sums over the lanes of a wave by DPP, and the order of its LDS
// accesses.
#pragma once
#include "common.hpp"

namespace moeq {

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, dpp_i<CTRL>(__builtin_bit_cast(int, v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{(uint32_t)dpp_i<CTRL>((int)b[0]), (uint32_t)dpp_i<CTRL>((int)b[1])});
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_into(int v, int old) {   // lanes of the other rows keep old
  return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_into(float v, float old) {
  return __builtin_bit_cast(float, dpp_into<CTRL, ROWS>(__builtin_bit_cast(int, v), __builtin_bit_cast(int, old)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_into(double v, double old) {
  const u32x2 b = __builtin_bit_cast(u32x2, v), o = __builtin_bit_cast(u32x2, old);
  return __builtin_bit_cast(double, u32x2{(uint32_t)dpp_into<CTRL, ROWS>((int)b[0], (int)o[0]),
                                          (uint32_t)dpp_into<CTRL, ROWS>((int)b[1], (int)o[1])});
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)b[0], lane),
                                          (uint32_t)__builtin_amdgcn_readlane((int)b[1], lane)});
}
// Sum over the wave, the same in every lane: within rows of 16 by exchanges,
// then row_bcast:15 and row_bcast:31 into lane 63.
template <typename V>
__device__ __forceinline__ V all_sum(V v) {
  v += dpp<0xb1>(v);
  v += dpp<0x4e>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  v += dpp_into<0x142, 0xa>(v, (V)0);
  v += dpp_into<0x143, 0xc>(v, (V)0);
  return lane_value(v, 63);
}

// Between LDS accesses of one wave that may not change places (the hardware
// keeps their order; this keeps the compiler to it).
__device__ __forceinline__ void lds_order() { asm volatile("" ::: "memory"); }

}  // namespace moeq
