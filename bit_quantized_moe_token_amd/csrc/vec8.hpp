// Eight consecutive values of a row in 16 or 32 bits, as the kernels that
// work along rows read and write them.
#pragma once
#include "common.hpp"

namespace moeq {

typedef u32x4 u32x4_a2 __attribute__((aligned(2)));   // 16 bytes at the alignment of an element
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

template <int TY> struct Val;
template <> struct Val<MOEQ_F16> {
  static constexpr int size = 2;
  using Loose = u32x4_a2;
  static __device__ __forceinline__ float get(uint32_t bits) { return (float)__builtin_bit_cast(f16, (uint16_t)bits); }
  static __device__ __forceinline__ uint32_t put(float v) { return __builtin_bit_cast(uint16_t, (f16)v); }
};
template <> struct Val<MOEQ_BF16> {
  static constexpr int size = 2;
  using Loose = u32x4_a2;
  static __device__ __forceinline__ float get(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }
  static __device__ __forceinline__ uint32_t put(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
template <> struct Val<MOEQ_F32> {
  static constexpr int size = 4;
  using Loose = u32x4_a4;
  static __device__ __forceinline__ float get(uint32_t bits) { return __builtin_bit_cast(float, bits); }
  static __device__ __forceinline__ uint32_t put(float v) { return __builtin_bit_cast(uint32_t, v); }
};

// Eight consecutive elements as stored.  Loads and stores need no alignment
// beyond an element's; of a row's last piece only the first n exist.
template <int TY>
struct Oct {
  static constexpr int W = Val<TY>::size * 2;   // dwords
  using Loose = typename Val<TY>::Loose;
  uint32_t w[W];

  // (NT: non-temporal, past the caches; no run-time argument, since a choice
  // between two accesses to one address is merged into an ordinary one)
  template <bool NT = false>
  __device__ __forceinline__ void load(const void *base, int64_t i, int n) {
    const uint8_t *p = (const uint8_t *)base + i * Val<TY>::size;
    if (n >= 8) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const auto at = &((const __attribute__((address_space(1))) Loose *)p)[q];
        u32x4 v;
        if constexpr (NT) v = __builtin_nontemporal_load(at);
        else v = *at;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * q + j] = v[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j] = 0;
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < n) {
          if constexpr (TY == MOEQ_F32) w[j] = gld<uint32_t>(p + 4 * j);
          else w[j / 2] |= (uint32_t)gld<uint16_t>(p + 2 * j) << (16 * (j & 1));
        }
    }
  }
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (TY == MOEQ_F32) return Val<TY>::get(w[j]);
    else return Val<TY>::get((w[j / 2] >> (16 * (j & 1))) & 0xffffu);
  }
  __device__ __forceinline__ void fill(float v) {
    const uint32_t b = Val<TY>::put(v);
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = TY == MOEQ_F32 ? b : b | (b << 16);
  }
  // the same bits, which the compiler takes for new ones
  __device__ __forceinline__ void opaque() {
#pragma unroll
    for (int j = 0; j < W; ++j) asm volatile("" : "+v"(w[j]));
  }
  __device__ __forceinline__ void pack(const float *v) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if constexpr (TY == MOEQ_F32) w[j] = Val<TY>::put(v[j]);
      else w[j] = Val<TY>::put(v[2 * j]) | (Val<TY>::put(v[2 * j + 1]) << 16);
    }
  }
  template <bool NT = false>
  __device__ __forceinline__ void store(void *base, int64_t i, int n) const {
    uint8_t *p = (uint8_t *)base + i * Val<TY>::size;
    if (n >= 8) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const auto at = &((__attribute__((address_space(1))) Loose *)p)[q];
        const Loose v = u32x4{w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]};
        if constexpr (NT) __builtin_nontemporal_store(v, at);
        else *at = v;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < n) {
          if constexpr (TY == MOEQ_F32) *(uint32_t *)(p + 4 * j) = w[j];
          else *(uint16_t *)(p + 2 * j) = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
        }
    }
  }
};

}  // namespace moeq
