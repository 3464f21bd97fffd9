// Per-row 8-bit coding shared by the quantizer and the products.
#pragma once
#include "common.hpp"

namespace moeq {

struct RowScale {
  float scale;   // code = rint(x / scale), value = code * scale
  bool zero;     // every code is 0
};

// The row's scale from its largest magnitude.  A row below 2^-118, whose
// scale would be subnormal, is coded as zeros.
__device__ __forceinline__ RowScale row_scale_of(float top, bool bad) {
  if (bad) return RowScale{__builtin_nanf(""), true};
  if (top < 0x1p-118f) return RowScale{1.f, true};
  return RowScale{top / 127.f, false};
}

// x / scale rounded to the nearest integer, half to even; |x| <= top keeps
// it within 127.  The quotient is a correctly rounded division: for 16-bit
// x it then rounds as the exact 127 x / top does, but for x = +-top / 2.
// (With integers X, A < 2^11 and powers of two aside, 127 X / A differs from
// a half n + 1/2 by 0 or by at least 1 / (2 A), far above the fp32 error;
// and where it is a half with 2 n + 1 != 127, A is a multiple of 127 and the
// scale exact.  A product with 127 / top would round some of those halves the
// wrong way.)
__device__ __forceinline__ int i8_code(float x, RowScale r) {
  return r.zero ? 0 : (int)__builtin_rintf(x / r.scale);
}

// The codes of eight values, a byte each.  x * (1 / scale) is within 3
// roundings (2^-24 of at most 127 each) of the quotient: only next to a half
// (here 2^-14) can it round otherwise, and the division is made.
__device__ __forceinline__ u32x2 i8_codes(const float *x, RowScale r) {
  const float inv = r.zero ? 0.f : 1.f / r.scale;
  float q[8];
  bool near = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = x[j] * inv;
    q[j] = __builtin_rintf(t);
    near |= __builtin_fabsf(__builtin_fabsf(t - q[j]) - 0.5f) < 0x1p-14f;
  }
  if (near) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = (float)i8_code(x[j], r);
  }
  u32x2 c = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) c[j / 4] |= (r.zero ? 0u : (uint32_t)(int)q[j] & 0xffu) << (8 * (j & 3));
  return c;
}

// row_scale_of for a workgroup of NW waves that each hold part of one row
// (s_top: NW floats; the result is the same in every thread).
template <int NW>
__device__ __forceinline__ RowScale row_scale(float top, bool bad, float *s_top) {
  if (bad) top = __builtin_inff();
#pragma unroll
  for (int o = 32; o; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o, kWave));
  if constexpr (NW == 1) return row_scale_of(top, top == __builtin_inff());
  if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) top = __builtin_fmaxf(top, s_top[w]);
  return row_scale_of(top, top == __builtin_inff());
}

moeq_status launch_quantize_i8(const void *x, int64_t ldx, int32_t rows, int32_t cols, int32_t dtype, int8_t *codes,
                               int64_t ldc, float *scales, hipStream_t s);

}  // namespace moeq
