// Per-row 8-bit coding shared by the quantizer and the products.
#pragma once
#include "common.hpp"

namespace moeq {

struct RowScale {
  float inv, scale;   // code = rint(x * inv), value = code * scale
};

// The row's scale from its largest magnitude.  Below 2^-118 the reciprocal
// would leave the fp32 range: such a row is coded as zeros.
__device__ __forceinline__ RowScale row_scale_of(float top, bool bad) {
  if (bad) return RowScale{0.f, __builtin_nanf("")};
  if (top < 0x1p-118f) return RowScale{0.f, 1.f};
  return RowScale{127.f / top, top / 127.f};
}

// x * inv rounded to the nearest integer, half to even.  |x| <= top keeps it
// within 127.  (inv = 0: the row's codes are 0, also for an infinity or NaN.)
__device__ __forceinline__ int i8_code(float x, float inv) {
  return inv == 0.f ? 0 : (int)__builtin_rintf(x * inv);
}

// row_scale_of for a workgroup of NW waves that each hold part of one row
// (s_top: NW floats; the result is the same in every thread).
template <int NW>
__device__ __forceinline__ RowScale row_scale(float top, bool bad, float *s_top) {
  if (bad) top = __builtin_inff();
#pragma unroll
  for (int o = 32; o; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o, kWave));
  if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) top = __builtin_fmaxf(top, s_top[w]);
  return row_scale_of(top, top == __builtin_inff());
}

moeq_status launch_quantize_i8(const void *x, int64_t ldx, int32_t rows, int32_t cols, int32_t dtype, int8_t *codes,
                               int64_t ldc, float *scales, hipStream_t s);

}  // namespace moeq
