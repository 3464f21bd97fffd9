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
