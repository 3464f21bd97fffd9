// Symmetric 8-bit coding of rows: one scale per token, or per output channel
// of a weight matrix ([MxMoE] abstract: linear blocks at different
// precisions).
#include "gemm.hpp"
#include "quant_i8.hpp"

namespace moeq {

template <int TY>
__device__ __forceinline__ float elt_at(const void *p, int64_t i) {
  if constexpr (TY == MOEQ_F32) return gld<float>((const float *)p + i);
  else if constexpr (TY == MOEQ_BF16) return __builtin_bit_cast(float, (uint32_t)gld<uint16_t>((const uint16_t *)p + i) << 16);
  else return (float)__builtin_bit_cast(f16, gld<uint16_t>((const uint16_t *)p + i));
}

// One workgroup per row.
template <int TY>
__global__ void __launch_bounds__(256) quantize_i8_kernel(const void *__restrict__ x, int64_t ldx, int32_t cols,
                                                          int8_t *__restrict__ codes, int64_t ldc,
                                                          float *__restrict__ scales) {
  const int64_t row = blockIdx.x;
  const uint8_t *src = (const uint8_t *)x + row * ldx * (TY == MOEQ_F32 ? 4 : 2);
  float top = 0.f;
  bool bad = false;
  for (int c = threadIdx.x; c < cols; c += 256) {
    const float v = __builtin_fabsf(elt_at<TY>(src, c));
    bad |= !(v <= 3.4028234663852886e38f);
    top = __builtin_fmaxf(top, v);
  }
  __shared__ float s_top[4];
  const RowScale r = row_scale<4>(top, bad, s_top);
  int8_t *dst = codes + row * ldc;
  for (int c = threadIdx.x; c < cols; c += 256) dst[c] = (int8_t)i8_code(elt_at<TY>(src, c), r);
  if (threadIdx.x == 0) scales[row] = r.scale;
}

moeq_status launch_quantize_i8(const void *x, int64_t ldx, int32_t rows, int32_t cols, int32_t dtype, int8_t *codes,
                               int64_t ldc, float *scales, hipStream_t s) {
  if (rows == 0) return MOEQ_OK;
  prof_begin("quantize_i8", s);
  const dim3 g((unsigned)rows), b(256);
  if (dtype == MOEQ_F16) hipLaunchKernelGGL(quantize_i8_kernel<MOEQ_F16>, g, b, 0, s, x, ldx, cols, codes, ldc, scales);
  else if (dtype == MOEQ_BF16) hipLaunchKernelGGL(quantize_i8_kernel<MOEQ_BF16>, g, b, 0, s, x, ldx, cols, codes, ldc, scales);
  else hipLaunchKernelGGL(quantize_i8_kernel<MOEQ_F32>, g, b, 0, s, x, ldx, cols, codes, ldc, scales);
  prof_end("quantize_i8", s);
  return check_launch("quantize_i8");
}

}  // namespace moeq
