// Symmetric 8-bit coding of rows: one scale per token, or per output channel
// of a weight matrix ([MxMoE] abstract: linear blocks at different
// precisions).
#include "quant_i8.hpp"
#include "vec8.hpp"

namespace moeq {

typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

// Eight codes at p, of which n exist.
__device__ __forceinline__ void store_codes(int8_t *p, u32x2 c, int n) {
  if (n >= 8) {
    *(__attribute__((address_space(1))) u32x2_a1 *)p = c;
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < n) p[j] = (int8_t)(c[j / 4] >> (8 * (j & 3)));
  }
}

template <int TY>
__device__ __forceinline__ void oct_max(const Oct<TY> &v, float *top, bool *bad) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = __builtin_fabsf(v[j]);
    *bad |= !(m <= 3.4028234663852886e38f);
    *top = __builtin_fmaxf(*top, m);
  }
}

template <int TY>
__device__ __forceinline__ u32x2 oct_codes(const Oct<TY> &v, RowScale r) {
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = v[j];
  return i8_codes(x, r);
}

// One pass: NT threads hold a row in registers (thread t the pieces of eight
// t, t + NT, ...) between its maximum and its codes.  NT = 64: four rows per
// workgroup.  Bound by memory (4096 rows of 14336 in bf16: 36 us, 4.9 TB/s;
// reading them twice, an element at a time, took 92).
template <int TY, int NT, int CH>
__global__ void __launch_bounds__(NT == 64 ? 256 : NT) quantize_i8_kernel(const void *__restrict__ x, int64_t ldx,
                                                                         int32_t rows, int32_t cols,
                                                                         int8_t *__restrict__ codes, int64_t ldc,
                                                                         float *__restrict__ scales) {
  constexpr int RW = NT == 64 ? 4 : 1;
  __shared__ float s_top[NT / 64];
  const int t = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * RW + threadIdx.x / NT;
  if (row >= rows) return;      // (whole waves; only with RW > 1, where no barrier follows)
  Oct<TY> v[CH];
  float top = 0.f;
  bool bad = false;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * NT + t) * 8;
    v[c].load(x, row * ldx + i, cols - i);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) oct_max(v[c], &top, &bad);
  const RowScale r = row_scale<NT / 64>(top, bad, s_top);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * NT + t) * 8;
    store_codes(codes + row * ldc + i, oct_codes(v[c], r), cols - i);
  }
  if (t == 0) scales[row] = r.scale;
}

// Rows of any length, read twice.
template <int TY>
__global__ void __launch_bounds__(1024) quantize_i8_long_kernel(const void *__restrict__ x, int64_t ldx, int32_t cols,
                                                                int8_t *__restrict__ codes, int64_t ldc,
                                                                float *__restrict__ scales) {
  __shared__ float s_top[16];
  const int64_t row = blockIdx.x;
  float top = 0.f;
  bool bad = false;
  for (int i = threadIdx.x * 8; i < cols; i += 8192) {
    Oct<TY> v;
    v.load(x, row * ldx + i, cols - i);
    oct_max(v, &top, &bad);
  }
  const RowScale r = row_scale<16>(top, bad, s_top);
  for (int i = threadIdx.x * 8; i < cols; i += 8192) {
    Oct<TY> v;
    v.load(x, row * ldx + i, cols - i);
    store_codes(codes + row * ldc + i, oct_codes(v, r), cols - i);
  }
  if (threadIdx.x == 0) scales[row] = r.scale;
}

constexpr int32_t kMaxBlocks = (1 << 22) - 1;     // of 1024 threads: a launch has fewer than 2^32

template <int TY, int NT, int CH>
static void launch_rows(const void *x, int64_t ldx, int32_t rows, int32_t cols, int8_t *codes, int64_t ldc, float *scales,
                        hipStream_t s) {
  constexpr int RW = NT == 64 ? 4 : 1;
  hipLaunchKernelGGL((quantize_i8_kernel<TY, NT, CH>), dim3((unsigned)((rows + RW - 1) / RW)), dim3(NT * RW), 0, s, x, ldx, rows,
                     cols, codes, ldc, scales);
}

template <int TY>
static void launch_type(const void *x, int64_t ldx, int32_t rows, int32_t cols, int8_t *codes, int64_t ldc, float *scales,
                        hipStream_t s) {
  if (cols <= 512) launch_rows<TY, 64, 1>(x, ldx, rows, cols, codes, ldc, scales, s);
  else if (cols <= 1024) launch_rows<TY, 64, 2>(x, ldx, rows, cols, codes, ldc, scales, s);
  else if (cols <= 2048) launch_rows<TY, 256, 1>(x, ldx, rows, cols, codes, ldc, scales, s);
  else if (cols <= 4096) launch_rows<TY, 512, 1>(x, ldx, rows, cols, codes, ldc, scales, s);
  else if (cols <= 8192) launch_rows<TY, 512, 2>(x, ldx, rows, cols, codes, ldc, scales, s);
  else if (cols <= 16384) launch_rows<TY, 1024, 2>(x, ldx, rows, cols, codes, ldc, scales, s);
  else
    hipLaunchKernelGGL(quantize_i8_long_kernel<TY>, dim3((unsigned)rows), dim3(1024), 0, s, x, ldx, cols, codes, ldc, scales);
}

moeq_status launch_quantize_i8(const void *x, int64_t ldx, int32_t rows, int32_t cols, int32_t dtype, int8_t *codes,
                               int64_t ldc, float *scales, hipStream_t s) {
  if (rows == 0) return MOEQ_OK;
  if (rows > kMaxBlocks) return fail(MOEQ_ERR_UNSUPPORTED, "quantize_i8: %d rows above %d", rows, kMaxBlocks);
  prof_begin("quantize_i8", s);
  if (dtype == MOEQ_F16) launch_type<MOEQ_F16>(x, ldx, rows, cols, codes, ldc, scales, s);
  else if (dtype == MOEQ_BF16) launch_type<MOEQ_BF16>(x, ldx, rows, cols, codes, ldc, scales, s);
  else launch_type<MOEQ_F32>(x, ldx, rows, cols, codes, ldc, scales, s);
  prof_end("quantize_i8", s);
  return check_launch("quantize_i8");
}

}  // namespace moeq
