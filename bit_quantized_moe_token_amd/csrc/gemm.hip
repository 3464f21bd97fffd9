// Host side of the expert-sorted products in 16 and 8 bits: argument checks
// and dispatch (kernels in gemm.hpp, quant_i8.hip).
#include "check.hpp"
#include "gemm_kernels.hpp"
#include "quant_i8.hpp"

using namespace moeq;

namespace {

constexpr int32_t kMaxI8K = 131071;      // 128^2 K stays within 31 bits

moeq_status check_groups(const char *who, const moeq_groups *g) {
  if (!g) return fail(MOEQ_ERR_INVALID, "%s: null groups", who);
  if (g->E < 1 || g->E > 256) return fail(MOEQ_ERR_INVALID, "%s: E=%d not in 1..256", who, g->E);
  if (g->P < 0 || g->T < 0) return fail(MOEQ_ERR_INVALID, "%s: negative P=%d or T=%d", who, g->P, g->T);
  if (g->P > kMaxRows) return fail(MOEQ_ERR_UNSUPPORTED, "%s: P=%d above %d", who, g->P, kMaxRows);
  if (g->P && !g->T) return fail(MOEQ_ERR_INVALID, "%s: P=%d rows without source rows", who, g->P);
  if (!g->offsets && g->E != 1) return fail(MOEQ_ERR_INVALID, "%s: no offsets with E=%d", who, g->E);
  if (g->pairs && g->k < 1) return fail(MOEQ_ERR_INVALID, "%s: k=%d must be positive", who, g->k);
  if (!g->pairs && g->T < g->P) return fail(MOEQ_ERR_INVALID, "%s: T=%d source rows for P=%d rows", who, g->T, g->P);
  if (((uintptr_t)g->offsets | (uintptr_t)g->pairs) & 3)
    return fail(MOEQ_ERR_INVALID, "%s: offsets and pairs must be 4-byte aligned", who);
  return MOEQ_OK;
}

GemmArgs base_args(const moeq_groups *g) {
  GemmArgs a{};
  a.off = g->offsets;
  a.pairs = g->pairs;
  a.E = g->E;
  a.P = g->P;
  a.T = g->T;
  a.kdiv = g->pairs ? (uint32_t)g->k : 1u;
  if (a.kdiv > 1) {     // see pair_row
    int L = 1;
    while ((1ull << L) < a.kdiv) ++L;
    a.kmul = (uint32_t)((1ull << (31 + L)) / a.kdiv + 1);
    a.kshift = L - 1;
  }
  return a;
}

moeq_status check_i8(const char *who, const moeq_groups *g, const void *x, int64_t ldx, int32_t x_dtype,
                     const int8_t *wq, int64_t ldw, int64_t stride_w, const float *sw, int32_t N, int32_t K,
                     const void *y, int64_t ldy, int32_t y_dtype) {
  MOEQ_TRY(check_groups(who, g));
  MOEQ_TRY(check_len(who, "N", N, kMaxLen));
  MOEQ_TRY(check_len(who, "K", K, kMaxI8K));
  if (!okout(y_dtype)) return fail(MOEQ_ERR_INVALID, "%s: bad y_dtype %d", who, y_dtype);
  if (!g->P) return MOEQ_OK;
  MOEQ_TRY(check_matrix(who, "x", x, ldx, K, x_dtype));
  MOEQ_TRY(check_matrix(who, "wq", wq, ldw, K, kI8));
  MOEQ_TRY(check_stride(who, "wq", stride_w, N, ldw, K, g->E, false));
  MOEQ_TRY(check_matrix(who, "y", y, ldy, N, y_dtype));
  if (!sw || ((uintptr_t)sw & 3)) return fail(MOEQ_ERR_INVALID, "%s: null or misaligned sw", who);
  return MOEQ_OK;
}

moeq_status run_i8(const moeq_groups *g, const int8_t *xq, int64_t ldx, const float *sx, const int8_t *wq, int64_t ldw,
                   int64_t stride_w, const float *sw, int32_t N, int32_t K, void *y, int64_t ldy, int32_t y_dtype,
                   hipStream_t stream) {
  GemmArgs a = base_args(g);
  a.I = (const uint8_t *)wq;
  a.J = (const uint8_t *)xq;
  a.out = y;
  a.si = sw;
  a.sj = sx;
  a.ldi = ldw;
  a.ldj = ldx;
  a.ldo = ldy;
  a.e_i = stride_w;
  a.ni = N;
  a.nr = K;
  a.out_type = y_dtype;
  return launch_gemm_i8(a, stream);
}

// Workspace of moeq_linear_i8: codes with rows padded to 128 bytes, then the
// scales.
int64_t code_ld(int32_t K) { return ((int64_t)K + 127) / 128 * 128; }

}  // namespace

MOEQ_API moeq_status moeq_grouped_gemm(const moeq_groups *g, const void *x, int64_t ldx, const void *w, int64_t ldw,
                                       int64_t stride_w, int32_t trans, int32_t N, int32_t K, int32_t dtype, void *y,
                                       int64_t ldy, int32_t y_dtype, hipStream_t stream) {
  const char *who = "grouped_gemm";
  MOEQ_TRY(check_groups(who, g));
  MOEQ_TRY(check_len(who, "N", N, kMaxLen));
  MOEQ_TRY(check_len(who, "K", K, kMaxLen));
  if (trans != 0 && trans != 1) return fail(MOEQ_ERR_INVALID, "%s: trans=%d", who, trans);
  if (!ok16(dtype)) return fail(MOEQ_ERR_INVALID, "%s: bad dtype %d", who, dtype);
  if (y_dtype != dtype && y_dtype != MOEQ_F32) return fail(MOEQ_ERR_INVALID, "%s: bad y_dtype %d", who, y_dtype);
  if (!g->P) return MOEQ_OK;
  MOEQ_TRY(check_matrix(who, "x", x, ldx, K, dtype));
  MOEQ_TRY(check_matrix(who, "w", w, ldw, trans ? N : K, dtype));
  MOEQ_TRY(check_stride(who, "w", stride_w, trans ? K : N, ldw, trans ? N : K, g->E, false));
  MOEQ_TRY(check_matrix(who, "y", y, ldy, N, y_dtype));
  GemmArgs a = base_args(g);
  a.I = (const uint8_t *)w;
  a.J = (const uint8_t *)x;
  a.out = y;
  a.ldi = ldw;
  a.ldj = ldx;
  a.ldo = ldy;
  a.e_i = stride_w;
  a.ni = N;
  a.nr = K;
  a.out_type = y_dtype;
  const GemmMode mode = trans ? kRows : kFwd;
  return dtype == MOEQ_F16 ? launch_gemm_f16(a, mode, stream) : launch_gemm_bf16(a, mode, stream);
}

MOEQ_API moeq_status moeq_grouped_wgrad(const moeq_groups *g, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                        int32_t N, int32_t K, int32_t dtype, void *dw, int64_t lddw, int64_t stride_dw,
                                        int32_t dw_dtype, hipStream_t stream) {
  const char *who = "grouped_wgrad";
  MOEQ_TRY(check_groups(who, g));
  MOEQ_TRY(check_len(who, "N", N, kMaxLen));
  MOEQ_TRY(check_len(who, "K", K, kMaxLen));
  if (!ok16(dtype)) return fail(MOEQ_ERR_INVALID, "%s: bad dtype %d", who, dtype);
  if (dw_dtype != dtype && dw_dtype != MOEQ_F32) return fail(MOEQ_ERR_INVALID, "%s: bad dw_dtype %d", who, dw_dtype);
  if (g->P) {   // without rows the gradients are zeros and the operands are not read
    MOEQ_TRY(check_matrix(who, "dy", dy, lddy, N, dtype));
    MOEQ_TRY(check_matrix(who, "x", x, ldx, K, dtype));
  }
  MOEQ_TRY(check_matrix(who, "dw", dw, lddw, K, dw_dtype));
  MOEQ_TRY(check_stride(who, "dw", stride_dw, N, lddw, K, g->E, true));
  GemmArgs a = base_args(g);
  a.I = (const uint8_t *)x;
  a.J = (const uint8_t *)dy;
  a.out = dw;
  a.ldi = ldx;
  a.ldj = lddy;
  a.ldo = lddw;
  a.e_out = stride_dw;
  a.ni = K;
  a.nj = N;
  a.out_type = dw_dtype;
  return dtype == MOEQ_F16 ? launch_gemm_f16(a, kMats, stream) : launch_gemm_bf16(a, kMats, stream);
}

MOEQ_API moeq_status moeq_quantize_i8(const void *x, int64_t ldx, int32_t rows, int32_t cols, int32_t dtype,
                                      int8_t *codes, int64_t ldc, float *scales, hipStream_t stream) {
  const char *who = "quantize_i8";
  if (rows < 0) return fail(MOEQ_ERR_INVALID, "%s: negative rows=%d", who, rows);
  MOEQ_TRY(check_len(who, "cols", cols, kMaxLen));
  if (!okout(dtype)) return fail(MOEQ_ERR_INVALID, "%s: bad dtype %d", who, dtype);
  if (!rows) return MOEQ_OK;
  MOEQ_TRY(check_matrix(who, "x", x, ldx, cols, dtype));
  MOEQ_TRY(check_matrix(who, "codes", codes, ldc, cols, kI8));
  if (!scales || ((uintptr_t)scales & 3)) return fail(MOEQ_ERR_INVALID, "%s: null or misaligned scales", who);
  return launch_quantize_i8(x, ldx, rows, cols, dtype, codes, ldc, scales, stream);
}

MOEQ_API moeq_status moeq_gemm_i8(const moeq_groups *g, const int8_t *xq, int64_t ldx, const float *sx,
                                  const int8_t *wq, int64_t ldw, int64_t stride_w, const float *sw, int32_t N,
                                  int32_t K, void *y, int64_t ldy, int32_t y_dtype, hipStream_t stream) {
  const char *who = "gemm_i8";
  MOEQ_TRY(check_i8(who, g, xq, ldx, kI8, wq, ldw, stride_w, sw, N, K, y, ldy, y_dtype));
  if (!g->P) return MOEQ_OK;
  if (!sx || ((uintptr_t)sx & 3)) return fail(MOEQ_ERR_INVALID, "%s: null or misaligned sx", who);
  return run_i8(g, xq, ldx, sx, wq, ldw, stride_w, sw, N, K, y, ldy, y_dtype, stream);
}

MOEQ_API moeq_status moeq_linear_i8_workspace_size(int32_t T, int32_t K, size_t *bytes) {
  const char *who = "linear_i8_workspace_size";
  if (!bytes) return fail(MOEQ_ERR_INVALID, "%s: null bytes", who);
  if (T < 0) return fail(MOEQ_ERR_INVALID, "%s: negative T=%d", who, T);
  MOEQ_TRY(check_len(who, "K", K, kMaxI8K));
  *bytes = (size_t)T * (size_t)(code_ld(K) + 4);
  return MOEQ_OK;
}

MOEQ_API moeq_status moeq_linear_i8(const moeq_groups *g, const void *x, int64_t ldx, int32_t dtype, const int8_t *wq,
                                    int64_t ldw, int64_t stride_w, const float *sw, int32_t N, int32_t K, void *y,
                                    int64_t ldy, int32_t y_dtype, void *ws, size_t ws_bytes, hipStream_t stream) {
  const char *who = "linear_i8";
  if (!okout(dtype)) return fail(MOEQ_ERR_INVALID, "%s: bad dtype %d", who, dtype);
  MOEQ_TRY(check_i8(who, g, x, ldx, dtype, wq, ldw, stride_w, sw, N, K, y, ldy, y_dtype));
  if (!g->P) return MOEQ_OK;
  const size_t need = (size_t)g->T * (size_t)(code_ld(K) + 4);
  if (need && (!ws || ((uintptr_t)ws & 15))) return fail(MOEQ_ERR_INVALID, "%s: null or misaligned workspace", who);
  if (ws_bytes < need) return fail(MOEQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, ws_bytes, need);
  int8_t *q = (int8_t *)ws;
  float *sx = (float *)(q + (size_t)g->T * (size_t)code_ld(K));
  MOEQ_TRY(launch_quantize_i8(x, ldx, g->T, K, dtype, q, code_ld(K), sx, stream));
  return run_i8(g, q, code_ld(K), sx, wq, ldw, stride_w, sw, N, K, y, ldy, y_dtype, stream);
}
