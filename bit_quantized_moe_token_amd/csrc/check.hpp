// Checks of the arguments that several entry points share (host).
#pragma once
#include "common.hpp"

namespace moeq {

constexpr int kI8 = 3;                   // element type of 8-bit codes, beside the moeq_dtype values
constexpr int32_t kMaxLen = 1 << 20;     // row length of an operand
constexpr int32_t kMaxRows = 1 << 29;    // sorted rows: 4 bytes of pair id each within 31 bits
constexpr int32_t kMaxTokens = (1 << 22) - 1;   // a workgroup of up to 1024 threads each: a grid below 2^32 threads

inline int elt_size(int dtype) { return dtype == MOEQ_F32 ? 4 : dtype == kI8 ? 1 : 2; }

inline moeq_status check_len(const char *who, const char *name, int32_t n, int32_t most) {
  if (n < 1) return fail(MOEQ_ERR_INVALID, "%s: %s=%d must be positive", who, name, n);
  if (n > most) return fail(MOEQ_ERR_UNSUPPORTED, "%s: %s=%d above %d", who, name, n, most);
  return MOEQ_OK;
}

// A matrix operand: present, aligned to its elements, rows at least `cols`
// apart and below 2^31 elements.
inline moeq_status check_matrix(const char *who, const char *name, const void *p, int64_t ld, int64_t cols, int dtype) {
  if (!p) return fail(MOEQ_ERR_INVALID, "%s: null %s", who, name);
  if ((uintptr_t)p & (uintptr_t)(elt_size(dtype) - 1))
    return fail(MOEQ_ERR_INVALID, "%s: %s is not aligned to its elements", who, name);
  if (ld < cols)
    return fail(MOEQ_ERR_INVALID, "%s: row stride %lld of %s below its %lld columns", who, (long long)ld, name, (long long)cols);
  if (ld > 0x7fffffff) return fail(MOEQ_ERR_UNSUPPORTED, "%s: row stride of %s above 2^31 - 1", who, name);
  return MOEQ_OK;
}

// E matrices of `rows` rows `ld` apart: far enough from each other (only
// outputs; inputs may repeat a matrix with stride 0), and addressable.
inline moeq_status check_stride(const char *who, const char *name, int64_t stride, int64_t rows, int64_t ld, int64_t cols,
                                int32_t E, bool output) {
  if (stride < 0) return fail(MOEQ_ERR_INVALID, "%s: negative stride of %s", who, name);
  if (output && E > 1 && stride < (rows - 1) * ld + cols)
    return fail(MOEQ_ERR_INVALID, "%s: matrices of %s overlap", who, name);
  if (stride > ((int64_t)1 << 52)) return fail(MOEQ_ERR_UNSUPPORTED, "%s: stride of %s too large", who, name);
  return MOEQ_OK;
}

inline bool ok16(int dtype) { return dtype == MOEQ_F16 || dtype == MOEQ_BF16; }
inline bool okout(int dtype) { return ok16(dtype) || dtype == MOEQ_F32; }

}  // namespace moeq

// Returns from the calling entry point with a failed check's status.
#define MOEQ_TRY(e) do { const moeq_status st_ = (e); if (st_ != MOEQ_OK) return st_; } while (0)
