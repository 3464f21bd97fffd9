// Launchers of the products of gemm.hpp, one source file per element type.
#pragma once
#include "gemm.hpp"

namespace moeq {

moeq_status launch_gemm_f16(const GemmArgs &a, GemmMode mode, hipStream_t s);
moeq_status launch_gemm_bf16(const GemmArgs &a, GemmMode mode, hipStream_t s);
moeq_status launch_gemm_i8(const GemmArgs &a, hipStream_t s);

template <int TY, int MODE, int BI, int BJ, int WI, int WJ>
moeq_status launch_staged(const GemmArgs &a, hipStream_t s, const char *name) {
  const int64_t n_it = (a.ni + BI - 1) / BI;
  // row tiles: at most one partial tile per expert that has rows
  const int64_t n_jt = MODE == kMats ? (int64_t)a.E * ((a.nj + BJ - 1) / BJ) : a.P / BJ + std::min(a.E, a.P);
  const int64_t grid = (n_it * n_jt + 7) / 8 * 8;
  if (grid > 0x7fffff00) return fail(MOEQ_ERR_UNSUPPORTED, "%s: too many tiles", name);
  prof_begin(name, s);
  hipLaunchKernelGGL((gemm_staged_kernel<TY, MODE, BI, BJ, WI, WJ>), dim3((unsigned)grid), dim3(64 * WI * WJ),
                     2 * (BI + BJ) * kStepBytes, s, a);
  prof_end(name, s);
  return check_launch(name);
}

template <int TY>
moeq_status launch_gemm_16bit(const GemmArgs &a, GemmMode mode, hipStream_t s) {
  switch (mode) {
    case kFwd: return launch_staged<TY, kFwd, 128, 128, 2, 2>(a, s, "grouped_gemm");
    case kRows: return launch_staged<TY, kRows, 128, 128, 2, 2>(a, s, "grouped_gemm_trans");
    default: return launch_staged<TY, kMats, 128, 128, 2, 2>(a, s, "grouped_wgrad");
  }
}

}  // namespace moeq
