// Launchers of the products of gemm.hpp, one source file per element type.
#pragma once
#include "gemm.hpp"

namespace moeq {

moeq_status launch_gemm_f16(const GemmArgs &a, GemmMode mode, hipStream_t s);
moeq_status launch_gemm_bf16(const GemmArgs &a, GemmMode mode, hipStream_t s);
moeq_status launch_gemm_i8(const GemmArgs &a, hipStream_t s);

// Workgroups of a launch with tiles of BI x BJ: row tiles are bounded by one
// partial tile per expert that has rows.
template <int MODE, int BI, int BJ>
int64_t tile_grid(const GemmArgs &a) {
  const int64_t n_it = (a.ni + BI - 1) / BI;
  const int64_t n_jt = MODE == kMats ? (int64_t)a.E * ((a.nj + BJ - 1) / BJ) : a.P / BJ + std::min(a.E, a.P);
  return (n_it * n_jt + 7) / 8 * 8;
}
constexpr int64_t kMaxGrid = 0x7fffff00 / 512;   // (threads of a launch fit 32 bits)

template <int TY, int MODE, int BI, int BJ, int WI, int WJ, bool DMA>
moeq_status launch_tiles(const GemmArgs &a, hipStream_t s, const char *name) {
  const int64_t grid = tile_grid<MODE, BI, BJ>(a);
  if (grid > kMaxGrid) return fail(MOEQ_ERR_UNSUPPORTED, "%s: too many tiles", name);
  prof_begin(name, s);
  hipLaunchKernelGGL((gemm_tile_kernel<TY, MODE, BI, BJ, WI, WJ, DMA, DMA>), dim3((unsigned)grid), dim3(64 * WI * WJ),
                     (tile_lds<MODE, BI, BJ, WI * WJ, DMA>()), s, a);
  prof_end(name, s);
  return check_launch(name);
}

// Whether the operands can be moved by DMA: 16-byte aligned bases and rows
// (and matrices), whole 16-byte pieces along a contiguous r, and 32-bit
// offsets over a tile's rows, or over all source rows where they are
// gathered.
template <int TY, int MODE>
bool dma_ok(const GemmArgs &a) {
  constexpr int ES = Elt<TY>::size;
  const int64_t lim = 0x7fffffff;
  if (((uintptr_t)a.I | (uintptr_t)a.J) & 15) return false;
  if (a.ldi * ES % 16 || a.ldj * ES % 16 || a.e_i * ES % 16) return false;
  if (MODE != kMats && (int64_t)a.nr * ES % 16) return false;
  if (256 * a.ldi * ES > lim || 256 * a.ldj * ES > lim) return false;
  if (MODE == kMats) return (int64_t)a.T * a.ldi * ES <= lim;
  return !a.pairs || (int64_t)a.T * a.ldj * ES <= lim;
}

template <int TY, int MODE>
moeq_status launch_mode(const GemmArgs &a, hipStream_t s, const char *name) {
  if (!dma_ok<TY, MODE>(a)) return launch_tiles<TY, MODE, 128, 128, 2, 2, false>(a, s, name);
  if (tile_grid<MODE, 256, 256>(a) >= 256) return launch_tiles<TY, MODE, 256, 256, 2, 4, true>(a, s, name);
  return launch_tiles<TY, MODE, 128, 128, 2, 2, true>(a, s, name);
}

template <int TY>
moeq_status launch_gemm_16bit(const GemmArgs &a, GemmMode mode, hipStream_t s) {
  switch (mode) {
    case kFwd: return launch_mode<TY, kFwd>(a, s, "grouped_gemm");
    case kRows: return launch_mode<TY, kRows>(a, s, "grouped_gemm_trans");
    default: return launch_mode<TY, kMats>(a, s, "grouped_wgrad");
  }
}

}  // namespace moeq
