// Launchers of the products of gemm.hpp, one source file per element type.
#pragma once
#include "gemm.hpp"

namespace moeq {

moeq_status launch_gemm_f16(const GemmArgs &a, GemmMode mode, hipStream_t s);
moeq_status launch_gemm_bf16(const GemmArgs &a, GemmMode mode, hipStream_t s);
moeq_status launch_gemm_i8(const GemmArgs &a, hipStream_t s);

constexpr int64_t kMaxGrid = 0x7fffff00 / 512;   // (threads of a launch fit 32 bits)

// Workgroups of a launch with tiles of BI x BJ: row tiles are bounded by one
// partial tile per expert that has rows.
template <int MODE>
int64_t tile_grid(const GemmArgs &a, int BI, int BJ) {
  const int64_t n_it = (a.ni + BI - 1) / BI;
  if constexpr (MODE == kMats) {                 // whole rounds of runs on the 8 XCDs
    const int64_t all = n_it * ((a.nj + BJ - 1) / BJ) * a.E;
    if (all > kMaxGrid) return all;
    const int run = 8 * mats_run((int)all, BI, BJ);
    return (all + run - 1) / run * run;
  }
  const int64_t n_jt = a.P / BJ + std::min(a.E, a.P);
  return (n_it * n_jt + 7) / 8 * 8;
}

template <int TY, int MODE, int BI, int BJ, int WI, int WJ, int RI, int RJ, bool DMA>
moeq_status launch_tiles(const GemmArgs &a, hipStream_t s, const char *name) {
  const int64_t grid = tile_grid<MODE>(a, BI, BJ);
  if (grid > kMaxGrid) return fail(MOEQ_ERR_UNSUPPORTED, "%s: too many tiles", name);
  prof_begin(name, s);
  hipLaunchKernelGGL((gemm_tile_kernel<TY, MODE, BI, BJ, WI, WJ, RI, RJ, DMA>), dim3((unsigned)grid), dim3(64 * WI * WJ),
                     (tile_lds<MODE, BI, BJ, RI, RJ, DMA>()), s, a);
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

// The tile: as large as the mean rows of an expert fill and as leaves about
// one workgroup per CU.  Larger tiles read the operands less often (8 experts
// of 1000 rows, K 4096, N 14336, bf16: 256 x 256 716 us, 128 x 128 989, 128
// x 64 1323, 64 x 64 1629), smaller ones spend less on rows that do not
// exist and spread few rows over more CUs (one matrix of 4096 x 4096: 200
// rows 64 x 32 22 us, 128 x 128 30; 64 rows of each expert above: 128 x 64
// 176, 128 x 128 183, 256 x 256 220).  Small tiles take a longer ring where
// rows are long or workgroups few, so that a workgroup does not wait for
// every stage (8 experts of 14336 x 4096, 4 rows each: 153 us with four
// stages, 203 with two; 16 experts of 120 rows, K 1000, N 760: 10.3 us with
// three, 12.5 with two); else more workgroups per CU are better (128 experts
// of 512 x 768, one row each: 20 us with four, 18 with two).
// Where 64 x 32 gives fewer workgroups than CUs, tiles of 32 x 16 and a ring
// of eight (bf16, one row, a matrix of 4096 x 4096: 19.0 -> 13.9 us, of 4096 x
// 14336 58.5 -> 39.8; 64 rows, 4096 x 4096 19.5 -> 17.4; rows of no alignment,
// 4097 x 4097, one 53 -> 46, 32 58 -> 48); with more workgroups it is slower
// (8 experts of 14336 x 4096, 4 rows each: 153 -> 163 us).
// Through registers (rows that are not 16-byte aligned) the largest tile has
// no room: 128 x 128 at most.
constexpr int kFewTiles = 200;
constexpr int kLongRow = 4096;     // bytes
constexpr int kFewPerCu = 512;     // workgroups: two per CU
constexpr int kCus = 256;

template <int TY, int MODE>
moeq_status launch_mode(const GemmArgs &a, hipStream_t s, const char *name) {
  const int rows = a.P / a.E + (a.P % a.E != 0);       // mean rows per expert
  const bool wide = MODE == kMats || (rows >= 80 && tile_grid<MODE>(a, 128, 128) >= kFewTiles);
  const bool tiny = MODE == kFwd && tile_grid<MODE>(a, 64, 32) < kCus;
  if (!dma_ok<TY, MODE>(a)) {
    if (wide) return launch_tiles<TY, MODE, 128, 128, 4, 2, 2, 2, false>(a, s, name);
    if constexpr (MODE == kRows) return launch_tiles<TY, MODE, 128, 64, 4, 2, 2, 2, false>(a, s, name);
    if constexpr (MODE == kFwd) {
      if (tiny) return launch_tiles<TY, MODE, 32, 16, 2, 1, 2, 2, false>(a, s, name);
      if (rows >= 16 && tile_grid<MODE>(a, 128, 64) >= kFewTiles) return launch_tiles<TY, MODE, 128, 64, 4, 2, 2, 2, false>(a, s, name);
      return launch_tiles<TY, MODE, 64, 32, 4, 1, 2, 2, false>(a, s, name);
    }
  }
  if constexpr (MODE == kMats) {
    // (here the outputs are most of the traffic: the larger tile is better
    // wherever the extents fill it and there are tiles for all CUs.  Few small
    // experts leave CUs idle with either tile, since r is not split: two of
    // 512 x 512, 16384 rows, are 8 workgroups and take 177 us)
    if (std::min(a.ni, a.nj) > 128) return launch_tiles<TY, MODE, 256, 256, 2, 4, 2, 2, true>(a, s, name);
    return launch_tiles<TY, MODE, 128, 128, 4, 2, 2, 2, true>(a, s, name);
  } else {
    constexpr int BI = MODE == kRows ? 128 : 64;       // (transposing reads need 128 columns)
    const bool longrow = (int64_t)a.nr * Elt<TY>::size >= kLongRow;
    const auto deep = [&](int bi, int bj) { return longrow || tile_grid<MODE>(a, bi, bj) < kFewPerCu; };
    if (rows >= 160 && tile_grid<MODE>(a, 256, 256) >= kFewTiles)
      return launch_tiles<TY, MODE, 256, 256, 2, 4, 3, 2, true>(a, s, name);
    if (wide) {
      if (deep(128, 128)) return launch_tiles<TY, MODE, 128, 128, 4, 2, 3, 3, true>(a, s, name);
      return launch_tiles<TY, MODE, 128, 128, 4, 2, 2, 2, true>(a, s, name);
    }
    if (rows >= 40 && tile_grid<MODE>(a, 128, 64) >= kFewTiles) {
      if (deep(128, 64)) return launch_tiles<TY, MODE, 128, 64, 4, 2, 3, 3, true>(a, s, name);
      return launch_tiles<TY, MODE, 128, 64, 4, 2, 2, 2, true>(a, s, name);
    }
    if constexpr (MODE == kFwd) {
      if (tiny) return launch_tiles<TY, MODE, 32, 16, 2, 1, 8, 8, true>(a, s, name);
    }
    if (deep(BI, 32)) return launch_tiles<TY, MODE, BI, 32, 4, 1, 4, 4, true>(a, s, name);
    return launch_tiles<TY, MODE, BI, 32, 4, 1, 2, 2, true>(a, s, name);
  }
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
