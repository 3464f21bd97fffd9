// Products of expert-sorted rows with one matrix per expert, in 16-bit
// floating point and in 8-bit integers ([MxMoE] abstract: linear blocks of
// one layer at different precisions, uneven expert activation; these are
// the blocks that stay in 16 or 8 bits beside the low-bit ones).
//
// One problem serves the three products.  out[j][i] = sum_r I[i][r] J[j][r]
// over a reduction index r, where i is the contiguous index of the output:
//   forward   i = output channel n (rows of W_e),     j = sorted row,  r = input channel
//   rows'     i = input channel (columns of W_e),     j = sorted row,  r = output channel
//   gradient    (W_e is stored with r as its row index)
//   matrices' i = input channel (columns of x),       j = output channel (columns of dy),
//   gradient    r = the expert's rows (both operands store r as the row index)
// The MFMA takes I as its first operand, so a lane ends with four
// consecutive i of one j: outputs leave in 8- or 16-byte stores.
#pragma once
#include "common.hpp"

namespace moeq {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kI8 = 3;   // element type of the 8-bit products, beside MOEQ_F16 and MOEQ_BF16

enum GemmMode { kFwd = 0, kRows = 1, kMats = 2 };   // see above

struct GemmArgs {
  const uint8_t *I, *J;      // operands (bytes; element type of the kernel)
  void *out;
  const int32_t *off;        // [E + 1] first sorted row of each expert, or null: one expert, all P rows
  const int32_t *pairs;      // [P] pair ids (source row = pair / kdiv), or null: source row = sorted row
  const float *si, *sj;      // 8-bit: scale per (expert, i) and per source row
  int64_t ldi, ldj, ldo;     // elements between rows of I, J and out
  int64_t e_i, e_out;        // elements between experts' matrices in I and (gradient) in out
  int32_t E, P, T;           // experts, sorted rows, source rows
  uint32_t kdiv;
  int32_t ni, nj, nr;        // extents of i, j (kMats only) and r (not kMats)
  int32_t out_type;          // moeq_dtype
  int32_t out_vec;           // out rows and base allow stores of four elements
};

template <int TY>
struct Elt;
template <>
struct Elt<MOEQ_F16> {
  using acc = f32x4;
  static constexpr int size = 2;
  static __device__ __forceinline__ acc mma(u32x4 a, u32x4 b, acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Elt<MOEQ_BF16> {
  using acc = f32x4;
  static constexpr int size = 2;
  static __device__ __forceinline__ acc mma(u32x4 a, u32x4 b, acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Elt<kI8> {
  using acc = i32x4;
  static constexpr int size = 1;
  static __device__ __forceinline__ acc mma(u32x4 a, u32x4 b, acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};

// A tile step covers 128 bytes of every row along r: 64 elements of 16 bits,
// 128 of 8.  An MFMA consumes 64 of them (16 bytes per lane), two per step.
constexpr int kStepBytes = 128;

// First and one-past-last sorted row of expert e, within [0, P] whatever the
// offsets hold.
__device__ __forceinline__ void expert_rows(const GemmArgs &a, int e, int *lo, int *hi) {
  if (!a.off) {
    *lo = 0;
    *hi = a.P;
    return;
  }
  const int l = std::min(std::max(a.off[e], 0), a.P);
  *lo = l;
  *hi = std::min(std::max(a.off[e + 1], l), a.P);
}

// Source row of sorted row r; -1 (a row of zeros) when it lies outside [0, T).
__device__ __forceinline__ int source_row(const GemmArgs &a, int r) {
  uint32_t s = (uint32_t)r;
  if (a.pairs) {
    s = (uint32_t)a.pairs[r];
    if (a.kdiv != 1) s /= a.kdiv;
  }
  return s < (uint32_t)a.T ? (int)s : -1;
}

// Output tile of a workgroup: expert, first sorted row and rows left in the
// expert from there, first i.
struct Tile {
  int e, row, rows, i0;
};

// Workgroup -> tile.  Tiles are numbered expert by expert, within an expert
// in bands of kBand row tiles (all i tiles of a band before the next), so
// that workgroups that run together share rows and columns; each of the 8
// XCDs (workgroups are dealt to them in turn) gets a contiguous run of the
// numbering, for its own L2.  The count of row tiles is known only on the
// device: workgroups beyond it return false.
constexpr int kBand = 8;
template <int BJ>
__device__ __forceinline__ bool find_tile(const GemmArgs &a, int BI, Tile *t) {
  const int lane = threadIdx.x & 63;
  const int n_it = (a.ni + BI - 1) / BI;
  int total = 0;   // row tiles of all experts
  for (int b = 0; b < a.E; b += kWave) {
    int nc = 0, lo, hi;
    if (b + lane < a.E) {
      expert_rows(a, b + lane, &lo, &hi);
      nc = (hi - lo + BJ - 1) / BJ;
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) nc += __shfl_xor(nc, o, kWave);
    total += nc;
  }
  const int all = total * n_it, per = (all + 7) >> 3;
  const int idx = (int)blockIdx.x >> 3, L = ((int)blockIdx.x & 7) * per + idx;
  if (idx >= per || L >= all) return false;
  int carry = 0;
  for (int b = 0; b < a.E; b += kWave) {
    int nc = 0, lo = 0, hi = 0;
    if (b + lane < a.E) {
      expert_rows(a, b + lane, &lo, &hi);
      nc = (hi - lo + BJ - 1) / BJ;
    }
    int incl = nc;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
    }
    const int excl = carry + incl - nc;
    const uint64_t hit = __ballot(L >= excl * n_it && L < (excl + nc) * n_it);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      const int ex = __builtin_amdgcn_readfirstlane(__shfl(excl, src, kWave));
      const int n = __builtin_amdgcn_readfirstlane(__shfl(nc, src, kWave));
      const int l = __builtin_amdgcn_readfirstlane(__shfl(lo, src, kWave));
      const int h = __builtin_amdgcn_readfirstlane(__shfl(hi, src, kWave));
      const int local = L - ex * n_it, band = local / (kBand * n_it);
      const int in = local - band * kBand * n_it, width = std::min(kBand, n - band * kBand);
      const int jt = band * kBand + in % width;
      t->e = b + src;
      t->row = l + jt * BJ;
      t->rows = h - t->row;
      t->i0 = in / width * BI;
      return true;
    }
    carry += __builtin_amdgcn_readfirstlane(__shfl(incl, 63, kWave));
  }
  return false;
}

// 16 bytes at p of which the first n (elements of ES bytes) exist, the rest
// zero.  p need only be aligned to an element.
template <int ES>
__device__ __forceinline__ u32x4 load_piece(const uint8_t *p, int64_t n) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (n >= 16) {
    struct __attribute__((packed, aligned(ES))) Raw { u32x4 v; };
    return ((const __attribute__((address_space(1))) Raw *)p)->v;
  }
  if (n > 0) {
#pragma unroll
    for (int b = 0; b < 16; b += ES)
      if (b < n) {
        const uint32_t x = ES == 2 ? (uint32_t)gld<uint16_t>(p + b) : (uint32_t)gld<uint8_t>(p + b);
        v[b / 4] |= x << (8 * (b & 3));
      }
  }
  return v;
}

// ---- LDS layout of an operand tile of R rows (i or j) x 128 bytes of r,
// 128 R bytes, moved in blocks of 1 KiB (16 bytes per lane).
//
// Operand stored with r contiguous: row after row, 128 bytes each; the
// 16-byte piece c of row x sits in slot c ^ ((x / 2) % 8), so that the 16
// rows that an MFMA operand read touches (one piece each) cover all 64 banks
// once.
//
// Operand stored with r as the row index (16-bit only): 64 rows of r, R
// elements each; 32-byte pieces are permuted within each 256 bytes by
// XOR with kmaj_swz(r), so that the rows of a transposing read (four of
// 32 bytes per 16 lanes) fall into different banks.
__device__ __forceinline__ int kmaj_swz(int r) { return (r & 3) | ((r >> 1) & 4); }

// Fragment reads.  Lane l of an MFMA operand holds element l % 16 of the
// 16-wide tile and 16 bytes of r (piece l / 16 of the step half s).
template <int R, bool RMAJ>
struct FragReader {
  uint32_t base[2];
  __device__ __forceinline__ FragReader(uint32_t tile_base) {
    const int l = threadIdx.x & 63, g = l >> 4, x = l & 15;
    if constexpr (!RMAJ) {
#pragma unroll
      for (int s = 0; s < 2; ++s) base[s] = tile_base + x * 128 + 16 * ((4 * s + g) ^ (x >> 1));
    } else {
      // lane x of the 16 supplies 8 bytes of row r = 8 g + x / 4 (+ 4 for the
      // second read, + 32 for s = 1): columns 4 (x % 4) .. + 3 of the tile
      const int r = 8 * g + (x >> 2);
      base[0] = tile_base + r * (2 * R) + 8 * (x & 3) + 32 * kmaj_swz(r);
      base[1] = 0;
    }
  }
  // 16-wide tile f, step half s
  __device__ __forceinline__ u32x4 read(const uint8_t *lds, int f, int s) const {
    if constexpr (!RMAJ) {
      return *reinterpret_cast<const u32x4 *>(lds + base[s] + f * 2048);
    } else {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      const uint32_t o = (base[0] ^ (uint32_t)((f & 7) * 32)) + (f >> 3) * 256 + s * 32 * (2 * R);
      const auto p = (__attribute__((address_space(3))) s16x4 *)(lds + o);
      const auto q = (__attribute__((address_space(3))) s16x4 *)(lds + o + 4 * (2 * R));
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(q));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  }
};

// ---- Movement of an operand tile into LDS through registers: any element
// alignment and row stride, 64-bit addresses.
template <int ES, int R, int NW, bool RMAJ>
struct StagedOperand {
  static constexpr int NB = R / (8 * NW);   // 1 KiB blocks per wave
  static_assert(R % (8 * NW) == 0, "blocks per wave");
  static_assert(!RMAJ || (R % 128 == 0 && ES == 2), "256-byte swizzle groups of 16-bit elements");
  const uint8_t *p[NB];    // r contiguous: the row's first byte (null: no such row)
  int nr;                  // extent of r
  u32x4 v[NB];

  __device__ __forceinline__ static int block() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * NB; }

  // r contiguous: `row(x)` gives the first byte of tile row x or null
  template <class RowPtr>
  __device__ __forceinline__ void rows(RowPtr row, int n_r) {
    nr = n_r;
#pragma unroll
    for (int i = 0; i < NB; ++i) p[i] = row((block() + i) * 8 + ((threadIdx.x & 63) >> 3));
  }
  __device__ __forceinline__ void fetch_rows(int t) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int l = threadIdx.x & 63, x = (block() + i) * 8 + (l >> 3);
      const int64_t o = (int64_t)t * kStepBytes + 16 * ((l & 7) ^ ((x >> 1) & 7));
      v[i] = load_piece<ES>(p[i] + o, p[i] ? (int64_t)nr * ES - o : 0);
    }
  }
  // r as row index: `row(r)` gives the first byte of row r (column i0) or null
  template <class RowPtr>
  __device__ __forceinline__ void fetch_cols(int t, RowPtr row, int n_cols) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int l = threadIdx.x & 63, o = (block() + i) * 1024 + l * 16;
      const int r = o / (2 * R), s = (o % (2 * R)) / 16;
      const int c = 16 * (s ^ (2 * kmaj_swz(r)));      // byte column of the piece
      const uint8_t *q = row(t * 64 + r);
      v[i] = load_piece<ES>(q + c, q ? (int64_t)n_cols * ES - c : 0);
    }
  }
  __device__ __forceinline__ void store(uint8_t *tile) const {
#pragma unroll
    for (int i = 0; i < NB; ++i)
      *reinterpret_cast<u32x4 *>(tile + (block() + i) * 1024 + (threadIdx.x & 63) * 16) = v[i];
  }
};

// ---- output
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint16_t f16_bits(float v) { return __builtin_bit_cast(uint16_t, (f16)v); }

// Four consecutive elements at index o of which n exist, each rounded once.
__device__ __forceinline__ void store4(const GemmArgs &a, int64_t o, f32x4 v, int n) {
  if (a.out_type == MOEQ_F32) {
    float *p = (float *)a.out + o;
    if (a.out_vec && n >= 4) *reinterpret_cast<f32x4 *>(p) = v;
    else {
#pragma unroll
      for (int i = 0; i < 4; ++i) if (i < n) p[i] = v[i];
    }
    return;
  }
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = a.out_type == MOEQ_BF16 ? bf16_bits(v[i]) : f16_bits(v[i]);
  uint16_t *p = (uint16_t *)a.out + o;
  if (a.out_vec && n >= 4) {
    *reinterpret_cast<u32x2 *>(p) = u32x2{(uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16)};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) if (i < n) p[i] = h[i];
  }
}

// Output tile of a workgroup, the extent of r and, for the matrices'
// gradient, the first j; all in scalar registers.
template <int MODE, int BI, int BJ>
__device__ __forceinline__ bool pick_tile(const GemmArgs &a, Tile *t, int *nr, int *j0) {
  Tile v{};
  int r = a.nr, j = 0;
  if constexpr (MODE == kMats) {
    const int n_it = (a.ni + BI - 1) / BI, n_jt = (a.nj + BJ - 1) / BJ, all = a.E * n_it * n_jt;
    const int per = (all + 7) >> 3, idx = (int)blockIdx.x >> 3, L = ((int)blockIdx.x & 7) * per + idx;
    if (idx >= per || L >= all) return false;
    v.e = L / (n_it * n_jt);
    const int in = L - v.e * n_it * n_jt;
    j = in / n_it * BJ;
    v.i0 = in % n_it * BI;
    int lo, hi;
    expert_rows(a, v.e, &lo, &hi);
    v.row = lo;
    r = hi - lo;
    v.rows = a.nj - j;
  } else {
    if (!find_tile<BJ>(a, BI, &v)) return false;
  }
  t->e = __builtin_amdgcn_readfirstlane(v.e);
  t->row = __builtin_amdgcn_readfirstlane(v.row);
  t->rows = __builtin_amdgcn_readfirstlane(v.rows);
  t->i0 = __builtin_amdgcn_readfirstlane(v.i0);
  *nr = __builtin_amdgcn_readfirstlane(r);
  *j0 = __builtin_amdgcn_readfirstlane(j);
  return true;
}

// Writes the wave's TI x TJ accumulators (tiles of 16 x 16 from ib, jb).
template <int TY, int MODE, int TI, int TJ>
__device__ __forceinline__ void write_tile(const GemmArgs &a, const Tile &t, int j0, int ib, int jb,
                                           const typename Elt<TY>::acc (&acc)[TI][TJ]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int x = jb + j * 16 + (lane & 15);   // row of the tile
    if (x >= t.rows) continue;
    float sc = 1.f;
    if constexpr (TY == kI8) {
      const int s = source_row(a, t.row + x);
      sc = s >= 0 ? a.sj[s] : 0.f;
    }
    const int64_t ob = MODE == kMats ? (int64_t)t.e * a.e_out + (int64_t)(j0 + x) * a.ldo : (int64_t)(t.row + x) * a.ldo;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int c = t.i0 + ib + i * 16 + 4 * (lane >> 4);
      if (c >= a.ni) continue;
      f32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] = (float)acc[i][j][q];
        if constexpr (TY == kI8) v[q] = v[q] * sc * (c + q < a.ni ? a.si[(int64_t)t.e * a.ni + c + q] : 0.f);
      }
      store4(a, ob + c, v, a.ni - c);
    }
  }
}

// ---- tiled kernel: a workgroup of WI x WJ waves computes BI x BJ outputs.
template <int TY, int MODE, int BI, int BJ, int WI, int WJ>
__global__ void __launch_bounds__(64 * WI * WJ, 1) gemm_staged_kernel(GemmArgs a) {
  constexpr int ES = Elt<TY>::size, NW = WI * WJ, TI = BI / WI / 16, TJ = BJ / WJ / 16;
  constexpr bool RI = MODE != kFwd, RJ = MODE == kMats;
  constexpr uint32_t kTileI = BI * kStepBytes, kStage = kTileI + BJ * kStepBytes;
  using Acc = typename Elt<TY>::acc;
  extern __shared__ __attribute__((aligned(1024))) uint8_t gemm_lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave % WI, wj = wave / WI;

  Tile t;
  int nr, j0;          // extent of r; first j (kMats)
  if (!pick_tile<MODE, BI, BJ>(a, &t, &nr, &j0)) return;

  StagedOperand<ES, BI, NW, RI> si;
  StagedOperand<ES, BJ, NW, RJ> sj;
  const uint8_t *wmat = a.I + (int64_t)t.e * a.e_i * ES;   // the expert's matrix (not kMats)
  if constexpr (!RI) {
    si.rows([&](int x) { return t.i0 + x < a.ni ? wmat + (int64_t)(t.i0 + x) * a.ldi * ES : nullptr; }, nr);
  }
  if constexpr (!RJ) {
    sj.rows([&](int x) -> const uint8_t * {
      const int s = x < t.rows ? source_row(a, t.row + x) : -1;
      return s >= 0 ? a.J + (int64_t)s * a.ldj * ES : nullptr;
    }, nr);
  }
  auto fetch = [&](int k) {
    if constexpr (!RI) si.fetch_rows(k);
    else if constexpr (MODE == kRows)
      si.fetch_cols(k, [&](int r) { return r < nr ? wmat + ((int64_t)r * a.ldi + t.i0) * ES : nullptr; }, a.ni - t.i0);
    else
      si.fetch_cols(k, [&](int r) -> const uint8_t * {
        const int s = r < nr ? source_row(a, t.row + r) : -1;
        return s >= 0 ? a.I + ((int64_t)s * a.ldi + t.i0) * ES : nullptr;
      }, a.ni - t.i0);
    if constexpr (!RJ) sj.fetch_rows(k);
    else sj.fetch_cols(k, [&](int r) { return r < nr ? a.J + ((int64_t)(t.row + r) * a.ldj + j0) * ES : nullptr; }, a.nj - j0);
  };

  Acc acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = Acc{0, 0, 0, 0};
  const FragReader<BI, RI> fi(0);
  const FragReader<BJ, RJ> fj(kTileI);
  const int steps = (int)(((int64_t)nr * ES + kStepBytes - 1) / kStepBytes);
  if (steps > 0) {
    fetch(0);
    si.store(gemm_lds);
    sj.store(gemm_lds + kTileI);
  }
  for (int k = 0; k < steps; ++k) {
    if (k + 1 < steps) fetch(k + 1);
    __syncthreads();
    const uint8_t *st = gemm_lds + (k & 1) * kStage;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 x[TI], y[TJ];
#pragma unroll
      for (int i = 0; i < TI; ++i) x[i] = fi.read(st, wi * TI + i, s);
#pragma unroll
      for (int j = 0; j < TJ; ++j) y[j] = fj.read(st, wj * TJ + j, s);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = Elt<TY>::mma(x[i], y[j], acc[i][j]);
    }
    // the other stage was last read before this step's barrier
    if (k + 1 < steps) {
      si.store(gemm_lds + ((k + 1) & 1) * kStage);
      sj.store(gemm_lds + ((k + 1) & 1) * kStage + kTileI);
    }
  }

  write_tile<TY, MODE, TI, TJ>(a, t, j0, wi * TI * 16, wj * TJ * 16, acc);
}

// ---- Movement of an operand tile straight into LDS (buffer loads with an
// LDS destination): the data never occupies registers.  Rows and bases must
// be 16-byte aligned; what lies behind the buffer resource's range reads
// zero, which gives the zeros behind the last row and the last r.
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p) {   // into scalar registers
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (const uint8_t *)(((uint64_t)hi << 32) | lo);
}
constexpr uint32_t kNowhere = 0x80000000u;   // an offset behind every range used here

template <int ES, int R, int NW, bool RMAJ>
struct DmaOperand {
  static constexpr int NB = R / (8 * NW);   // 1 KiB blocks per wave
  static_assert(R % (8 * NW) == 0, "blocks per wave");
  static_assert(!RMAJ || (R % 128 == 0 && ES == 2), "256-byte swizzle groups of 16-bit elements");
  uint32_t voff[NB];       // lane's offset from the resource's base (kNowhere: no such row)
  __amdgpu_buffer_rsrc_t rs;
  const uint8_t *base;     // r as row index: row 0 at the tile's first column
  uint32_t ld, width;      // r as row index: bytes between rows, bytes of a row from the tile's first column
  int bytes;               // r contiguous: valid bytes of a row

  __device__ __forceinline__ static int block() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * NB; }
  // 16-byte piece of the row that the lane moves in block i (r contiguous)
  __device__ __forceinline__ static uint32_t piece(int i) {
    const int l = threadIdx.x & 63, x = (block() + i) * 8 + (l >> 3);
    return 16u * (uint32_t)((l & 7) ^ ((x >> 1) & 7));
  }
  // r contiguous: row(x) gives the tile row's offset from `from` or kNowhere
  template <class RowOff>
  __device__ __forceinline__ void rows(const uint8_t *from, uint32_t range, int row_bytes, RowOff row) {
    rs = make_rsrc(uniform(from), __builtin_amdgcn_readfirstlane((int)range));
    bytes = row_bytes;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const uint32_t o = row((block() + i) * 8 + ((int)(threadIdx.x & 63) >> 3));
      voff[i] = o == kNowhere ? kNowhere : o + piece(i);
    }
  }
  __device__ __forceinline__ void issue_rows(int t, uint8_t *tile) const {
    if ((t + 1) * kStepBytes <= bytes) {
#pragma unroll
      for (int i = 0; i < NB; ++i) lds_dma_buf<16>(rs, voff[i], (uint32_t)t * kStepBytes, tile + (block() + i) * 1024);
    } else {                 // the last step of a row that is no multiple of it
#pragma unroll
      for (int i = 0; i < NB; ++i)
        lds_dma_buf<16>(rs, (int)piece(i) < bytes - t * kStepBytes ? voff[i] : kNowhere, (uint32_t)t * kStepBytes,
                        tile + (block() + i) * 1024);
    }
  }
  // r as row index: row of r within the step and byte column that the lane
  // moves in block i
  __device__ __forceinline__ static int row_in(int i) { return ((block() + i) * 1024 + (int)(threadIdx.x & 63) * 16) / (2 * R); }
  __device__ __forceinline__ static uint32_t col_in(int i) {
    const int o = (block() + i) * 1024 + (int)(threadIdx.x & 63) * 16, s = (o % (2 * R)) / 16;
    return 16u * (uint32_t)(s ^ (2 * kmaj_swz(o / (2 * R))));
  }
  // consecutive rows from `from`
  __device__ __forceinline__ void cols(const uint8_t *from, int64_t row_stride, int row_bytes) {
    base = uniform(from);
    ld = (uint32_t)row_stride;
    width = (uint32_t)row_bytes;
#pragma unroll
    for (int i = 0; i < NB; ++i) voff[i] = (uint32_t)row_in(i) * ld + col_in(i);
  }
  __device__ __forceinline__ void issue_cols(int t, int nr, uint8_t *tile) const {
    const int left = std::min(64, nr - t * 64);
    const auto r = make_rsrc(uniform(base + (int64_t)t * 64 * ld), (uint32_t)(left - 1) * ld + width);
#pragma unroll
    for (int i = 0; i < NB; ++i) lds_dma_buf<16>(r, voff[i], 0, tile + (block() + i) * 1024);
  }
  // rows given one by one (gathered): src[i], or negative for a row of zeros
  __device__ __forceinline__ void gather(const uint8_t *from, uint32_t range, int64_t row_stride) {
    rs = make_rsrc(uniform(from), __builtin_amdgcn_readfirstlane((int)range));
    ld = (uint32_t)row_stride;
  }
  __device__ __forceinline__ void issue_gather(const int *src, uint8_t *tile) const {
#pragma unroll
    for (int i = 0; i < NB; ++i)
      lds_dma_buf<16>(rs, src[i] < 0 ? kNowhere : (uint32_t)src[i] * ld + col_in(i), 0, tile + (block() + i) * 1024);
  }
};

// The tiled kernel with both operands moved by DMA.  Two stages: while the
// waves multiply step k, step k + 1 is on its way; one barrier per step.
template <int TY, int MODE, int BI, int BJ, int WI, int WJ>
__global__ void __launch_bounds__(64 * WI * WJ, 1) gemm_dma_kernel(GemmArgs a) {
  constexpr int ES = Elt<TY>::size, NW = WI * WJ, TI = BI / WI / 16, TJ = BJ / WJ / 16;
  constexpr bool RI = MODE != kFwd, RJ = MODE == kMats;
  constexpr uint32_t kTileI = BI * kStepBytes, kStage = kTileI + BJ * kStepBytes;
  using Acc = typename Elt<TY>::acc;
  extern __shared__ __attribute__((aligned(1024))) uint8_t gemm_lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave % WI, wj = wave / WI;
  Tile t;
  int nr, j0;
  if (!pick_tile<MODE, BI, BJ>(a, &t, &nr, &j0)) return;

  using OpI = DmaOperand<ES, BI, NW, RI>;
  using OpJ = DmaOperand<ES, BJ, NW, RJ>;
  OpI di;
  OpJ dj;
  int src[OpI::NB];        // kMats: source rows of the next step to move
  auto sources = [&](int k) {
#pragma unroll
    for (int i = 0; i < OpI::NB; ++i) {
      const int r = k * 64 + OpI::row_in(i);
      src[i] = r < nr ? source_row(a, t.row + r) : -1;
    }
  };
  if constexpr (MODE == kMats) {
    di.gather(a.I + (int64_t)t.i0 * ES, (uint32_t)(((int64_t)(a.T - 1) * a.ldi + a.ni - t.i0) * ES), a.ldi * ES);
    dj.cols(a.J + ((int64_t)t.row * a.ldj + j0) * ES, a.ldj * ES, (a.nj - j0) * ES);
    sources(0);
  } else {
    const uint8_t *wmat = a.I + (int64_t)t.e * a.e_i * ES;   // the expert's matrix
    if constexpr (MODE == kRows) {
      di.cols(wmat + (int64_t)t.i0 * ES, a.ldi * ES, (a.ni - t.i0) * ES);
    } else {
      const int n = std::min(BI, a.ni - t.i0);
      di.rows(wmat + (int64_t)t.i0 * a.ldi * ES, (uint32_t)(((n - 1) * a.ldi + nr) * ES), nr * ES,
              [&](int x) { return x < n ? (uint32_t)x * (uint32_t)(a.ldi * ES) : kNowhere; });
    }
    if (a.pairs) {
      dj.rows(a.J, (uint32_t)(((int64_t)(a.T - 1) * a.ldj + nr) * ES), nr * ES, [&](int x) {
        const int s = x < t.rows ? source_row(a, t.row + x) : -1;
        return s >= 0 ? (uint32_t)s * (uint32_t)(a.ldj * ES) : kNowhere;
      });
    } else {
      const int n = std::min(BJ, t.rows);
      dj.rows(a.J + (int64_t)t.row * a.ldj * ES, (uint32_t)(((n - 1) * a.ldj + nr) * ES), nr * ES,
              [&](int x) { return x < n ? (uint32_t)x * (uint32_t)(a.ldj * ES) : kNowhere; });
    }
  }
  auto issue = [&](int k, uint8_t *st) {
    if constexpr (MODE == kMats) di.issue_gather(src, st);
    else if constexpr (MODE == kRows) di.issue_cols(k, nr, st);
    else di.issue_rows(k, st);
    if constexpr (RJ) dj.issue_cols(k, nr, st + kTileI);
    else dj.issue_rows(k, st + kTileI);
    if constexpr (MODE == kMats) sources(k + 1);
  };

  Acc acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = Acc{0, 0, 0, 0};
  const FragReader<BI, RI> fi(0);
  const FragReader<BJ, RJ> fj(kTileI);
  const int steps = (int)(((int64_t)nr * ES + kStepBytes - 1) / kStepBytes);
  if (steps > 0) issue(0, gemm_lds);
  uint32_t sb = 0;
#pragma unroll 1
  for (int k = 0; k < steps; ++k) {
    vm_wait<0>();
    __builtin_amdgcn_s_barrier();
    // every wave has read the other stage (step k - 1) to its end
    if (k + 1 < steps) issue(k + 1, gemm_lds + (sb ^ kStage));
    const uint8_t *st = gemm_lds + sb;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 x[TI], y[TJ];
#pragma unroll
      for (int i = 0; i < TI; ++i) x[i] = fi.read(st, wi * TI + i, s);
#pragma unroll
      for (int j = 0; j < TJ; ++j) y[j] = fj.read(st, wj * TJ + j, s);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = Elt<TY>::mma(x[i], y[j], acc[i][j]);
    }
    sb ^= kStage;
  }
  write_tile<TY, MODE, TI, TJ>(a, t, j0, wi * TI * 16, wj * TJ * 16, acc);
}

}  // namespace moeq
