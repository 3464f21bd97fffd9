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
#include <type_traits>
#include "check.hpp"

namespace moeq {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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
  uint32_t kdiv, kmul;       // pair / kdiv = mulhi(pair, kmul) >> kshift for 0 <= pair < 2^31, kdiv > 1
  int32_t kshift;
  int32_t ni, nj, nr;        // extents of i, j (kMats only) and r (not kMats)
  int32_t out_type;          // moeq_dtype
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

// A stage covers 128 bytes of every row along r (64 elements of 16 bits, 128
// of 8), a cache line: 64-byte stages, which would leave room for a deeper
// ring, measured 10% slower on matrices with r contiguous.  An MFMA consumes
// half a stage, 16 bytes per lane.
constexpr int kStageBytes = 128;
constexpr int kStageRows = 64;   // rows of a stage where r is the row index (16-bit elements)

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

// Source row of pair id p; -1 (a row of zeros) when it lies outside [0, T).
// The quotient: with kmul = floor(2^(31+L) / k) + 1 and 2^L >= k, the product
// exceeds p / k by less than 1 / k for p < 2^31.
__device__ __forceinline__ int pair_row(const GemmArgs &a, int p) {
  uint32_t s = (uint32_t)p;
  if (a.kdiv != 1) s = __umulhi(s, a.kmul) >> a.kshift;
  return p >= 0 && s < (uint32_t)a.T ? (int)s : -1;
}
// Source row of sorted row r.
__device__ __forceinline__ int source_row(const GemmArgs &a, int r) {
  if (a.pairs) return pair_row(a, a.pairs[r]);
  return r < a.T ? r : -1;
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
constexpr int kMaxExperts = 256;
template <int BJ>
__device__ __forceinline__ bool find_tile(const GemmArgs &a, int BI, Tile *t) {
  constexpr int NB = kMaxExperts / kWave;     // experts per lane
  const int lane = threadIdx.x & 63;
  const int n_it = (a.ni + BI - 1) / BI;
  int lo[NB], hi[NB], nc[NB], end[NB];        // rows, row tiles, row tiles up to and with the expert
  int total = 0;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b * kWave >= a.E) break;
    lo[b] = hi[b] = 0;
    if (b * kWave + lane < a.E) expert_rows(a, b * kWave + lane, &lo[b], &hi[b]);
    nc[b] = end[b] = (hi[b] - lo[b] + BJ - 1) / BJ;
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b * kWave >= a.E) break;
    const int last = std::min(kWave, a.E - b * kWave);
    for (int o = 1; o < last; o <<= 1) {
      const int v = __shfl_up(end[b], o, kWave);
      if (lane >= o) end[b] += v;
    }
    end[b] += total;
    total = __builtin_amdgcn_readlane(end[b], last - 1);
  }
  const int all = total * n_it, per = (all + 7) >> 3;
  const int idx = (int)blockIdx.x >> 3, L = ((int)blockIdx.x & 7) * per + idx;
  if (idx >= per || L >= all) return false;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b * kWave >= a.E) break;
    const uint64_t hit = __ballot(L >= (end[b] - nc[b]) * n_it && L < end[b] * n_it);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      const int n = __builtin_amdgcn_readlane(nc[b], src), ex = __builtin_amdgcn_readlane(end[b], src) - n;
      const int l = __builtin_amdgcn_readlane(lo[b], src), h = __builtin_amdgcn_readlane(hi[b], src);
      const int local = L - ex * n_it, band = local / (kBand * n_it);
      const int in = local - band * kBand * n_it, width = std::min(kBand, n - band * kBand);
      const int jt = band * kBand + in % width;
      t->e = b * kWave + src;
      t->row = l + jt * BJ;
      t->rows = h - t->row;
      t->i0 = in / width * BI;
      // (offsets that do not ascend can make the counts above overflow: such
      // a tile is none)
      return (uint32_t)jt < (uint32_t)n && (uint32_t)t->i0 < (uint32_t)a.ni;
    }
  }
  return false;
}

// 16 bytes at p of which the first n (elements of ES bytes) exist, the rest
// zero.  p need only be aligned to an element.
template <int ES>
__device__ __forceinline__ u32x4 load_piece(const uint8_t *p, int n) {
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
// 16-byte piece c of row x sits in slot c ^ kmaj_swz(x).  A 16-byte read of a
// wave goes through LDS in four passes of 16 lanes: lanes 0-3, 12-15, 20-27,
// the other 16 of the first 32, and the same of the last 32.  An MFMA
// operand read has row l % 16, piece l / 16 (+ 4 in the second half) in lane
// l: with this swizzle each pass covers all 64 banks once
// (SQ_LDS_BANK_CONFLICT is 0).
//
// Operand stored with r as the row index (16-bit only): 64 rows of r, R
// elements each; 32-byte pieces are permuted within each 256 bytes by
// XOR with rmaj_swz(r), so that the rows of a transposing read (four of
// 32 bytes per 16 lanes) fall into different banks.
__device__ __forceinline__ int kmaj_swz(int x) { return x >> 1 & 7; }
__device__ __forceinline__ int rmaj_swz(int r) { return (r & 3) | ((r >> 1) & 4); }

// Fragment reads.  Lane l of an MFMA operand holds element l % 16 of the
// 16-wide tile and 16 bytes of r (piece l / 16 of the half h of the stage).
template <int R, bool RMAJ>
struct FragReader {
  uint32_t base;
  // f0: first 16-wide tile of the wave
  __device__ __forceinline__ FragReader(uint32_t tile_base, int f0) {
    const int l = threadIdx.x & 63, g = l >> 4, x = l & 15;
    if constexpr (!RMAJ) {
      base = tile_base + (16 * f0 + x) * kStageBytes + 16 * (g ^ kmaj_swz(x));
    } else {
      // lane x of the 16 supplies 8 bytes of row r = 8 g + x / 4 (+ 4 for the
      // second read): columns 4 (x % 4) .. + 3 of the tile
      const int r = 8 * g + (x >> 2);
      base = tile_base + r * (2 * R) + (8 * (x & 3) | 32 * ((f0 & 7) ^ rmaj_swz(r))) + (f0 >> 3) * 256;
    }
  }
  __device__ __forceinline__ u32x4 read(const uint8_t *lds, int f, int h) const {
    if constexpr (!RMAJ) {
      return *reinterpret_cast<const u32x4 *>(lds + (base ^ (uint32_t)(64 * h)) + f * 16 * kStageBytes);
    } else {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      const uint32_t o = (base ^ (uint32_t)((f & 7) * 32)) + (f >> 3) * 256 + h * (kStageRows / 2) * (2 * R);
      const auto p = (__attribute__((address_space(3))) s16x4 *)(lds + o);
      const auto q = (__attribute__((address_space(3))) s16x4 *)(lds + o + 4 * (2 * R));
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(q));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  }
};

__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p) {   // into scalar registers
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (const uint8_t *)(((uint64_t)hi << 32) | lo);
}

// Buffer -> LDS transfer of SIZE (4 or 16) bytes per lane, as lds_dma_buf but
// unknown to the compiler (rs: the four words of the buffer resource): it
// puts a wait for all transfers before every transposing LDS read
// otherwise.  The kernel waits by count before the step that reads the
// data; the instruction has no register output.  m0 holds the LDS address;
// it is the compiler's to write, as an input of the asm, which changes no
// register (saving m0 and giving it back within the asm cost 1%).
// (s_nop 4: five wait states between a VALU write of a scalar register, as
// v_readfirstlane makes for rs, and a memory instruction that reads it; one
// after a write of m0; the compiler does not look into the asm for either.)
template <int SIZE>
__device__ __forceinline__ void lds_dma_raw(i32x4 rs, uint32_t voff, uint32_t soff, const uint8_t *lds) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)lds;
  if constexpr (SIZE == 16)
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" :: "v"(voff), "s"(rs), "s"(soff), "{m0}"(at) : "memory");
  else
    asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, %2 offen lds" :: "v"(voff), "s"(rs), "s"(soff), "{m0}"(at) : "memory");
}
__device__ __forceinline__ i32x4 raw_rsrc(const uint8_t *base, uint32_t bytes) {   // both uniform
  const uint64_t v = (uint64_t)uniform(base);
  return i32x4{(int)(uint32_t)v, (int)((uint32_t)(v >> 32) & 0xffffu), __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// ---- Movement of an operand's stages into LDS.  A wave moves NB blocks of 1
// KiB of every stage.
//
// DMA: buffer loads with an LDS destination; the data never occupies
// registers.  Bases and rows must be 16-byte aligned; what lies behind the
// buffer resource's range reads zero, which gives the zeros behind the last
// row and the last r.
// Otherwise through registers: any element alignment and row stride, 64-bit
// addresses; a stage is loaded one stage before it is stored.
constexpr uint32_t kNowhere = 0x80000000u;   // an offset behind every range used here

// Offsets of the 16 bytes `piece` of stage t of a row `width` bytes long whose
// lane offset is `row` (piece included): the lane's and the uniform one.  The
// range check takes the uniform offset from the range, so that it must not
// pass the range: a stage behind the row's end has none.
struct StageOffsets {
  uint32_t voff, soff;
};
__host__ __device__ constexpr StageOffsets stage_offsets(int t, int piece, int width, uint32_t row) {
  const int at = t * kStageBytes;
  return {piece < width - at ? row : kNowhere, at < width ? (uint32_t)at : 0u};
}

template <int ES, int R, int NW, bool RMAJ, bool DMA>
struct Operand {
  static constexpr int NB = R * kStageBytes / (1024 * NW);
  static_assert(R * kStageBytes % (1024 * NW) == 0, "blocks per wave");
  static_assert(!RMAJ || (R % 128 == 0 && ES == 2), "256-byte swizzle groups of 16-bit elements");
  i32x4 rs;
  uint32_t voff[NB];       // DMA: lane's offset from the resource's base (kNowhere: no such row)
  const uint8_t *p[NB];    // registers, r contiguous: the row's first byte (null: no such row)
  const uint8_t *base;     // r as row index: the matrix (row 0 of the run) at the tile's first column
  int64_t ld;              // bytes between rows
  int nr, width;           // extent of r; bytes of a row: valid ones (r contiguous), or from the tile's first column
  u32x4 v[NB];             // registers: the stage on its way

  int first;               // the wave's first block

  __device__ __forceinline__ explicit Operand(int wave) : first(wave * NB) {}
  __device__ __forceinline__ int block(int i) const { return first + i; }
  // r contiguous: tile row and byte in the stage that the lane moves in block i
  __device__ __forceinline__ int row_of(int i) const { return block(i) * 8 + (int)((threadIdx.x & 63) >> 3); }
  __device__ __forceinline__ int piece_of(int i) const { return 16 * ((int)(threadIdx.x & 7) ^ kmaj_swz(row_of(i))); }
  // r as row index: row in the stage and byte column
  __device__ __forceinline__ int r_of(int i) const { return (block(i) * 1024 + (int)(threadIdx.x & 63) * 16) / (2 * R); }
  __device__ __forceinline__ int col_of(int i) const {
    const int o = block(i) * 1024 + (int)(threadIdx.x & 63) * 16;
    return 16 * ((o % (2 * R)) / 16 ^ (2 * rmaj_swz(o / (2 * R))));
  }

  // The range check is by dword and wants a dword whole: the one that holds
  // the last element of an odd row counts in full.
  __device__ __forceinline__ uint32_t range_width() const { return ((uint32_t)width + 3u) & ~3u; }

  // r contiguous: row x of the tile starts `stride` bytes times index(x)
  // (negative: a row of zeros) behind `from`; `last` the largest index
  template <class Index>
  __device__ __forceinline__ void rows(const uint8_t *from, int64_t stride, int64_t last, int n_r, Index index) {
    nr = n_r;
    width = n_r * ES;
    if constexpr (DMA) rs = raw_rsrc(from, (uint32_t)(last * stride + width));
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int x = index(row_of(i));
      if constexpr (DMA) voff[i] = x < 0 ? kNowhere : (uint32_t)x * (uint32_t)stride + (uint32_t)piece_of(i);
      else p[i] = x < 0 ? nullptr : from + x * stride;
    }
  }
  // r as row index: consecutive rows from `from` (at the tile's first column)
  __device__ __forceinline__ void cols(const uint8_t *from, int64_t stride, int n_r, int row_bytes) {
    base = uniform(from);
    ld = stride;
    nr = n_r;
    width = row_bytes;
    if constexpr (DMA) {
#pragma unroll
      for (int i = 0; i < NB; ++i) voff[i] = (uint32_t)r_of(i) * (uint32_t)ld + (uint32_t)col_of(i);
    }
  }
  // r as row index: rows given stage by stage
  __device__ __forceinline__ void gather(const uint8_t *from, int64_t stride, int64_t last, int n_r, int row_bytes) {
    cols(from, stride, n_r, row_bytes);
    if constexpr (DMA) rs = raw_rsrc(base, (uint32_t)(last * stride + range_width()));
  }

  // DMA: block i of stage t into the tile at `dst` (stages behind the last:
  // zeros)
  __device__ __forceinline__ void dma_rows(int i, int t, uint8_t *dst) const {
    const StageOffsets o = stage_offsets(t, piece_of(i), width, voff[i]);
    lds_dma_raw<16>(rs, o.voff, o.soff, dst + block(i) * 1024);
  }
  __device__ __forceinline__ void dma_cols(int i, int t, uint8_t *dst) const {
    const int left = std::min(kStageRows, nr - t * kStageRows);
    const i32x4 r = raw_rsrc(base + (int64_t)t * kStageRows * ld, left > 0 ? (uint32_t)(left - 1) * (uint32_t)ld + range_width() : 0u);
    lds_dma_raw<16>(r, voff[i], 0, dst + block(i) * 1024);
  }
  __device__ __forceinline__ void dma_gather(int i, int src, uint8_t *dst) const {
    lds_dma_raw<16>(rs, src < 0 ? kNowhere : (uint32_t)src * (uint32_t)ld + (uint32_t)col_of(i), 0, dst + block(i) * 1024);
  }
  // registers: load stage t, store what is loaded
  __device__ __forceinline__ void load_rows(int t) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int o = t * kStageBytes + piece_of(i);
      v[i] = load_piece<ES>(p[i] + o, p[i] ? width - o : 0);
    }
  }
  __device__ __forceinline__ void load_cols(int t) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int r = t * kStageRows + r_of(i);
      v[i] = load_piece<ES>(base + r * ld + col_of(i), r < nr ? width - col_of(i) : 0);
    }
  }
  __device__ __forceinline__ void load_gather(const int *src) {
#pragma unroll
    for (int i = 0; i < NB; ++i) v[i] = load_piece<ES>(base + src[i] * ld + col_of(i), src[i] >= 0 ? width - col_of(i) : 0);
  }
  __device__ __forceinline__ void store(uint8_t *dst) const {
#pragma unroll
    for (int i = 0; i < NB; ++i) *reinterpret_cast<u32x4 *>(dst + block(i) * 1024 + (threadIdx.x & 63) * 16) = v[i];
  }
};

// ---- output
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint16_t f16_bits(float v) { return __builtin_bit_cast(uint16_t, (f16)v); }

typedef f32x4 f32x4_a4 __attribute__((aligned(4)));   // at the alignment of an element
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

// Four consecutive elements at index o of which n exist, each rounded once.
__device__ __forceinline__ void store4(const GemmArgs &a, int64_t o, f32x4 v, int n) {
  if (a.out_type == MOEQ_F32) {
    float *p = (float *)a.out + o;
    if (n >= 4) *(__attribute__((address_space(1))) f32x4_a4 *)p = v;
    else {
#pragma unroll
      for (int i = 0; i < 3; ++i) if (i < n) p[i] = v[i];
    }
    return;
  }
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = a.out_type == MOEQ_BF16 ? bf16_bits(v[i]) : f16_bits(v[i]);
  uint16_t *p = (uint16_t *)a.out + o;
  if (n >= 4) {
    *(__attribute__((address_space(1))) u32x2_a2 *)p =
        u32x2{(uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16)};
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) if (i < n) p[i] = h[i];
  }
}

// Tiles of the matrices' gradient take a time that depends on the expert's
// rows.  Each XCD gets short runs of tiles (in bands of kBand i tiles) of all
// the experts in turn, not one run of whole experts, and the experts with the
// most rows come first, so that no long tile starts last.  A run has up to 8
// tiles of 256 x 256, as many outputs of smaller ones, and as few as leave
// every XCD the same number of runs.  (64 experts of 1408 x 2048, 24576 rows,
// bf16, fp32 out: equal rows 309 us, runs of whole experts 298; shares falling
// with the root of the rank 336, whole experts 392, runs of 32 tiles 354;
// falling with the power 1.1 352, 605 and 462.)
__host__ __device__ constexpr int mats_run(int all, int BI, int BJ) {
  const int most = 8 * (256 * 256 / (BI * BJ));
  const int rounds = (all + 8 * most - 1) / (8 * most);
  return (all + 8 * rounds - 1) / (8 * rounds);
}

// The expert at place n of the order by rows, to a power of two times the
// mean (more exactly, E compares per lane would take longer than they save);
// its first row and its rows.
__device__ __forceinline__ int nth_expert(const GemmArgs &a, int n, int *row, int *rows) {
  constexpr int NB = kMaxExperts / kWave;     // experts per lane
  const int lane = threadIdx.x & 63, mean = a.P / a.E + 1;
  int lo[NB], len[NB], cls[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    lo[b] = len[b] = 0;
    cls[b] = -1;
    const int e = b * kWave + lane;
    if (e >= a.E) continue;
    int hi;
    expert_rows(a, e, &lo[b], &hi);
    len[b] = hi - lo[b];
    cls[b] = (len[b] >= mean / 2) + (len[b] >= mean) + (len[b] >= 2ll * mean) + (len[b] >= 4ll * mean);
  }
  for (int c = 4; c >= 0; --c) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b * kWave >= a.E) break;
      const uint64_t in = __ballot(cls[b] == c);
      const int count = __builtin_popcountll(in);
      if (n < count) {
        const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0));
        const int src = __builtin_ctzll(__ballot(cls[b] == c && before == n));
        *row = __builtin_amdgcn_readlane(lo[b], src);
        *rows = __builtin_amdgcn_readlane(len[b], src);
        return b * kWave + src;
      }
      n -= count;
    }
  }
  *row = *rows = 0;                            // (not reached: every expert is in a class)
  return 0;
}

// Output tile of a workgroup, the extent of r and, for the matrices'
// gradient, the first j; all in scalar registers.
template <int MODE, int BI, int BJ>
__device__ __forceinline__ bool pick_tile(const GemmArgs &a, Tile *t, int *nr, int *j0) {
  Tile v{};
  int r = a.nr, j = 0;
  if constexpr (MODE == kMats) {
    const int n_it = (a.ni + BI - 1) / BI, n_jt = (a.nj + BJ - 1) / BJ, all = a.E * n_it * n_jt;
    const int per = mats_run(all, BI, BJ), xcd = (int)blockIdx.x & 7, idx = (int)blockIdx.x >> 3;
    const int L = (idx / per * 8 + xcd) * per + idx % per;
    if (L >= all) return false;
    const int nth = L / (n_it * n_jt), local = L - nth * n_it * n_jt, band = local / (kBand * n_jt);
    const int in = local - band * kBand * n_jt, width = std::min(kBand, n_it - band * kBand);
    j = in / width * BJ;
    v.i0 = (band * kBand + in % width) * BI;
    v.e = nth_expert(a, nth, &v.row, &r);
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
    float sc = 1.f, up = 1.f;
    if constexpr (TY == kI8) {
      const int s = source_row(a, t.row + x);
      sc = s >= 0 ? a.sj[s] : 0.f;
      // (a sum of up to 2^31 times a scale of 2^96 and more could leave fp32
      // where the product with the channel's scale does not)
      if (__builtin_fabsf(sc) >= 0x1p96f) {
        sc *= 0x1p-40f;
        up = 0x1p40f;
      }
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
        if constexpr (TY == kI8) v[q] = v[q] * sc * (c + q < a.ni ? a.si[(int64_t)t.e * a.ni + c + q] : 0.f) * up;
      }
      store4(a, ob + c, v, a.ni - c);
    }
  }
}

// ---- tiled kernel: a workgroup of WI x WJ waves computes BI x BJ outputs,
// walking r through LDS rings of RI stages of I and RJ (RI or one less) of J.
//
// A wave multiplies half a stage out of registers while it reads the
// fragments of the next half into a second set, so that the matrix pipe does
// not wait for LDS.  Before the second half of stage k every wave has taken
// it into registers, which frees its places for stage k + RI of I and k + RJ
// of J; stage k + 1 has to be there by then, for its first fragments: one
// wait and one barrier per stage.
//
// With tiles of 256 x 256 the rings are the kernel's bound: without the DMA
// operations 1024 tiles of r 5632 take 541 us, without the MFMAs 640 (417
// when all of them hit the L2), with both 777 at two stages each.  The third
// stage of I, which is the matrices and comes from HBM, fills the LDS.
//
// LDS of a workgroup: the rings, and the pair ids of kMats.
template <int MODE, int BI, int BJ, int RI, int RJ, bool DMA>
constexpr size_t tile_lds() {
  return (RI * BI + RJ * BJ) * kStageBytes + (MODE == kMats && DMA ? 2 * (BI * kStageBytes / 1024) * 256 : 0);
}

template <int TY, int MODE, int BI, int BJ, int WI, int WJ, int RI, int RJ, bool DMA>
__global__ void __launch_bounds__(64 * WI * WJ, 1) gemm_tile_kernel(GemmArgs a) {
  constexpr int ES = Elt<TY>::size, NW = WI * WJ, TI = BI / WI / 16, TJ = BJ / WJ / 16;
  constexpr bool XI = MODE != kFwd, XJ = MODE == kMats;      // r is the row index of the operand
  constexpr uint32_t kTileI = BI * kStageBytes, kTileJ = BJ * kStageBytes, kJ = RI * kTileI;   // J's ring
  static_assert(RI == RJ || RI == RJ + 1, "see the wait counts");
  using Acc = typename Elt<TY>::acc;
  extern __shared__ __attribute__((aligned(1024))) uint8_t gemm_lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave % WI, wj = wave / WI;
  Tile t;
  int nr, j0;
  if (!pick_tile<MODE, BI, BJ>(a, &t, &nr, &j0)) return;

  using OpI = Operand<ES, BI, NW, XI, DMA>;
  using OpJ = Operand<ES, BJ, NW, XJ, DMA>;
  OpI di(wave);
  OpJ dj(wave);
  // kMats with pairs: the pair ids of the rows that this wave moves come by
  // DMA too, one stage before they are needed (a load into registers would
  // make the wave wait for every transfer before it).  Stage k's are in slot
  // k % 2, one dword per lane and block.
  constexpr bool kIdx = MODE == kMats && DMA;
  i32x4 prs{};
  auto idx_at = [&](int q, int k) { return gemm_lds + kJ + RJ * kTileJ + (((k & 1) * NW + wave) * OpI::NB + q) * 256; };
  auto fetch_idx = [&](int q, int k) {
    const int r = k * kStageRows + di.r_of(q);
    lds_dma_raw<4>(prs, r < nr ? (uint32_t)r * 4u : kNowhere, 0, idx_at(q, k));
  };
  auto source = [&](int q, int k) {      // source row of the lane's row in block q of stage k
    const int r = k * kStageRows + di.r_of(q);
    if (r >= nr) return -1;
    if constexpr (kIdx) {
      if (a.pairs) return pair_row(a, *reinterpret_cast<const int *>(idx_at(q, k) + (threadIdx.x & 63) * 4));
    }
    return source_row(a, t.row + r);
  };
  const int64_t si = a.ldi * ES, sj = a.ldj * ES;
  if constexpr (MODE == kMats) {
    di.gather(a.I + (int64_t)t.i0 * ES, si, a.T - 1, nr, (a.ni - t.i0) * ES);
    dj.cols(a.J + (int64_t)t.row * sj + (int64_t)j0 * ES, sj, nr, (a.nj - j0) * ES);
    if constexpr (kIdx) {
      if (a.pairs) {
        prs = raw_rsrc((const uint8_t *)(a.pairs + t.row), (uint32_t)nr * 4u);
#pragma unroll
        for (int q = 0; q < OpI::NB; ++q) fetch_idx(q, 0), fetch_idx(q, 1);
        vm_wait<0>();
      }
    }
  } else {
    const uint8_t *wmat = a.I + (int64_t)t.e * a.e_i * ES;   // the expert's matrix
    if constexpr (MODE == kRows) {
      di.cols(wmat + (int64_t)t.i0 * ES, si, nr, (a.ni - t.i0) * ES);
    } else {
      const int n = std::min(BI, a.ni - t.i0);
      di.rows(wmat + t.i0 * si, si, n - 1, nr, [&](int x) { return x < n ? x : -1; });
    }
    if (a.pairs) {
      dj.rows(a.J, sj, a.T - 1, nr, [&](int x) { return x < t.rows ? source_row(a, t.row + x) : -1; });
    } else {
      const int n = std::min(BJ, t.rows);
      dj.rows(a.J + t.row * sj, sj, n - 1, nr, [&](int x) { return x < n ? x : -1; });
    }
  }
  constexpr int kOps = DMA ? OpI::NB + OpJ::NB : 0;
  // DMA operations of a stage, J's first: q-th of stage kj of J to toj, or of
  // stage ki of I to toi
  auto move = [&](int q, int kj, uint8_t *toj, int ki, uint8_t *toi) {
    if constexpr (DMA) {
      if (q < OpJ::NB) {
        if constexpr (XJ) dj.dma_cols(q, kj, toj);
        else dj.dma_rows(q, kj, toj);
      } else {
        const int i = q - OpJ::NB;
        if constexpr (MODE == kMats) di.dma_gather(i, source(i, ki), toi);
        else if constexpr (MODE == kRows) di.dma_cols(i, ki, toi);
        else di.dma_rows(i, ki, toi);
      }
    }
  };
  auto load = [&](int k) {                       // stage k into registers
    if constexpr (!DMA) {
      if constexpr (MODE == kMats) {
        int src[OpI::NB];
#pragma unroll
        for (int q = 0; q < OpI::NB; ++q) src[q] = source(q, k);
        di.load_gather(src);
      } else if constexpr (MODE == kRows) {
        di.load_cols(k);
      } else {
        di.load_rows(k);
      }
      if constexpr (XJ) dj.load_cols(k);
      else dj.load_rows(k);
    }
  };
  auto store = [&](uint8_t *toj, uint8_t *toi) {   // and from there into its place
    if constexpr (!DMA) {
      di.store(toi);
      dj.store(toj);
    }
  };
  static_assert(RI == 2 || (DMA && MODE != kMats), "longer rings count DMA operations only");

  Acc acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = Acc{0, 0, 0, 0};
  const FragReader<BI, XI> fi(0, wi * TI);
  const FragReader<BJ, XJ> fj(kJ, wj * TJ);
  const int stages = (int)(((int64_t)nr * ES + kStageBytes - 1) / kStageBytes);
  if (stages > 0) {
#pragma unroll
    for (int k = 0; k < RI; ++k) {
      uint8_t *toj = gemm_lds + kJ + k * kTileJ, *toi = gemm_lds + k * kTileI;
      if (!DMA) {
        load(k);
        store(toj, toi);
      }
#pragma unroll
      for (int q = 0; q < kOps; ++q)
        if (k < RJ || q >= OpJ::NB) move(q, k, toj, k, toi);
    }
    if (!DMA) load(2);
    lgkm_vm_wait<DMA ? (RJ - 1) * OpJ::NB + (RI - 1) * OpI::NB : 0>();
    if constexpr (kIdx) {    // (both stages' ids have been read)
      if (a.pairs) {
#pragma unroll
        for (int q = 0; q < OpI::NB; ++q) fetch_idx(q, 2);
      }
    }
    __builtin_amdgcn_s_barrier();
    u32x4 x[2][TI], y[2][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i) x[0][i] = fi.read(gemm_lds, i, 0);
#pragma unroll
    for (int j = 0; j < TJ; ++j) y[0][j] = fj.read(gemm_lds, j, 0);
    // The MFMAs of a half stage (set C), with the reads of the next one
    // (half 1 - C of the stage at sti, stj) between them, in kSeg parts.  In the
    // second half a part starts with its share of the DMA operations (all at
    // once after the barrier they hold the waves up: a CU takes one in about
    // 16 cycles).  The last part has no reads, so that its MFMAs cover their
    // latency.
    auto half = [&](auto c, const uint8_t *sti, const uint8_t *stj, int k, uint8_t *toi, uint8_t *toj) {
      constexpr int C = decltype(c)::value, N = 1 - C;
      constexpr int kSeg = TI < 4 ? TI : 4, kRd = kSeg > 1 ? kSeg - 1 : 1, IS = TI / kSeg;
      constexpr int kReads = TI + TJ, kInsI = XI ? 2 : 1, kInsJ = XJ ? 2 : 1;
#pragma unroll
      for (int g = 0; g < kSeg; ++g) {
        if constexpr (C == 1) {
#pragma unroll
          for (int q = 0; q < kOps; ++q)
            if (q * kSeg / std::max(kOps, 1) == g) move(q, k + RJ, toj, k + RI, toi);
        }
        int ins = 0;
#pragma unroll
        for (int f = 0; f < kReads; ++f)
          if (f * kRd / kReads == g) {
            if (f < TJ) y[N][f] = fj.read(stj, f, N), ins += kInsJ;
            else x[N][f - TJ] = fi.read(sti, f - TJ, N), ins += kInsI;
          }
#pragma unroll
        for (int i = g * IS; i < (g + 1) * IS; ++i)
#pragma unroll
          for (int j = 0; j < TJ; ++j) acc[i][j] = Elt<TY>::mma(x[C][i], y[C][j], acc[i][j]);
#pragma unroll
        for (int f = 0; f < kReads * 2; ++f) {
          if (f < ins) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
          }
        }
        __builtin_amdgcn_sched_group_barrier(0x008, TI * TJ, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    uint32_t ai = 0, aj = 0; // where stage k is in the rings
    // the wait and the barrier before the second half of stage k
    auto turn = [&](int k) {
      lgkm_vm_wait<DMA ? (RJ - 2) * kOps + (RI - RJ) * OpI::NB : 0>();
      __builtin_amdgcn_s_barrier();
      if constexpr (!DMA) {
        store(gemm_lds + kJ + aj, gemm_lds + ai);
        load(k + 3);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto ids = [&](int k) {
      if constexpr (kIdx) {
        if (a.pairs) {
#pragma unroll
          for (int q = 0; q < OpI::NB; ++q) fetch_idx(q, k);
        }
      }
    };
    auto next = [&](uint32_t *n, uint32_t v, uint32_t tile, int ring) { *n = v == (ring - 1) * tile ? 0u : v + tile; };
    // a wave whose outputs do not exist (behind the expert's last row, or the
    // last i) only moves operands
    if (wj * TJ * 16 < t.rows && t.i0 + wi * TI * 16 < a.ni) {
#pragma unroll 1
      for (int k = 0; k < stages; ++k) {
        half(std::integral_constant<int, 0>{}, gemm_lds + ai, gemm_lds + aj, 0, nullptr, nullptr);
        turn(k);
        uint32_t ni, nj;
        next(&ni, ai, kTileI, RI);
        next(&nj, aj, kTileJ, RJ);
        half(std::integral_constant<int, 1>{}, gemm_lds + ni, gemm_lds + nj, k, gemm_lds + ai, gemm_lds + kJ + aj);
        ids(k + 3);
        ai = ni;
        aj = nj;
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < stages; ++k) {
        turn(k);
#pragma unroll
        for (int q = 0; q < kOps; ++q) move(q, k + RJ, gemm_lds + kJ + aj, k + RI, gemm_lds + ai);
        ids(k + 3);
        next(&ai, ai, kTileI, RI);
        next(&aj, aj, kTileJ, RJ);
      }
    }
    vm_wait<0>();            // (the zeros of stages behind the last are still on their way)
  }
  write_tile<TY, MODE, TI, TJ>(a, t, j0, wi * TI * 16, wj * TJ * 16, acc);
}

}  // namespace moeq
