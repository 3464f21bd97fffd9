// Low-rank adapters of many requests beside a shared projection:
// out[r] = y[r] + scale_i B_i (A_i x[r]), i = ids[r].
//
// Two kernels, z = A_i x with K in parts and out = y + scale_i B_i z, both by
// MFMA over tiles of 16 rows: the operations are few (4096 rows of 4096, rank
// 64: 4.3 GFLOP), the bytes of x, y and out bound long batches, latency short
// ones.  Measured by replays of a captured call: 4096 rows of 4096 in bf16 in
// runs of eight adapters 25.8 us for rank 16 and 37.9 us for rank 64 (101 and 109
// MB: 20 and 21 us at the rate of a large copy), one row of 4096 -> 14336 with
// rank 32 7.5 us, 64 rows of 32 adapters of rank 16 13.1 us (a kernel trace, which
// keeps the two launches apart, has 39.0, 9.1 and 16.0 us for the last three).
// What is left in long batches is A_i and B_i from L2 through LDS for every 16
// (32) rows; in the last, waves that have one chunk of K each and sixteen parts
// of z that every workgroup sums.
#include "check.hpp"
#include "vec8.hpp"
#include "wave.hpp"

namespace moeq {

constexpr int kAdaptersMaxR = 256;
constexpr int kAdaptersMaxN = 1 << 20;

constexpr int kRows = 16;        // rows (tokens) of an MFMA tile
constexpr int kChunk = 64;       // columns of x and A that a wave takes at a time: 128 bytes of a row

struct AdapterArgs {
  const void *x, *a, *b, *y;
  void *out;
  const int32_t *ids, *ranks;
  const float *scale;
  float *z;              // [splits, T, R]
  int64_t ldx, lda, stride_a, ldb, stride_b, ldy, ldo;
  int T, n, R, N, K;
  int splits, per;       // parts of K, chunks of each
  int width;             // outputs of a workgroup of the second kernel
  int tiles, parts, slots;   // the grid: tiles of rows, parts of K or N, workgroups that share the adapters of a tile
};

template <int TY> struct Frag;
template <> struct Frag<MOEQ_F16> {
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <> struct Frag<MOEQ_BF16> {
  typedef __bf16 vec __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(vec, a), __builtin_bit_cast(vec, b), c, 0, 0, 0);
  }
};

// Eight 16-bit values at p.
__device__ __forceinline__ u32x4 load8(const uint8_t *p) { return *(const __attribute__((address_space(1))) u32x4_a2 *)p; }

// Values col .. col + 7 of a row of `len` that begins at p, zeros from `valid`
// (<= len) on.  Near the end of the row the last eight of it are loaded and
// moved down, so that nothing behind it is touched.
__device__ __forceinline__ u32x4 load8(const uint8_t *p, int col, int len, int valid) {
  u32x4 v = {0, 0, 0, 0};
  if (len < 8) {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (col + j < valid) v[j / 2] |= (uint32_t)gld<uint16_t>(p + (col + j) * 2) << (16 * (j & 1));
    return v;
  }
  if (col >= valid) return v;
  const int at = std::min(col, len - 8), down = col - at, n = valid - col;
  v = load8(p + at * 2);
  if (down & 4) v = u32x4{v[2], v[3], 0, 0};
  if (down & 2) v = u32x4{v[1], v[2], v[3], 0};
  if (down & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = n >= 2 * i + 2 ? v[i] : n == 2 * i + 1 ? v[i] & 0xffffu : 0;
  return v;
}

__device__ __forceinline__ int rank_of(const AdapterArgs &a, int id) {
  const int r = a.ranks ? a.ranks[id] : a.R;
  return r < 0 ? 0 : r > a.R ? a.R : r;
}

// The rows of a tile of 16 TM and the adapters they use.  Every lane holds
// the adapters of rows lane % 16 + 16 tm (-1: none); next() names the tile's
// distinct adapters one after the other, in the order of their first rows.
template <int TM>
struct Tile {
  int id[TM];
  uint32_t left[TM];   // rows (bits) whose adapter has not been named

  __device__ __forceinline__ void load(const AdapterArgs &a, int r0) {
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const int r = r0 + m * kRows + (threadIdx.x & 15);
      id[m] = r < a.T ? a.ids[r] : -1;
      if ((uint32_t)id[m] >= (uint32_t)a.n) id[m] = -1;
    }
    restart();
  }
  __device__ __forceinline__ void restart() {
#pragma unroll
    for (int m = 0; m < TM; ++m) left[m] = (uint32_t)__ballot(id[m] >= 0) & 0xffffu;
  }
  // The next adapter and (row) the first row that uses it, or -1.
  __device__ __forceinline__ int next(int &row) {
    int cur = -1;
#pragma unroll
    for (int m = 0; m < TM; ++m)
      if (cur < 0 && left[m]) {
        const int at = __builtin_ctz(left[m]);
        row = m * kRows + at;
        cur = __builtin_amdgcn_readlane(id[m], at);
      }
#pragma unroll
    for (int m = 0; m < TM; ++m) left[m] &= ~(uint32_t)__ballot(id[m] == cur);
    return cur;
  }
};

// A workgroup's place.  Workgroups are dealt to the eight XCDs in turn; each
// XCD gets consecutive tiles, which mostly use the same few adapters, so that
// these stay in its L2.
struct Place {
  int tile, part, slot;
  __device__ __forceinline__ Place(const AdapterArgs &a) {
    const int each = gridDim.x / 8, at = (blockIdx.x % 8) * each + blockIdx.x / 8;
    const int per = a.parts * a.slots;
    tile = at / per;          // (beyond the last: no work)
    part = at % per / a.slots;
    slot = at % a.slots;
  }
};
static dim3 place_grid(const AdapterArgs &a) { return dim3((a.tiles * a.parts * a.slots + 7) / 8 * 8); }

// What a workgroup takes of the adapters of its tile: every slots-th of them.
struct Turn {
  int left;
  __device__ __forceinline__ Turn(const Place &p) : left(p.slot) {}
  __device__ __forceinline__ bool mine(const AdapterArgs &a) {
    const bool m = left == 0;
    left = m ? a.slots - 1 : left - 1;
    return m;
  }
};

// The terms of z and each row's power of two.
template <int TM, int NT, int TERMS>
struct ZTerms {
  static constexpr int RP = (NT + 1) / 2 * 32;   // ranks, whole MFMA steps
  __attribute__((aligned(16))) uint16_t z[TERMS][TM * kRows][RP + 8];
  float up[TM * kRows];
};

// Row r = tid / 16, ranks 16 q + tid % 16 (v[q]; 0 from the rank on): brought
// to a power of two near 1 per row and split into TERMS 16-bit numbers, whose
// products with B_i are exact in the MFMA.  Two terms keep 22 bits of z's
// largest in fp16 and 16 in bf16, more than a 16-bit output shows; an fp32
// output takes three.
template <int TY, int TM, int NT, int TERMS>
__device__ __forceinline__ void put_terms(ZTerms<TM, NT, TERMS> &s, int r, const float (&v)[NT], int rank) {
  const int j = threadIdx.x & 15;
  float top = 0.f;
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const float f = q * kRows + j < rank ? __builtin_fabsf(v[q]) : 0.f;
    if (f < __builtin_inff()) top = __builtin_fmaxf(top, f);
  }
  top = dpp_row_max(top);
  const int e = top > 0.f ? std::max(ilogb_f32(top), -120) : 0;   // (2^e and 2^-e are normal numbers)
  if (j == 0) s.up[r] = __builtin_ldexpf(1.f, e);
#pragma unroll
  for (int q = 0; q < ZTerms<TM, NT, TERMS>::RP / kRows; ++q) {
    float rest = 0.f;
    if (q < NT && q * kRows + j < rank) rest = __builtin_ldexpf(v[q < NT ? q : 0], -e);
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      const uint32_t bits = Val<TY>::put(rest);
      s.z[t][r][q * kRows + j] = (uint16_t)bits;
      // (an infinity or NaN is in the first term whole)
      rest = __builtin_fabsf(rest) < __builtin_inff() ? rest - Val<TY>::get(bits) : 0.f;
    }
  }
}

// Both kernels: an MFMA operand's lanes lie in 16 different rows, and such a
// load keeps the address path busy 2.6 times as long as one along the rows (1 KB
// from the caches: 77 clocks of 2.4 GHz against 29), which bounds a stream of
// them.  So every operand comes along its rows, eight lanes to 128 bytes, and changes places in
// a part of LDS that belongs to its wave alone: no barriers, since the LDS
// operations of a wave stay in order.
constexpr int kAdapterWaves = 4, kAdapterThreads = kAdapterWaves * kWave;

// [rows][64] 16-bit values, 128 bytes a row, in pieces of 16 bytes: piece p of
// row r stands at p ^ (r % 8), so that neither side has bank conflicts.
template <int ROWS>
struct Stage {
  __attribute__((aligned(16))) uint8_t b[ROWS * 128];
  __device__ __forceinline__ void put(int r, int p, u32x4 v) { *(u32x4 *)(b + r * 128 + (p ^ (r & 7)) * 16) = v; }
  // MFMA operand: row 16 t + lane % 16, columns 32 h + 8 (lane / 16) ..
  __device__ __forceinline__ u32x4 get(int t, int h) const {
    const int lane = threadIdx.x & 63, r = lane & 15;
    return *(const u32x4 *)(b + (t * kRows + r) * 128 + ((h * 4 + (lane >> 4)) ^ (r & 7)) * 16);
  }
};

// Sixty-four outputs of 16 rows in fp32.
struct OutTile {
  float v[kRows][64 + 4];
};

// Sums of a tile's z over the waves: 16 NT ranks.
template <int TM, int NT>
using Red = float[kAdapterWaves][TM * kRows][NT * kRows + 4];

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Partial sums of z = A_i x over one part of K, 16 NT ranks from j0: one
// workgroup per tile of 16 TM rows, part, group of ranks and slot.  The waves
// take chunks of 64 columns in turn, each the products of 16 TM rows with
// 16 NT rows of A_i, with D - 1 chunks under way while one is multiplied (as
// many as leave room for four workgroups on a CU).  Rows of the tile with
// another adapter (or none), and rows of A_i beyond R, read a valid row
// instead: they only reach sums that are not stored.
template <int TY, int TM, int NT, int D>
__global__ void __launch_bounds__(kAdapterThreads, TM + NT < 3 ? 4 : NT < 4 ? 3 : 2)
adapters_down_kernel(AdapterArgs a) {
  constexpr int NW = kAdapterWaves, GR = NT * kRows;
  constexpr int XI = TM * 2, AI = NT * 2;       // loads of 1 KB: a chunk of x and of A
  union Part {
    Stage<kRows *(TM + NT)> in[NW];
    Red<TM, NT> red;
  };
  __shared__ Part part;
  const Place place(a);
  const int r0 = place.tile * (TM * kRows), tid = threadIdx.x, lane = tid & 63, wave = wave_id(), l16 = lane & 15, g = lane >> 4;
  if (place.tile >= a.tiles) return;
  const int j0 = place.part / a.splits * GR, split = place.part % a.splits;
  const int c0 = split * a.per, chunks = std::min(c0 + a.per, (a.K + kChunk - 1) / kChunk) - c0;
  Tile<TM> tile;
  tile.load(a, r0);
  auto &st = part.in[wave];
  const int pr = lane >> 3, pc = lane & 7;   // row and piece of a load along the rows
  int row = 0;
  Turn turn(place);
  Tile<TM> left = tile;
  const int whole = std::min(c0 + chunks, a.K / kChunk) - c0;
  for (int cur = left.next(row); cur >= 0; cur = left.next(row)) {
    if (!turn.mine(a)) continue;
    const uint8_t *xp[XI], *ap[AI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int r = i * 8 + pr;
      const bool mine = __shfl(tile.id[i / 2], r & 15, kWave) == cur;
      xp[i] = (const uint8_t *)a.x + ((r0 + (mine ? r : row)) * a.ldx + pc * 8) * 2;
    }
#pragma unroll
    for (int i = 0; i < AI; ++i) {
      const int j = j0 + i * 8 + pr;
      ap[i] = (const uint8_t *)a.a + (cur * a.stride_a + (j < a.R ? j : 0) * a.lda + pc * 8) * 2;
    }
    f32x4 acc[TM][NT];
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const auto fetch = [&](int i, u32x4 (&x)[XI], u32x4 (&w)[AI]) {   // the i-th whole chunk
      const int c = c0 + i;
#pragma unroll
      for (int q = 0; q < XI; ++q) x[q] = load8(xp[q] + c * (kChunk * 2));
#pragma unroll
      for (int q = 0; q < AI; ++q) w[q] = load8(ap[q] + c * (kChunk * 2));
    };
    const auto step = [&](const u32x4 (&x)[XI], const u32x4 (&w)[AI]) {
#pragma unroll
      for (int q = 0; q < XI; ++q) st.put(q * 8 + pr, pc, x[q]);
#pragma unroll
      for (int q = 0; q < AI; ++q) st.put((XI + q) * 8 + pr, pc, w[q]);
      lds_order();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 xf[TM];
#pragma unroll
        for (int m = 0; m < TM; ++m) xf[m] = st.get(m, h);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const u32x4 af = st.get(TM + t, h);
#pragma unroll
          for (int m = 0; m < TM; ++m) acc[m][t] = Frag<TY>::mfma(af, xf[m], acc[m][t]);
        }
      }
      lds_order();
    };
    u32x4 x[D][XI], w[D][AI];
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (wave + d * NW < whole) fetch(wave + d * NW, x[d], w[d]);
    for (int i = wave; i < whole; i += D * NW) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i + (d + D - 1) * NW < whole) fetch(i + (d + D - 1) * NW, x[(d + D - 1) % D], w[(d + D - 1) % D]);
        if (i + d * NW < whole) step(x[d], w[d]);
      }
    }
    if (whole < chunks && whole % NW == wave) {   // the last columns, by the wave whose turn it is
      const int col = (c0 + whole) * kChunk + pc * 8;
#pragma unroll
      for (int q = 0; q < XI; ++q) x[0][q] = load8(xp[q] - pc * 16, col, a.K, a.K);
#pragma unroll
      for (int q = 0; q < AI; ++q) w[0][q] = load8(ap[q] - pc * 16, col, a.K, a.K);
      step(x[0], w[0]);
    }
    // the waves' sums, in wave order
    __syncthreads();
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) *(f32x4 *)&part.red[wave][m * kRows + l16][t * kRows + g * 4] = acc[m][t];
    __syncthreads();
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const int r = m * kRows + (tid >> 4);
      const bool mine = __shfl(tile.id[m], tid >> 4, kWave) == cur;
      float *z = a.z + ((int64_t)split * a.T + r0 + r) * a.R;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int j = t * kRows + (tid & 15);
        float v = part.red[0][r][j];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += part.red[w][r][j];
        if (mine && j0 + j < a.R) z[j0 + j] = v;
      }
    }
    __syncthreads();
  }
}

// out = y + scale_i B_i z: one workgroup per tile of 16 rows, `width` outputs
// and slot.  The waves take 64 outputs in turn (MFMA rows 16 t + m are outputs
// n0 + 16 t + m, columns the rows); the next turn's y and the next step's B (64
// ranks of one adapter) are loaded meanwhile.
template <int TY, int TO, int RM>
__global__ void __launch_bounds__(kAdapterThreads, RM == 16 && TO != MOEQ_F32 ? 4 : RM > 32 && TO == MOEQ_F32 ? 2 : 3)
adapters_up_kernel(AdapterArgs a) {
  constexpr int NW = kAdapterWaves, TERMS = TO == MOEQ_F32 ? 3 : 2, NT = RM / kRows;
  constexpr int PB = std::min(RM / 8, 8), BI = PB;   // pieces of a row of B; loads of 64 rows
  union Part {                              // of one wave, in turn
    Stage<64> in;
    OutTile out;
  };
  __shared__ Part part[NW];
  __shared__ ZTerms<1, NT, TERMS> zt;
  const Place place(a);
  const int r0 = place.tile * kRows, tid = threadIdx.x, lane = tid & 63, wave = wave_id(), l16 = lane & 15, g = lane >> 4;
  const int pr = lane >> 3, pc = lane & 7;
  if (place.tile >= a.tiles) return;
  Tile<1> tile;
  tile.load(a, r0);
  // this workgroup's adapters (lane q: the q-th of them) and rows
  int cur_of = -1, count = 0, row = 0;
  bool own = place.slot == 0 && tile.id[0] < 0 && r0 + l16 < a.T;
  {
    Turn turn(place);
    for (int cur = tile.next(row); cur >= 0; cur = tile.next(row))
      if (turn.mine(a)) {
        own |= tile.id[0] == cur;
        if (lane == count) cur_of = cur;
        ++count;
      }
  }
  if (!__ballot(own)) return;
  const int n1 = std::min(a.N, (place.part + 1) * a.width);
  // y and out along their rows: row pr + 8 h, outputs n0 + 8 pc ..
  const uint8_t *yp = (const uint8_t *)a.y + ((r0 + pr) * a.ldy + pc * 8) * Val<TO>::size;
  uint8_t *op = (uint8_t *)a.out + ((r0 + pr) * a.ldo + pc * 8) * Val<TO>::size;
  bool mine[2], plain[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    mine[h] = __shfl((int)own, h * 8 + pr, kWave);
    plain[h] = __shfl(tile.id[0], h * 8 + pr, kWave) < 0;
  }
  const auto load_y = [&](int n0, Oct<TO> (&y)[2]) {
    const int n = n0 + 64 <= a.N ? 8 : a.N - n0 - pc * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (mine[h]) y[h].load(yp, h * 8 * a.ldy + n0, n);
  };
  const int pb = lane % PB;
  const auto load_b = [&](int n0, int q, int k, u32x4 (&w)[BI]) {   // 64 ranks from k of the q-th adapter
    const int cur = __builtin_amdgcn_readlane(cur_of, q), rank = rank_of(a, cur);
    const uint8_t *base = (const uint8_t *)a.b + (cur * a.stride_b + n0 * a.ldb) * 2;
    if (n0 + 64 <= a.N && k + PB * 8 <= rank) {
      const uint8_t *at = base + (lane / PB * a.ldb + k + pb * 8) * 2;
#pragma unroll
      for (int i = 0; i < BI; ++i) w[i] = load8(at + i * (64 / PB) * a.ldb * 2);
    } else {
#pragma unroll
      for (int i = 0; i < BI; ++i)
        w[i] = load8(base + std::min(i * (64 / PB) + lane / PB, a.N - 1 - n0) * a.ldb * 2, k + pb * 8, a.R, rank);
    }
  };
  constexpr int DN = NW * 64;   // from turn to turn of a wave
  const int first = place.part * a.width + wave * 64;
  Oct<TO> y[2], yn[2];
  u32x4 w[BI];
  if (first < n1) {
    load_y(first, y);
    if (count) load_b(first, 0, 0, w);
  }
  {
    const int id = __shfl(tile.id[0], tid >> 4, kWave), j = tid & 15;
    float v[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) v[q] = 0.f;
    if (id >= 0) {
      const float *z = a.z + (int64_t)(r0 + (tid >> 4)) * a.R + j;
      constexpr int B = NT <= 2 ? 8 : NT <= 4 ? 4 : 2;   // parts of K loaded at a time
      for (int s = 0; s < a.splits; s += B) {
        float part[B][NT];
#pragma unroll
        for (int u = 0; u < B; ++u)
#pragma unroll
          for (int q = 0; q < NT; ++q)
            part[u][q] = s + u < a.splits && q * kRows + j < a.R ? z[(int64_t)(s + u) * a.T * a.R + q * kRows] : 0.f;
#pragma unroll
        for (int u = 0; u < B; ++u)
#pragma unroll
          for (int q = 0; q < NT; ++q) v[q] += part[u][q];
      }
      if (a.scale) {
        const float f = a.scale[id];
#pragma unroll
        for (int q = 0; q < NT; ++q) v[q] *= f;
      }
    }
    put_terms<TY>(zt, tid >> 4, v, id >= 0 ? rank_of(a, id) : 0);
  }
  __syncthreads();
  Stage<64> &st = part[wave].in;
  OutTile &ot = part[wave].out;
  for (int n0 = first; n0 < n1; n0 += DN) {
    const bool more = n0 + DN < n1;
    if (more) load_y(n0 + DN, yn);
    // the products with each adapter go to the rows that use it
    f32x4 res[4];
    for (int q = 0; q < count; ++q) {
      const int cur = __builtin_amdgcn_readlane(cur_of, q), rank = rank_of(a, cur);
      f32x4 acc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      int k = 0;
      do {
#pragma unroll
        for (int i = 0; i < BI; ++i) st.put(i * (64 / PB) + lane / PB, pb, w[i]);
        lds_order();
        const bool on = RM > 64 && k + 64 < rank, other = q + 1 < count;
        if (on || other || more) load_b(on || other ? n0 : n0 + DN, on ? q : other ? q + 1 : 0, on ? k + 64 : 0, w);
#pragma unroll
        for (int h = 0; h < (RM > 32 ? 2 : 1); ++h) {
          if (h && k + 32 >= rank) continue;
          u32x4 bf[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            bf[t] = st.get(t, h);
            if (RM == 16 && g >= 2) bf[t] = u32x4{0, 0, 0, 0};   // (no such ranks)
          }
#pragma unroll
          for (int e = 0; e < TERMS; ++e) {
            const u32x4 z = *(const u32x4 *)&zt.z[e][l16][k + h * 32 + g * 8];
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t] = Frag<TY>::mfma(bf[t], z, acc[t]);
          }
        }
        lds_order();
        k += 64;
      } while (RM > 64 && k < rank);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) res[t][i] = q == 0 || tile.id[0] == cur ? acc[t][i] : res[t][i];
    }
    if (count) {
#pragma unroll
      for (int t = 0; t < 4; ++t) *(f32x4 *)&ot.v[l16][t * kRows + g * 4] = res[t];
      lds_order();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 d[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) d[i] = *(const f32x4 *)&ot.v[h * 8 + pr][pc * 8 + i * 4];
      const int n = n0 + 64 <= a.N ? 8 : a.N - n0 - pc * 8;
      if (!mine[h] || n <= 0) continue;
      if (!plain[h]) {
        const float up = zt.up[h * 8 + pr];
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(d[i >> 2][i & 3], up, y[h][i]);
        y[h].pack(v);
      }
      y[h].template store<true>(op, h * 8 * a.ldo + n0, n);
    }
    lds_order();
#pragma unroll
    for (int h = 0; h < 2; ++h) y[h] = yn[h];
  }
}

// How a call is cut: rows per workgroup of the first kernel (16 tm), ranks it
// forms at a time (16 nt), parts of K.  Thirty-two rows read A_i half as often
// (4096 rows of 4096: 25.4 against 26.3 us for rank 16, 37.4 against 38.8 for
// 64) but leave few workgroups of short batches (256 rows: 17.1 us against
// 13.7).  K is cut into as many parts as give two workgroups a CU, each wave at
// least one chunk (one workgroup a CU: 4096 rows of rank 64 70 us where these
// took 59, four: 59).
constexpr int kLongBatch = 2048;
struct AdapterPlan {
  int tm, nt, groups, splits, per;
};
static AdapterPlan adapter_plan(int T, int R, int K) {
  AdapterPlan p;
  p.tm = T >= kLongBatch ? 2 : 1;
  p.nt = R <= 16 ? 1 : R <= 32 ? 2 : 4;
  p.groups = (R + p.nt * kRows - 1) / (p.nt * kRows);
  const int tiles = std::max(1, (T + p.tm * kRows - 1) / (p.tm * kRows)) * p.groups, chunks = (K + kChunk - 1) / kChunk;
  const int most = std::min(16, (chunks + kAdapterWaves - 1) / kAdapterWaves);
  p.splits = std::max(1, std::min(most, 512 / tiles));
  p.per = (chunks + p.splits - 1) / p.splits;
  p.splits = (chunks + p.per - 1) / p.per;
  return p;
}

// Workgroups that share a tile's adapters: as many as a tile can use, as long
// as the grid stays within the workgroups that the card holds at a time, 256
// times what the kernel's registers leave a CU: most of them have no work where
// rows of one adapter stand together, and beyond that they are in the way of
// those that have (1024 rows of rank 64 in runs of one adapter: 18.8 us with one
// a tile, 24 with two; 64 rows of 32 adapters of rank 16 in any order: 13.6 us
// with 16, 27.7 with one).
static int adapter_slots(const AdapterArgs &a, int rows, int most) {
  const int64_t wgs = (int64_t)a.tiles * a.parts;
  return (int)std::max((int64_t)1, std::min((int64_t)std::min(std::min(a.n, a.T), rows), most / wgs));
}

template <int TY, int TM, int NT, int D>
static void launch_down(AdapterArgs a, const AdapterPlan &p, hipStream_t s) {
  a.tiles = (a.T + TM * kRows - 1) / (TM * kRows);
  a.parts = p.splits * p.groups;
  a.slots = adapter_slots(a, TM * kRows, NT == 1 ? 1024 : NT == 2 ? 768 : 512);
  hipLaunchKernelGGL((adapters_down_kernel<TY, TM, NT, D>), place_grid(a), dim3(kAdapterThreads), 0, s, a);
}

template <int TY, int TO, int RM>
static void launch_up(AdapterArgs a, hipStream_t s) {
  a.tiles = (a.T + kRows - 1) / kRows;
  const int turn = kAdapterWaves * 64, turns = (a.N + turn - 1) / turn;
  // one round of what the card holds at a time, but no more than eight turns a
  // workgroup (8192 rows of 14336, rank 32: 163 us against 218 in one round)
  const int parts = std::max((turns + 7) / 8, std::min(turns, (RM == 16 ? 1024 : 768) / a.tiles));
  a.width = (turns + parts - 1) / parts * turn;
  a.parts = (a.N + a.width - 1) / a.width;
  a.slots = adapter_slots(a, kRows, RM == 16 ? 1024 : 768);
  hipLaunchKernelGGL((adapters_up_kernel<TY, TO, RM>), place_grid(a), dim3(kAdapterThreads), 0, s, a);
}

template <int TY, int TO>
static void launch_adapters(AdapterArgs a, hipStream_t s) {
  const AdapterPlan p = adapter_plan(a.T, a.R, a.K);
  a.splits = p.splits;
  a.per = p.per;
  if (p.tm == 2) {
    if (p.nt == 1) launch_down<TY, 2, 1, 3>(a, p, s);
    else if (p.nt == 2) launch_down<TY, 2, 2, 2>(a, p, s);
    else launch_down<TY, 2, 4, 2>(a, p, s);
  } else {
    if (p.nt == 1) launch_down<TY, 1, 1, 4>(a, p, s);
    else if (p.nt == 2) launch_down<TY, 1, 2, 3>(a, p, s);
    else launch_down<TY, 1, 4, 2>(a, p, s);
  }
  if (a.R <= 16) launch_up<TY, TO, 16>(a, s);
  else if (a.R <= 32) launch_up<TY, TO, 32>(a, s);
  else if (a.R <= 64) launch_up<TY, TO, 64>(a, s);
  else if (a.R <= 128) launch_up<TY, TO, 128>(a, s);
  else launch_up<TY, TO, 256>(a, s);
}

static size_t adapters_workspace(int T, int R, int K) { return (size_t)adapter_plan(T, R, K).splits * T * R * 4; }

static moeq_status check_adapter_sizes(const char *who, int32_t T, int32_t R, int32_t K) {
  if (T < 0) return fail(MOEQ_ERR_INVALID, "%s: negative T=%d", who, T);
  if (T > kMaxTokens) return fail(MOEQ_ERR_UNSUPPORTED, "%s: T=%d above %d", who, T, kMaxTokens);
  MOEQ_TRY(check_len(who, "R", R, kAdaptersMaxR));
  return check_len(who, "K", K, kMaxLen);
}

}  // namespace moeq

using namespace moeq;

MOEQ_API moeq_status moeq_adapters_workspace_size(int32_t T, int32_t R, int32_t K, size_t *bytes) {
  const char *who = "adapters_workspace_size";
  if (!bytes) return fail(MOEQ_ERR_INVALID, "%s: null bytes", who);
  MOEQ_TRY(check_adapter_sizes(who, T, R, K));
  *bytes = adapters_workspace(T, R, K);
  return MOEQ_OK;
}

MOEQ_API moeq_status moeq_adapters(const moeq_adapters_set *s, const void *x, int64_t ldx, const int32_t *ids, int32_t T,
                                   const void *y, int64_t ldy, void *out, int64_t ldo, int32_t y_dtype, void *ws,
                                   size_t ws_bytes, hipStream_t stream) {
  const char *who = "adapters";
  if (!s) return fail(MOEQ_ERR_INVALID, "%s: null adapters", who);
  MOEQ_TRY(check_adapter_sizes(who, T, s->R, s->K));
  MOEQ_TRY(check_len(who, "N", s->N, kMaxLen));
  MOEQ_TRY(check_len(who, "n", s->n, kAdaptersMaxN));
  if (!ok16(s->dtype)) return fail(MOEQ_ERR_INVALID, "%s: bad dtype %d", who, s->dtype);
  if (y_dtype != s->dtype && y_dtype != MOEQ_F32) return fail(MOEQ_ERR_INVALID, "%s: bad y_dtype %d", who, y_dtype);
  MOEQ_TRY(check_matrix(who, "a", s->a, s->lda, s->K, s->dtype));
  MOEQ_TRY(check_stride(who, "a", s->stride_a, s->R, s->lda, s->K, s->n, false));
  MOEQ_TRY(check_matrix(who, "b", s->b, s->ldb, s->R, s->dtype));
  MOEQ_TRY(check_stride(who, "b", s->stride_b, s->N, s->ldb, s->R, s->n, false));
  if (((uintptr_t)s->scale | (uintptr_t)s->ranks) & 3) return fail(MOEQ_ERR_INVALID, "%s: misaligned scale or ranks", who);
  if (!T) return MOEQ_OK;
  MOEQ_TRY(check_matrix(who, "x", x, ldx, s->K, s->dtype));
  MOEQ_TRY(check_matrix(who, "y", y, ldy, s->N, y_dtype));
  MOEQ_TRY(check_matrix(who, "out", out, ldo, s->N, y_dtype));
  if (!ids || ((uintptr_t)ids & 3)) return fail(MOEQ_ERR_INVALID, "%s: null or misaligned ids", who);
  const size_t need = adapters_workspace(T, s->R, s->K);
  if (need && (!ws || ((uintptr_t)ws & 15))) return fail(MOEQ_ERR_INVALID, "%s: null or misaligned workspace", who);
  if (ws_bytes < need) return fail(MOEQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, ws_bytes, need);
  AdapterArgs a{};
  a.x = x;
  a.a = s->a;
  a.b = s->b;
  a.y = y;
  a.out = out;
  a.ids = ids;
  a.ranks = s->ranks;
  a.scale = s->scale;
  a.z = (float *)ws;
  a.ldx = ldx;
  a.lda = s->lda;
  a.stride_a = s->stride_a;
  a.ldb = s->ldb;
  a.stride_b = s->stride_b;
  a.ldy = ldy;
  a.ldo = ldo;
  a.T = T;
  a.n = s->n;
  a.R = s->R;
  a.N = s->N;
  a.K = s->K;
  prof_begin("adapters", stream);
  if (s->dtype == MOEQ_F16) {
    if (y_dtype == MOEQ_F16) launch_adapters<MOEQ_F16, MOEQ_F16>(a, stream);
    else launch_adapters<MOEQ_F16, MOEQ_F32>(a, stream);
  } else {
    if (y_dtype == MOEQ_BF16) launch_adapters<MOEQ_BF16, MOEQ_BF16>(a, stream);
    else launch_adapters<MOEQ_BF16, MOEQ_F32>(a, stream);
  }
  prof_end("adapters", stream);
  return check_launch("adapters");
}
