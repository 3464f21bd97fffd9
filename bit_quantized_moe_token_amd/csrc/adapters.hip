// Low-rank adapters of many requests beside a shared projection:
// out[r] = y[r] + scale_i B_i (A_i x[r]), i = ids[r].
#include "check.hpp"
#include "vec8.hpp"

namespace moeq {

constexpr int kAdaptersMaxR = 256;
constexpr int kAdaptersMaxN = 1 << 20;

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kRows = 16;        // rows (tokens) of an MFMA tile
constexpr int kChunk = 64;       // columns of x and A that a wave takes at a time: 128 bytes of a row
constexpr int kCols = 256;       // outputs of a workgroup of the second kernel: 64 a wave

struct AdapterArgs {
  const void *x, *a, *b, *y;
  void *out;
  const int32_t *ids, *ranks;
  const float *scale;
  float *z;              // [splits, T, R]
  int64_t ldx, lda, stride_a, ldb, stride_b, ldy, ldo;
  int T, n, R, N, K;
  int splits, per;       // parts of K, chunks of each
  int slots;             // workgroups that share the adapters of a tile
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

// Eight 16-bit values at p, of which the first n exist (zeros behind them).
__device__ __forceinline__ u32x4 load8(const uint8_t *p) { return *(const __attribute__((address_space(1))) u32x4_a2 *)p; }
__device__ __forceinline__ u32x4 load8(const uint8_t *p, int n) {
  Oct<MOEQ_F16> o;
  o.load(p, 0, n);
  return u32x4{o.w[0], o.w[1], o.w[2], o.w[3]};
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

// Partial sums of z = A_i x over one part of K.  One workgroup per tile of
// 16 TM rows, part of K and slot; the waves take chunks of the part in turn,
// each the products of 16 TM rows with 16 NT rows of A_i, read straight into
// operand registers (an element of either feeds 16 products: nothing is gained
// by LDS).  Lane l takes columns 16 (l / 16) .. + 15 of a chunk, two MFMA steps
// of eight, so that four lanes read a row's 128 bytes.  Rows of the tile with
// another adapter (or none), and rows of A_i beyond its rank, read a valid row
// instead: they only reach outputs that are not stored.
template <int TY, int TM, int NT>
__global__ void __launch_bounds__(kThreads)
adapters_down_kernel(AdapterArgs a) {
  __shared__ float red[kWaves][TM * kRows][kRows + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.x * (TM * kRows);
  const int c0 = blockIdx.y * a.per, c1 = std::min(c0 + a.per, (a.K + kChunk - 1) / kChunk);
  Tile<TM> tile;
  tile.load(a, r0);
  int slot = 0, row = 0;
  for (int cur = tile.next(row); cur >= 0; cur = tile.next(row)) {
    const bool mine = slot == (int)blockIdx.z;
    slot = slot + 1 == a.slots ? 0 : slot + 1;
    if (!mine) continue;
    const int rank = rank_of(a, cur);
    if (!rank) continue;
    const uint8_t *xp[TM], *ap[NT];
#pragma unroll
    for (int m = 0; m < TM; ++m)
      xp[m] = (const uint8_t *)a.x + ((r0 + (tile.id[m] == cur ? m * kRows + l16 : row)) * a.ldx + g * 16) * 2;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int j = t * kRows + l16;
      ap[t] = (const uint8_t *)a.a + (cur * a.stride_a + (j < rank ? j : 0) * a.lda + g * 16) * 2;
    }
    f32x4 acc[TM][NT];
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const auto step = [&](const u32x4 (&x)[TM][2], const u32x4 (&w)[NT][2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[m][t] = Frag<TY>::mfma(w[t][h], x[m][h], acc[m][t]);
    };
    const int whole = std::min(c1, a.K / kChunk);
    const auto fetch = [&](int c, u32x4 (&x)[TM][2], u32x4 (&w)[NT][2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int m = 0; m < TM; ++m) x[m][h] = load8(xp[m] + c * (kChunk * 2) + h * 16);
#pragma unroll
        for (int t = 0; t < NT; ++t) w[t][h] = load8(ap[t] + c * (kChunk * 2) + h * 16);
      }
    };
    int c = c0 + wave;
    if constexpr (NT <= 4)
      for (; c + kWaves < whole; c += 2 * kWaves) {   // two chunks in flight
        u32x4 x0[TM][2], w0[NT][2], x1[TM][2], w1[NT][2];
        fetch(c, x0, w0);
        fetch(c + kWaves, x1, w1);
        step(x0, w0);
        step(x1, w1);
      }
    for (; c < whole; c += kWaves) {
      u32x4 x[TM][2], w[NT][2];
      fetch(c, x, w);
      step(x, w);
    }
    if (c < c1) {   // the last columns
      u32x4 x[TM][2], w[NT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = a.K - c * kChunk - g * 16 - h * 8;
#pragma unroll
        for (int m = 0; m < TM; ++m) x[m][h] = load8(xp[m] + c * (kChunk * 2) + h * 16, n);
#pragma unroll
        for (int t = 0; t < NT; ++t) w[t][h] = load8(ap[t] + c * (kChunk * 2) + h * 16, n);
      }
      step(x, w);
    }
    // the waves' sums, 16 ranks at a time, in wave order
    float *z = a.z + ((int64_t)blockIdx.y * a.T + r0) * a.R;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t * kRows >= rank) continue;
      __syncthreads();
#pragma unroll
      for (int m = 0; m < TM; ++m) *(f32x4 *)&red[wave][m * kRows + l16][g * 4] = acc[m][t];
      __syncthreads();
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const int r = m * kRows + (tid >> 4), j = tid & 15;
        const int id = __shfl(tile.id[m], tid >> 4, kWave);
        if (id == cur && t * kRows + j < rank) {
          float s = red[0][r][j];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) s += red[w][r][j];
          z[(int64_t)r * a.R + t * kRows + j] = s;
        }
      }
    }
  }
}

// out = y + scale_i B_i z.  One workgroup per tile of 16 TM rows, 256 outputs
// and slot.  z is summed over the parts of K, brought to a power of two near 1
// per row and split into TERMS 16-bit numbers, whose products with B_i are
// exact in the MFMA: two terms keep 22 bits of it in fp16 and 16 in bf16, more
// than a 16-bit output shows; an fp32 output takes three.  The MFMA's rows
// are outputs, dealt so that a lane ends with 16 consecutive ones of one row.
template <int TY, int TO, int TM, int NT>
__global__ void __launch_bounds__(kThreads)
adapters_up_kernel(AdapterArgs a) {
  constexpr int TERMS = TO == MOEQ_F32 ? 3 : 2;
  constexpr int RP = (NT + 1) / 2 * 32, LD = RP + 8;
  __shared__ __attribute__((aligned(16))) uint16_t zs[TERMS][TM * kRows][LD];
  __shared__ int s_exp[TM * kRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.x * (TM * kRows), n0 = blockIdx.y * kCols + wave * 64;
  Tile<TM> tile;
  tile.load(a, r0);
  // the rows that this workgroup writes: those of its share of the adapters,
  // and slot 0 those without one
  bool own[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m) own[m] = blockIdx.z == 0 && tile.id[m] < 0 && r0 + m * kRows + l16 < a.T;
  int slot = 0, row = 0;
  for (int cur = tile.next(row); cur >= 0; cur = tile.next(row)) {
    if (slot == (int)blockIdx.z) {
#pragma unroll
      for (int m = 0; m < TM; ++m) own[m] |= tile.id[m] == cur;
    }
    slot = slot + 1 == a.slots ? 0 : slot + 1;
  }
  bool any = false;
#pragma unroll
  for (int m = 0; m < TM; ++m) any |= own[m];
  if (!__ballot(any)) return;
  Oct<TO> y[TM][2];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = n0 + g * 16 + h * 8;
      if (own[m] && c < a.N) y[m][h].load(a.y, (r0 + m * kRows + l16) * a.ldy + c, a.N - c);
    }
  // z of row m * 16 + tid / 16, ranks tid % 16 + 16 q
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int r = m * kRows + (tid >> 4), id = __shfl(tile.id[m], tid >> 4, kWave);
    const int rank = id >= 0 ? rank_of(a, id) : 0;
    float v[RP / kRows], top = 0.f;
#pragma unroll
    for (int q = 0; q < RP / kRows; ++q) {
      const int j = (tid & 15) + q * kRows;
      v[q] = 0.f;
      if (j < rank) {
        const float *p = a.z + (int64_t)(r0 + r) * a.R + j;
        v[q] = p[0];
        for (int s = 1; s < a.splits; ++s) v[q] += p[(int64_t)s * a.T * a.R];
      }
      const float f = __builtin_fabsf(v[q]);
      if (f < __builtin_inff()) top = __builtin_fmaxf(top, f);
    }
    top = dpp_row_max(top);
    const int e = top > 0.f ? ilogb_f32(top) : 0;
    if ((tid & 15) == 0) s_exp[r] = e;
#pragma unroll
    for (int q = 0; q < RP / kRows; ++q) {
      float rest = __builtin_ldexpf(v[q], -e);
#pragma unroll
      for (int t = 0; t < TERMS; ++t) {
        const uint32_t bits = Val<TY>::put(rest);
        zs[t][r][(tid & 15) + q * kRows] = (uint16_t)bits;
        // (an infinity or NaN is in the first term whole)
        rest = __builtin_fabsf(rest) < __builtin_inff() ? rest - Val<TY>::get(bits) : 0.f;
      }
    }
  }
  __syncthreads();
  f32x4 sum[TM][4];
  tile.restart();
  slot = 0;
  bool served[TM];
  float factor[TM];
  int expo[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    served[m] = false;
    expo[m] = s_exp[m * kRows + l16];
    factor[m] = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) sum[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  for (int cur = tile.next(row); cur >= 0; cur = tile.next(row)) {
    const bool mine = slot == (int)blockIdx.z;
    slot = slot + 1 == a.slots ? 0 : slot + 1;
    if (!mine) continue;
    const int rank = rank_of(a, cur);
    if (!rank) continue;
    const uint8_t *bp[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      // row l16 of MFMA tile t is output 16 (l16 / 4) + 4 t + l16 % 4
      const int c = std::min(n0 + (l16 >> 2) * 16 + t * 4 + (l16 & 3), a.N - 1);
      bp[t] = (const uint8_t *)a.b + (cur * a.stride_b + c * a.ldb + g * 8) * 2;
    }
    f32x4 acc[TM][4];
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < RP; k += 32) {
      if (k >= rank) continue;
      u32x4 w[4];
      if (k + 32 <= rank) {
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = load8(bp[t] + k * 2);
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = load8(bp[t] + k * 2, rank - k - g * 8);
      }
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int q = 0; q < TERMS; ++q) {
          const u32x4 z = *(const u32x4 *)&zs[q][m * kRows + l16][k + g * 8];
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[m][t] = Frag<TY>::mfma(w[t], z, acc[m][t]);
        }
    }
    const float f = a.scale ? a.scale[cur] : 1.f;
#pragma unroll
    for (int m = 0; m < TM; ++m)
      if (tile.id[m] == cur) {
        served[m] = true;
        factor[m] = f;
#pragma unroll
        for (int t = 0; t < 4; ++t) sum[m][t] = acc[m][t];
      }
  }
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = n0 + g * 16 + h * 8;
      if (!own[m] || c >= a.N) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = factor[m] * __builtin_ldexpf(sum[m][h * 2 + (i >> 2)][i & 3], expo[m]);
        v[i] = served[m] ? y[m][h][i] + d : y[m][h][i];
      }
      Oct<TO> o;
      o.pack(v);
      o.store(a.out, (r0 + m * kRows + l16) * a.ldo + c, a.N - c);
    }
}

// How a call is cut: rows per workgroup, parts of K.
struct AdapterPlan {
  int tm, splits, per;
};
static AdapterPlan adapter_plan(int T, int R, int K) {
  AdapterPlan p;
  p.tm = T >= 512 && R <= 64 ? 4 : 1;
  const int tiles = (T + p.tm * kRows - 1) / (p.tm * kRows), chunks = (K + kChunk - 1) / kChunk;
  const int most = std::min(16, (chunks + kWaves - 1) / kWaves);
  p.splits = std::max(1, std::min(most, 256 / std::max(tiles, 1)));
  p.per = (chunks + p.splits - 1) / p.splits;
  p.splits = (chunks + p.per - 1) / p.per;
  return p;
}

template <int TY, int TO, int TM, int NT>
static void launch_adapters(AdapterArgs a, hipStream_t s) {
  const int tiles = (a.T + TM * kRows - 1) / (TM * kRows), cols = (a.N + kCols - 1) / kCols;
  const int most = std::min(a.n, TM * kRows);
  a.slots = std::max(1, std::min(most, 2048 / (tiles * a.splits)));
  hipLaunchKernelGGL((adapters_down_kernel<TY, TM, NT>), dim3(tiles, a.splits, a.slots), dim3(kThreads), 0, s, a);
  a.slots = (int)std::max((int64_t)1, std::min((int64_t)most, 4096 / ((int64_t)tiles * cols)));
  hipLaunchKernelGGL((adapters_up_kernel<TY, TO, TM, NT>), dim3(tiles, cols, a.slots), dim3(kThreads), 0, s, a);
}

template <int TY, int TO>
static void launch_adapters_r(AdapterArgs a, hipStream_t s) {
  const AdapterPlan p = adapter_plan(a.T, a.R, a.K);
  a.splits = p.splits;
  a.per = p.per;
  if (p.tm == 4) {
    if (a.R <= 16) launch_adapters<TY, TO, 4, 1>(a, s);
    else if (a.R <= 32) launch_adapters<TY, TO, 4, 2>(a, s);
    else launch_adapters<TY, TO, 4, 4>(a, s);
  } else {
    if (a.R <= 16) launch_adapters<TY, TO, 1, 1>(a, s);
    else if (a.R <= 32) launch_adapters<TY, TO, 1, 2>(a, s);
    else if (a.R <= 64) launch_adapters<TY, TO, 1, 4>(a, s);
    else if (a.R <= 128) launch_adapters<TY, TO, 1, 8>(a, s);
    else launch_adapters<TY, TO, 1, 16>(a, s);
  }
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
  if (!ws || ((uintptr_t)ws & 15)) return fail(MOEQ_ERR_INVALID, "%s: null or misaligned workspace", who);
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
    if (y_dtype == MOEQ_F16) launch_adapters_r<MOEQ_F16, MOEQ_F16>(a, stream);
    else launch_adapters_r<MOEQ_F16, MOEQ_F32>(a, stream);
  } else {
    if (y_dtype == MOEQ_BF16) launch_adapters_r<MOEQ_BF16, MOEQ_BF16>(a, stream);
    else launch_adapters_r<MOEQ_BF16, MOEQ_F32>(a, stream);
  }
  prof_end("adapters", stream);
  return check_launch("adapters");
}
