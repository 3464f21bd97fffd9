// The experts' rows back to their tokens, weighted by the gates, and the
// gradients of rows and gates.  Both are bound by their bytes: 4096 tokens of
// six rows of 2048 in bf16 23.0 us (134 MB, 5.8 TB/s), their gradients 38.9 us
// (218 MB, 5.6 TB/s).
//
// Past the caches or not, each against the other way (us): rows of more than 80
// MiB are read past them (4096 tokens of six rows of 2048: 23.0 / 25.6, the
// gradients 38.9 / 46.4), fewer by ordinary loads (1024 of eight, 32 MiB: 8.5 /
// 9.3 and 15.3 / 16.7; 333 of four rows of 757: 4.3 / 5.4 and 6.3 / 8.2; at 80 MiB
// 18.5 / 19.0 and 33.0 / 35.0).  Tokens' outputs are always written past them
// (23.0 / 24.7, small ones within 0.2).  Gradients of rows only where the rows
// are read by ordinary loads (2048 tokens of six: 19.7 / 22.7): of more they are
// slower so (40.6 / 38.9), and so is the product that reads them next (both
// together 210 / 200).
#include "check.hpp"
#include "vec8.hpp"
#include "wave.hpp"

namespace moeq {

constexpr int kCombineThreads = 256;
constexpr int kMaxSlots = 256;   // pairs per token

struct CombineArgs {
  const void *rows;      // [P, N]
  const int32_t *pos;    // [T * k]
  const float *gates;    // [T * k] or null (ones)
  const void *tok;       // base [T, N] or null; gradient: dy [T, N]
  void *out;             // [T, N]; gradient: d_rows [P, N]
  float *d_gates;        // gradient: [T * k] or null
  int64_t ldr, ldt, ldo;
  int T, k, N, P;
  int lanes;             // forward: log2 of the threads along a row
};
constexpr int64_t kBigRows = (int64_t)80 << 20;   // bytes of the pairs' rows, see above

// TR: type of the rows, TO: of base and out.  2^lanes threads along a row,
// eight columns each; four rows under way at a time (decoding steps and long
// batches: 3.0 and 25.4 us, one at a time 3.0 and 27.2, eight 3.2 and 24.7).
template <int TR, int TO, bool BIG>
__global__ void __launch_bounds__(kCombineThreads)
combine_kernel(CombineArgs a) {
  constexpr int SLOTS = 4;
  const int t = blockIdx.x * (kCombineThreads >> a.lanes) + (threadIdx.x >> a.lanes);
  const int c = ((blockIdx.y << a.lanes) + (threadIdx.x & ((1 << a.lanes) - 1))) * 8;
  const int n = a.N - c;
  if (t >= a.T || n <= 0) return;
  float acc[8];
  if (a.tok) {
    Oct<TO> b;
    b.template load<BIG>(a.tok, t * a.ldt + c, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  }
  for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
    const int64_t p = (int64_t)t * a.k + j0;
    int at[SLOTS];
    float g[SLOTS];
    Oct<TR> r[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      at[j] = j0 + j < a.k ? a.pos[p + j] : -1;
      g[j] = j0 + j < a.k && a.gates ? a.gates[p + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
      if ((uint32_t)at[j] < (uint32_t)a.P) r[j].template load<BIG>(a.rows, at[j] * a.ldr + c, n);
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
      if ((uint32_t)at[j] < (uint32_t)a.P) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += g[j] * r[j][i];
      }
  }
  Oct<TO> o;
  o.pack(acc);
  o.template store<true>(a.out, t * a.ldo + c, n);
}

// One workgroup per token: dy is read once for SLOTS pairs at a time, whose rows
// are all loaded before the first is used.
template <int TR, int TO, bool BIG>
__global__ void __launch_bounds__(kCombineThreads)
combine_grad_kernel(CombineArgs a) {
  constexpr int SLOTS = TR == MOEQ_F32 ? 4 : 8, NW = kCombineThreads / kWave;
  __shared__ float part[2][NW][SLOTS];
  const int t = blockIdx.x, tid = threadIdx.x;
  for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
    int at[SLOTS];
    float g[SLOTS], dot[SLOTS];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      const int64_t p = (int64_t)t * a.k + j0 + j;
      const bool in = j0 + j < a.k;
      at[j] = in ? a.pos[p] : -1;
      g[j] = in && a.gates ? a.gates[p] : 1.f;
      if ((uint32_t)at[j] >= (uint32_t)a.P) at[j] = -1;
      dot[j] = 0.f;
    }
    for (int c = tid * 8; c < a.N; c += kCombineThreads * 8) {
      const int n = a.N - c;
      Oct<TO> d;
      Oct<TR> r[SLOTS];
      d.template load<BIG>(a.tok, t * a.ldt + c, n);
      if (a.d_gates) {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
          if (at[j] >= 0) r[j].template load<BIG>(a.rows, at[j] * a.ldr + c, n);
      }
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        if (at[j] < 0) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = g[j] * d[i];
          if (a.d_gates) dot[j] += d[i] * r[j][i];
        }
        Oct<TR> o;
        o.pack(v);
        o.template store<!BIG>(a.out, at[j] * a.ldo + c, n);
      }
    }
    if (!a.d_gates) continue;
    // (two halves in turn: a wave may be in the next slots before all have read)
    float (*p)[SLOTS] = part[(j0 / SLOTS) & 1];
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
      const float v = all_sum(dot[j]);
      if ((tid & 63) == 0) p[tid >> 6][j] = v;
    }
    __syncthreads();
    if (tid < SLOTS && j0 + tid < a.k) {
      float v = p[0][tid];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += p[w][tid];
      a.d_gates[(int64_t)t * a.k + j0 + tid] = v;
    }
  }
}

template <int TR, int TO, bool BIG>
static void launch_combine_sized(CombineArgs a, bool grad, hipStream_t s) {
  if (grad) {
    hipLaunchKernelGGL((combine_grad_kernel<TR, TO, BIG>), dim3(a.T), dim3(kCombineThreads), 0, s, a);
    return;
  }
  a.lanes = 0;
  while (a.lanes < 8 && (8 << a.lanes) < a.N) ++a.lanes;
  const int per = kCombineThreads >> a.lanes, cols = 8 << a.lanes;
  hipLaunchKernelGGL((combine_kernel<TR, TO, BIG>), dim3((a.T + per - 1) / per, (a.N + cols - 1) / cols),
                     dim3(kCombineThreads), 0, s, a);
}

template <int TR, int TO>
static void launch_combine(const CombineArgs &a, bool grad, hipStream_t s) {
  if ((int64_t)a.T * a.k * a.N * Val<TR>::size > kBigRows) launch_combine_sized<TR, TO, true>(a, grad, s);
  else launch_combine_sized<TR, TO, false>(a, grad, s);
}

static void launch_combine_types(const CombineArgs &a, int tr, int to, bool grad, hipStream_t s) {
  if (tr == MOEQ_F16) {
    if (to == MOEQ_F16) launch_combine<MOEQ_F16, MOEQ_F16>(a, grad, s);
    else launch_combine<MOEQ_F16, MOEQ_F32>(a, grad, s);
  } else if (tr == MOEQ_BF16) {
    if (to == MOEQ_BF16) launch_combine<MOEQ_BF16, MOEQ_BF16>(a, grad, s);
    else launch_combine<MOEQ_BF16, MOEQ_F32>(a, grad, s);
  } else {
    if (to == MOEQ_F16) launch_combine<MOEQ_F32, MOEQ_F16>(a, grad, s);
    else if (to == MOEQ_BF16) launch_combine<MOEQ_F32, MOEQ_BF16>(a, grad, s);
    else launch_combine<MOEQ_F32, MOEQ_F32>(a, grad, s);
  }
}

static moeq_status check_combine(const char *who, int32_t P, int32_t dtype, const int32_t *pos, const float *gates,
                                 int32_t T, int32_t k, int32_t N, int32_t other) {
  if (T < 0 || P < 0) return fail(MOEQ_ERR_INVALID, "%s: negative T=%d or P=%d", who, T, P);
  if (k < 1 || k > kMaxSlots) return fail(MOEQ_ERR_INVALID, "%s: k=%d not in 1..%d", who, k, kMaxSlots);
  if (T > kMaxTokens || P > kMaxRows || (int64_t)T * k > kMaxRows)
    return fail(MOEQ_ERR_UNSUPPORTED, "%s: T=%d above %d, or P=%d or T*k above %d", who, T, kMaxTokens, P, kMaxRows);
  MOEQ_TRY(check_len(who, "N", N, kMaxLen));
  if (!okout(dtype)) return fail(MOEQ_ERR_INVALID, "%s: bad dtype %d", who, dtype);
  if (!okout(other) || (other != dtype && other != MOEQ_F32 && dtype != MOEQ_F32))
    return fail(MOEQ_ERR_INVALID, "%s: dtype %d beside rows of dtype %d", who, other, dtype);
  if (T && (!pos || ((uintptr_t)pos & 3))) return fail(MOEQ_ERR_INVALID, "%s: null or misaligned pair_pos", who);
  if ((uintptr_t)gates & 3) return fail(MOEQ_ERR_INVALID, "%s: misaligned gates", who);
  return MOEQ_OK;
}

}  // namespace moeq

using namespace moeq;

MOEQ_API moeq_status moeq_combine(const void *rows, int64_t ldr, int32_t P, int32_t dtype, const int32_t *pair_pos,
                                  const float *gates, int32_t T, int32_t k, int32_t N, const void *base, int64_t ldb,
                                  void *out, int64_t ldo, int32_t out_dtype, hipStream_t stream) {
  const char *who = "combine";
  MOEQ_TRY(check_combine(who, P, dtype, pair_pos, gates, T, k, N, out_dtype));
  if (!T) return MOEQ_OK;
  if (P) MOEQ_TRY(check_matrix(who, "rows", rows, ldr, N, dtype));
  if (base) MOEQ_TRY(check_matrix(who, "base", base, ldb, N, out_dtype));
  MOEQ_TRY(check_matrix(who, "out", out, ldo, N, out_dtype));
  CombineArgs a{};
  a.rows = rows;
  a.pos = pair_pos;
  a.gates = gates;
  a.tok = base;
  a.out = out;
  a.ldr = ldr;
  a.ldt = ldb;
  a.ldo = ldo;
  a.T = T;
  a.k = k;
  a.N = N;
  a.P = P;
  prof_begin("combine", stream);
  launch_combine_types(a, dtype, out_dtype, false, stream);
  prof_end("combine", stream);
  return check_launch("combine");
}

MOEQ_API moeq_status moeq_combine_grad(const void *dy, int64_t ldy, int32_t dy_dtype, const int32_t *pair_pos,
                                       const float *gates, int32_t T, int32_t k, int32_t N, const void *rows,
                                       int64_t ldr, int32_t P, int32_t dtype, void *d_rows, int64_t ldd, float *d_gates,
                                       hipStream_t stream) {
  const char *who = "combine_grad";
  MOEQ_TRY(check_combine(who, P, dtype, pair_pos, gates, T, k, N, dy_dtype));
  if (d_gates && !gates) return fail(MOEQ_ERR_INVALID, "%s: d_gates without gates", who);
  if ((uintptr_t)d_gates & 3) return fail(MOEQ_ERR_INVALID, "%s: misaligned d_gates", who);
  if (!T) return MOEQ_OK;
  MOEQ_TRY(check_matrix(who, "dy", dy, ldy, N, dy_dtype));
  if (P) {
    if (d_gates) MOEQ_TRY(check_matrix(who, "rows", rows, ldr, N, dtype));
    MOEQ_TRY(check_matrix(who, "d_rows", d_rows, ldd, N, dtype));
  }
  CombineArgs a{};
  a.rows = rows;
  a.pos = pair_pos;
  a.gates = gates;
  a.tok = dy;
  a.out = d_rows;
  a.d_gates = d_gates;
  a.ldr = ldr;
  a.ldt = ldy;
  a.ldo = ldd;
  a.T = T;
  a.k = k;
  a.N = N;
  a.P = P;
  prof_begin("combine_grad", stream);
  launch_combine_types(a, dtype, dy_dtype, true, stream);
  prof_end("combine_grad", stream);
  return check_launch("combine_grad");
}
