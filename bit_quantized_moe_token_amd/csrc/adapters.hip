// Low-rank adapters of many requests beside a shared projection:
// out[r] = y[r] + scale_i B_i (A_i x[r]), i = ids[r].
#include "check.hpp"
#include "vec8.hpp"

namespace moeq {

constexpr int kAdaptersMaxR = 256;
constexpr int kAdaptersMaxN = 1 << 20;

struct AdapterArgs {
  const void *x, *a, *b, *y;
  void *out;
  const int32_t *ids, *ranks;
  const float *scale;
  float *z;              // [T, R]
  int64_t ldx, lda, stride_a, ldb, stride_b, ldy, ldo;
  int T, n, R, N, K;
};

// Adapter of row r: its number (-1: none) and its rank.
struct Adapter {
  int id, rank;
};
__device__ __forceinline__ Adapter adapter_of(const AdapterArgs &a, int r) {
  int id = a.ids[r];
  if ((uint32_t)id >= (uint32_t)a.n) return {-1, 0};
  const int rank = a.ranks ? a.ranks[id] : a.R;
  return {id, rank < 0 ? 0 : rank > a.R ? a.R : rank};
}

// z[r, j] = A_i[j] . x[r]: a wave per row and j.
template <int TY>
__global__ void __launch_bounds__(256)
adapters_down_kernel(AdapterArgs a) {
  const int r = blockIdx.x, lane = threadIdx.x & 63;
  const int j = blockIdx.y * 4 + (threadIdx.x >> 6);
  const Adapter ad = adapter_of(a, r);
  if (j >= ad.rank) return;
  float acc = 0.f;
  for (int c = lane * 8; c < a.K; c += kWave * 8) {
    Oct<TY> x, w;
    x.load(a.x, r * a.ldx + c, a.K - c);
    w.load(a.a, ad.id * a.stride_a + j * a.lda + c, a.K - c);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc += x[i] * w[i];
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) acc += __shfl_xor(acc, m, kWave);
  if (lane == 0) a.z[(int64_t)r * a.R + j] = acc;
}

template <int TY, int TO>
__global__ void __launch_bounds__(256)
adapters_up_kernel(AdapterArgs a) {
  const int r = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 8, n = a.N - c;
  if (n <= 0) return;
  const Adapter ad = adapter_of(a, r);
  Oct<TO> y;
  y.load(a.y, r * a.ldy + c, n);
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int j = 0; j < ad.rank; ++j) {
    const float z = a.z[(int64_t)r * a.R + j];
    for (int i = 0; i < 8 && i < n; ++i) {
      const uint8_t *p = (const uint8_t *)a.b + (ad.id * a.stride_b + (c + i) * a.ldb + j) * Val<TY>::size;
      acc[i] += z * Val<TY>::get(gld<uint16_t>(p));
    }
  }
  const float s = ad.id < 0 ? 0.f : a.scale ? a.scale[ad.id] : 1.f;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = ad.rank ? y[i] + s * acc[i] : y[i];
  Oct<TO> o;
  o.pack(v);
  o.store(a.out, r * a.ldo + c, n);
}

template <int TY, int TO>
static void launch_adapters(const AdapterArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((adapters_down_kernel<TY>), dim3(a.T, (a.R + 3) / 4), dim3(256), 0, s, a);
  hipLaunchKernelGGL((adapters_up_kernel<TY, TO>), dim3(a.T, (a.N + 2047) / 2048), dim3(256), 0, s, a);
}

static size_t adapters_workspace(int T, int R) { return (size_t)T * R * 4; }

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
  *bytes = adapters_workspace(T, R);
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
  const size_t need = adapters_workspace(T, s->R);
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
    if (y_dtype == MOEQ_F16) launch_adapters<MOEQ_F16, MOEQ_F16>(a, stream);
    else launch_adapters<MOEQ_F16, MOEQ_F32>(a, stream);
  } else {
    if (y_dtype == MOEQ_BF16) launch_adapters<MOEQ_BF16, MOEQ_BF16>(a, stream);
    else launch_adapters<MOEQ_BF16, MOEQ_F32>(a, stream);
  }
  prof_end("adapters", stream);
  return check_launch("adapters");
}
