// Norms around a block: the block's output is normed, gated and added to the
// scaled residual, and the sum is normed for the next block, in one pass
// over the rows; and the gradients of all of it.  (What joins expert layers:
// the layer's y becomes the next layer's x.)
//
//   b = 1 / sqrt(mean(y^2) + eps),   p = w_post * y * b   (p = y without post norm)
//   r' = alpha r + gate * p          rounded to the residual's type
//   a = 1 / sqrt(mean(r'^2) + eps),  n = w_pre * r' * a
//
// Gradients from d_r' and d_n (u = r' a, v = y b, mean over the row):
//   g = d_n w_pre,   dr = d_r' + a (g - u mean(g u)),   d_r = alpha dr
//   c = dr gate w_post,  d_y = b (c - v mean(c v))      (d_y = dr gate without post norm)
//   d_w_pre = sum_t d_n u,  d_w_post = sum_t dr gate v,  d_gate = dr p (summed
//   over the tokens for a gate that all tokens share)
//
// Bound by memory: every row is read once and kept in registers (as stored)
// through the row's two reductions (16384 rows of 4096, bf16 beside an fp32
// residual: 150 us, 5.4 TB/s; gradients of 8192 rows of 4096 in bf16 with a
// gate per token: 123 us and 5 for the column sums, 4.2 TB/s); the gradients
// of rows above 8192 values read theirs twice.  Sums, statistics and gradients
// are fp32; the backward pass reads the rows in any case, so it recomputes 1 /
// a and 1 / b from them and needs no saved statistics.
#include "vec8.hpp"

namespace moeq {

struct NormArgs {
  const void *res, *y, *w_pre, *w_post, *gate;
  const void *d_res, *d_n;
  void *res_out, *n, *d_y, *d_r, *d_gate;
  float *part;                       // [units][3][H] column sums of each run of rows
  struct RowStats *stats;            // [T], wide rows only; null: no column sum is wanted
  int64_t ld_gate;                   // 0: one gate row for all tokens
  int32_t T, H, post, cols;          // cols: any column sum is wanted
  float alpha, eps;
};

__device__ __forceinline__ float scalar(float v) {   // a value that all lanes have
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// Sums of N values over the NT threads of a row, in scalar registers.  NT >
// 64: the waves' sums meet in LDS; the caller alternates `buf` (0, 1) between
// reductions, so that one barrier each is enough.
template <int NT, int N>
__device__ __forceinline__ void row_sum(float *v, float *s, int buf) {
#pragma unroll
  for (int o = 32; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], o, kWave);
  if constexpr (NT > 64) {
    constexpr int NW = NT / 64;
    float *p = s + buf * 3 * 16;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i * 16 + (threadIdx.x >> 6)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v[i] += p[i * 16 + w];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = scalar(v[i]);
}

// The largest of the NT threads' values, buf as above.
template <int NT>
__device__ __forceinline__ float row_top(float v, float *s, int buf) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o, kWave));
  if constexpr (NT > 64) {
    float *p = s + buf * 3 * 16;
    if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
    __syncthreads();
    v = p[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v = __builtin_fmaxf(v, p[w]);
  }
  return scalar(v);
}

// mean(v^2) + eps in fp32 is as good as the sum of squares, which is exact to
// its roundings between these.  Beyond them (rows of bf16 and fp32 values
// around 2^64 and more; values that vanish when squared beside an eps as
// small) the row is summed again, times row_unit.
__device__ __forceinline__ bool plain_square(float q) { return q >= 0x1p-90f && q < __builtin_inff(); }

// The power of two that brings the larger of a row's largest magnitude and
// sqrt(eps) to between 1 and 2 (2^-127 for an infinite one): no square
// overflows then, and what vanishes does not count beside 1.
__device__ __forceinline__ float row_unit(float top, float eps) {
  return __builtin_ldexpf(1.f, -std::min(ilogb_f32(__builtin_fmaxf(top, __builtin_sqrtf(eps))), 127));
}

// Threads per workgroup: a row's NT, or four waves of one row each.
constexpr int norm_block(int NT) { return NT == 64 ? 256 : NT; }

// 1 / sqrt(mean(v^2) + eps) of the row whose pieces the threads hold, zeros
// behind its end, from this thread's sum of squares.  Uses buffers buf, 2 and
// 3 of s.
template <int NT, int TV, int CH>
__device__ __forceinline__ float inverse_rms(const Oct<TV> (&v)[CH], float sum, float rh, float eps, float *s, int buf) {
  float ss[1] = {sum};
  row_sum<NT, 1>(ss, s, buf);
  const float q = ss[0] * rh + eps;
  if (__builtin_expect(plain_square(q), 1)) return 1.f / __builtin_sqrtf(q);
  // (opaque: the compiler would share fp32 values of the row with the usual
  // path, whose registers they would take)
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    Oct<TV> w = v[c];
    w.opaque();
#pragma unroll
    for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, __builtin_fabsf(w[j]));
  }
  const float u = row_unit(row_top<NT>(top, s, 2), eps);
  ss[0] = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    Oct<TV> w = v[c];
    w.opaque();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = w[j] * u;
      ss[0] += x * x;
    }
  }
  row_sum<NT, 1>(ss, s, 3);
  return u / __builtin_sqrtf(ss[0] * rh + eps * u * u);
}

// Thread t of a row holds the pieces of eight elements t, t + NT, ...
template <int TY, int TR, int NT, int CH>
__global__ void __launch_bounds__(norm_block(NT)) block_norm_kernel(NormArgs a) {
  __shared__ float s[4 * 3 * 16];
  const int t = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * (norm_block(NT) / NT) + threadIdx.x / NT;
  if (row >= a.T) return;      // (whole waves, and only where no barrier follows)
  const int64_t at = row * a.H;
  const float rh = 1.f / (float)a.H;
  Oct<TR> r[CH];
  Oct<TY> x[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * NT + t) * 8;
    r[c].load(a.res, at + i, a.H - i);
    if (a.y) x[c].load(a.y, at + i, a.H - i);
  }
  if (a.y) {
    float ss = 0.f, b = 1.f;
    if (a.post) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += x[c][j] * x[c][j];
      b = inverse_rms<NT>(x, ss, rh, a.eps, s, 0);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * NT + t) * 8;
      Oct<TY> w, g;
      if (a.w_post) w.load(a.w_post, i, a.H - i);
      if (a.gate) g.load(a.gate, row * a.ld_gate + i, a.H - i);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float p = x[c][j] * b;
        if (a.w_post) p *= w[j];
        if (a.gate) p *= g[j];
        v[j] = a.alpha * r[c][j] + p;
      }
      r[c].pack(v);
      r[c].store(a.res_out, at + i, a.H - i);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * NT + t) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += i + j < a.H ? r[c][j] * r[c][j] : 0.f;
  }
  const float k = inverse_rms<NT>(r, ss, rh, a.eps, s, 1);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = (c * NT + t) * 8;
    Oct<TY> w, o;
    if (a.w_pre) w.load(a.w_pre, i, a.H - i);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = r[c][j] * k;
      if (a.w_pre) v[j] *= w[j];
    }
    o.pack(v);
    o.store(a.n, at + i, a.H - i);
  }
}

// Element `at` (uniform) of a matrix: a scalar address, beside which a thread's
// columns are a 32-bit offset.
template <int T, class P>
__device__ __forceinline__ P *row_at(P *base, int64_t at) {
  using Bytes = std::conditional_t<std::is_const_v<P>, const uint8_t, uint8_t>;
  return (P *)((Bytes *)base + at * Val<T>::size);
}

// Eight columns of the gradients' row operands and of the weights, as stored.
template <int TY, int TR>
struct GradPiece {
  Oct<TR> r, dr;
  Oct<TY> x, dn, wq, wp, gt;

  __device__ __forceinline__ void load_weights(const NormArgs &a, int i) {
    if (a.w_pre) wq.load(a.w_pre, i, a.H - i);
    else wq.fill(1.f);
    if (a.w_post) wp.load(a.w_post, i, a.H - i);
    else wp.fill(1.f);
    if (a.gate && !a.ld_gate) gt.load(a.gate, i, a.H - i);
    else gt.fill(1.f);
  }
  __device__ __forceinline__ void load_row(const NormArgs &a, int64_t at, int i) {
    r.load(row_at<TR>(a.res, at), i, a.H - i);
    dn.load(row_at<TY>(a.d_n, at), i, a.H - i);
    if (a.d_res) dr.load(row_at<TR>(a.d_res, at), i, a.H - i);
    else dr.fill(0.f);
    if (a.y) x.load(row_at<TY>(a.y, at), i, a.H - i);
    else x.fill(0.f);
    if (a.gate && a.ld_gate) gt.load(row_at<TY>(a.gate, at), i, a.H - i);
  }
  // opaque to the compiler, the row after its sums and the weights in every
  // row: it would keep their fp32 values in registers otherwise
  __device__ __forceinline__ void opaque_row() {
    r.opaque();
    dr.opaque();
    x.opaque();
    dn.opaque();
  }
  __device__ __forceinline__ void opaque_weights() {
    wq.opaque();
    wp.opaque();
    gt.opaque();
  }
};

// g - u m, of the g that the row's sums took: rounded before the difference.
__device__ __forceinline__ float off_mean(float d_n, float w, float u, float m) {
#pragma clang fp contract(off)
  const float g = d_n * w;
  return __builtin_fmaf(-u, m, g);
}

// Column sums of a run of rows: d_w_pre, d_w_post, d_gate.  They leave once,
// as one row of a.part per unit, for the summing kernel below (no atomics:
// the order is fixed).
struct ColumnSums {
  float v[3][8];
  __device__ __forceinline__ ColumnSums() {
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[q][j] = 0.f;
  }
  __device__ __forceinline__ void store(const NormArgs &a, int64_t unit, int i) const {
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      float *p = a.part + (unit * 3 + q) * a.H + i;
#pragma unroll
      for (int j = 0; j < 8; ++j) if (i + j < a.H) p[j] = v[q][j];
    }
  }
};

// Powers of two (row_unit) for r' and y, from the largest magnitudes that the
// threads met.  Uses buffers 2 and 3 of s.
struct RowUnits {
  float r = 1.f, y = 1.f;
};
template <int NT>
__device__ __forceinline__ RowUnits row_units(float top_r, float top_y, float eps, float *s) {
  top_r = row_top<NT>(top_r, s, 2);
  top_y = row_top<NT>(top_y, s, 3);
  return RowUnits{row_unit(top_r, eps), row_unit(top_y, eps)};
}

// Gradients of rows of up to 8 NT columns, one piece of eight a thread.  A
// workgroup takes a contiguous run of rows and keeps its column sums in
// registers: with a row in flight they fit the 128 registers of 16 waves per
// CU, where addresses and row sums are scalar (with vector ones 6 to 120 of
// them went through scratch: 4096 rows of 8192 in fp32 275 us, now 183).  Two
// pieces of 256 threads took 138 us for the rows above.
template <int TY, int TR, int NT>
__global__ void __launch_bounds__(norm_block(NT), 4) block_norm_grad_kernel(NormArgs a) {
  constexpr int RW = norm_block(NT) / NT;   // rows at a time
  __shared__ float s[4 * 3 * 16];
  const int i = threadIdx.x % NT * 8;
  const int64_t unit = (int64_t)blockIdx.x * RW + __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  const int64_t units = (int64_t)gridDim.x * RW, lo = unit * a.T / units, hi = (unit + 1) * a.T / units;
  const float rh = 1.f / (float)a.H;
  ColumnSums sums;
  GradPiece<TY, TR> p;
  p.load_weights(a, i);
  const bool tok = a.gate && a.ld_gate;     // a gate row per token
  for (int64_t row = lo; row < hi; ++row) {
    const int64_t at = row * a.H;
    p.load_row(a, at, i);
    p.opaque_weights();
    float q3[3] = {0.f, 0.f, 0.f};         // sums of r^2, g r, y^2
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float g = p.dn[j] * p.wq[j];
      q3[0] += p.r[j] * p.r[j];
      q3[1] += g * p.r[j];
      q3[2] += p.x[j] * p.x[j];
    }
    row_sum<NT, 3>(q3, s, 0);
    const float qr = q3[0] * rh + a.eps, qy = q3[2] * rh + a.eps;
    float k, m, b;                          // 1 / rms(r'), mean(g u), 1 / rms(y)
    if (__builtin_expect(plain_square(qr) && (!a.post || plain_square(qy)) && __builtin_fabsf(q3[1]) < __builtin_inff(), 1)) {
      k = 1.f / __builtin_sqrtf(qr);
      m = q3[1] * k * rh;
      b = a.post ? 1.f / __builtin_sqrtf(qy) : 1.f;
    } else {                                // as inverse_rms
      float top_r = 0.f, top_y = 0.f;
      p.opaque_row();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        top_r = __builtin_fmaxf(top_r, __builtin_fabsf(p.r[j]));
        top_y = __builtin_fmaxf(top_y, __builtin_fabsf(p.x[j]));
      }
      const RowUnits u = row_units<NT>(top_r, top_y, a.eps, s);
      q3[0] = q3[1] = q3[2] = 0.f;
      p.opaque_row();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float r = p.r[j] * u.r, y = p.x[j] * u.y;
        q3[0] += r * r;
        q3[1] += p.dn[j] * p.wq[j] * r;
        q3[2] += y * y;
      }
      row_sum<NT, 3>(q3, s, 0);             // (the barriers above lie behind its first use)
      const float h = 1.f / __builtin_sqrtf(q3[0] * rh + a.eps * u.r * u.r);
      k = u.r * h;
      m = q3[1] * h * rh;
      b = a.post ? u.y / __builtin_sqrtf(q3[2] * rh + a.eps * u.y * u.y) : 1.f;
    }
    p.opaque_row();
    const float al = a.y ? a.alpha : 1.f;
    float d[8], z[1] = {0.f};               // c, sum of c v
    float ov[8], dv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = p.r[j] * k;
      const float e = k * off_mean(p.dn[j], p.wq[j], u, m) + p.dr[j];
      sums.v[0][j] += p.dn[j] * u;
      ov[j] = al * e;
      const float v = p.x[j] * b, eg = e * p.gt[j];
      sums.v[1][j] += eg * v;
      dv[j] = e * v * p.wp[j];
      sums.v[2][j] += dv[j];
      d[j] = eg * p.wp[j];
      z[0] += d[j] * v;
    }
    Oct<TR> out;
    out.pack(ov);
    out.store(row_at<TR>(a.d_r, at), i, a.H - i);
    Oct<TY> o;
    if (tok) {
      o.pack(dv);
      o.store(row_at<TY>(a.d_gate, at), i, a.H - i);
    }
    // (also a barrier between this row's sums in s and the next one's)
    row_sum<NT, 1>(z, s, 1);
    if (a.y) {
      const float mz = a.post ? z[0] * rh : 0.f;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xb = a.post ? p.x[j] * b : 0.f;     // (without post norm y may be anything)
        v[j] = b * (d[j] - xb * mz);
      }
      o.pack(v);
      o.store(row_at<TY>(a.d_y, at), i, a.H - i);
    }
  }
  if (a.cols) sums.store(a, unit, i);
}

// Gradients of wide rows.  A row in flight with its column sums does not fit
// the registers of 1024 threads from two pieces on (held in scratch: 339 us
// where this takes 161, 2048 rows of 16384 in bf16, and 1116 against 373,
// 1024 rows of 32768 in fp32): one workgroup per row forms what its gradients
// need of the whole row, then workgroups of 2048 columns and a run of rows
// apply it, a piece of every row a thread.  The rows are read twice.  Without
// column sums the row's own workgroup applies it.
struct RowStats {
  float k, m, b, mz;   // 1 / rms(r'), mean(g u), 1 / rms(y) (1 without post norm), mean(c v) (0)
};

// The row's gradients at the columns of p, and (SUMS) their part of the column
// sums.
template <bool SUMS, int TY, int TR>
__device__ __forceinline__ void apply_stats(const NormArgs &a, const GradPiece<TY, TR> &p, int64_t at, int i, RowStats st,
                                            ColumnSums &sums) {
  const float al = a.y ? a.alpha : 1.f;
  float ov[8], gv[8], yv[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float u = p.r[j] * st.k, v = p.x[j] * st.b;
    const float e = st.k * off_mean(p.dn[j], p.wq[j], u, st.m) + p.dr[j], eg = e * p.gt[j];
    ov[j] = al * e;
    gv[j] = e * v * p.wp[j];
    yv[j] = st.b * (eg * p.wp[j] - (a.post ? v : 0.f) * st.mz);   // (without post norm y may be anything)
    if constexpr (SUMS) {
      sums.v[0][j] += p.dn[j] * u;
      sums.v[1][j] += eg * v;
      sums.v[2][j] += gv[j];
    }
  }
  Oct<TR> o;
  o.pack(ov);
  o.store(row_at<TR>(a.d_r, at), i, a.H - i);
  Oct<TY> q;
  if (a.gate && a.ld_gate) {
    q.pack(gv);
    q.store(row_at<TY>(a.d_gate, at), i, a.H - i);
  }
  if (a.y) {
    q.pack(yv);
    q.store(row_at<TY>(a.d_y, at), i, a.H - i);
  }
}

// Sums of r^2, g r, y^2 and, with f = gate w_post y, of f dr, f g and f r:
// c v = f b (dr + k g - k^2 m r) sums to mean(c v) without another pass.
template <int TY, int TR>
__global__ void __launch_bounds__(1024) norm_stats_kernel(NormArgs a) {
  __shared__ float s[4 * 3 * 16];
  const int64_t row = blockIdx.x, at = row * a.H;
  const float rh = 1.f / (float)a.H;
  float q[6];
  const auto sums = [&](RowUnits u) {          // of the row with r' times u.r and y times u.y
#pragma unroll
    for (int n = 0; n < 6; ++n) q[n] = 0.f;
#pragma unroll 1
    for (int i = threadIdx.x * 8; i < a.H; i += 8192) {
      GradPiece<TY, TR> p;
      p.load_weights(a, i);
      p.load_row(a, at, i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float r = p.r[j] * u.r, x = p.x[j] * u.y, g = p.dn[j] * p.wq[j], f = p.gt[j] * p.wp[j] * x;
        q[0] += r * r;
        q[1] += g * r;
        q[2] += x * x;
        q[3] += f * p.dr[j];
        q[4] += f * g;
        q[5] += f * r;
      }
    }
    row_sum<1024, 6>(q, s, 0);
  };
  RowUnits u;
  sums(RowUnits{1.f, 1.f});
  float qr = q[0] * rh + a.eps, qy = q[2] * rh + a.eps, sum = __builtin_fabsf(q[1]);
  if (a.post) sum += __builtin_fabsf(q[3]) + __builtin_fabsf(q[4]) + __builtin_fabsf(q[5]);
  if (__builtin_expect(!(plain_square(qr) && (!a.post || plain_square(qy)) && sum < __builtin_inff()), 0)) {
    float top_r = 0.f, top_y = 0.f;            // as inverse_rms
#pragma unroll 1
    for (int i = threadIdx.x * 8; i < a.H; i += 8192) {
      GradPiece<TY, TR> p;
      p.load_row(a, at, i);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        top_r = __builtin_fmaxf(top_r, __builtin_fabsf(p.r[j]));
        top_y = __builtin_fmaxf(top_y, __builtin_fabsf(p.x[j]));
      }
    }
    u = row_units<1024>(top_r, top_y, a.eps, s);
    sums(u);
    qr = q[0] * rh + a.eps * u.r * u.r;
    qy = q[2] * rh + a.eps * u.y * u.y;
  }
  const float hr = 1.f / __builtin_sqrtf(qr), hy = 1.f / __builtin_sqrtf(qy);   // 1 / rms of r' u.r and of y u.y
  RowStats st;
  st.k = u.r * hr;
  st.m = q[1] * hr * rh;
  st.b = a.post ? u.y * hy : 1.f;
  st.mz = a.post ? hy * rh * (q[3] + st.k * q[4] - (st.k * st.m) * (hr * q[5])) : 0.f;
  if (a.stats) {
    if (threadIdx.x == 0) a.stats[row] = st;
    return;
  }
  ColumnSums none;
#pragma unroll 1
  for (int i = threadIdx.x * 8; i < a.H; i += 8192) {
    GradPiece<TY, TR> p;
    p.load_weights(a, i);
    p.load_row(a, at, i);
    apply_stats<false>(a, p, at, i, st, none);
  }
}

template <int TY, int TR>
__global__ void __launch_bounds__(256, 4) norm_apply_kernel(NormArgs a) {
  const int i = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 8;
  if (i >= a.H) return;
  const int64_t unit = blockIdx.y, units = gridDim.y;
  const int64_t lo = unit * a.T / units, hi = (unit + 1) * a.T / units;
  GradPiece<TY, TR> p;
  p.load_weights(a, i);
  ColumnSums sums;
  for (int64_t row = lo; row < hi; ++row) {
    p.load_row(a, row * a.H, i);
    p.opaque_weights();
    apply_stats<true>(a, p, row * a.H, i, a.stats[row], sums);
  }
  sums.store(a, unit, i);
}

// Column sums of the units' partial sums: 32 columns per workgroup, 32
// threads a column, joined in a fixed order.
__global__ void __launch_bounds__(1024) norm_columns_kernel(const float *__restrict__ part, int32_t units, int32_t H,
                                                            float *d_w_pre, float *d_w_post, float *d_gate) {
  __shared__ float s[32][33];
  const int q = blockIdx.y, x = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  float *out = q == 0 ? d_w_pre : q == 1 ? d_w_post : d_gate;
  if (!out) return;
  float v = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int u = w; u < units; u += 32) v += part[((int64_t)u * 3 + q) * H + c];
  }
  s[w][x] = v;
  __syncthreads();
  if (w == 0 && c < H) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][x];
    out[c] = v;
  }
}

constexpr int kNormMaxH = 32768;
constexpr int kNormMaxT = (1 << 22) - 1;   // workgroups of 1024 threads: a launch has fewer than 2^32

// Threads per row of the gradient kernel for rows of H up to kGradMaxH: one
// piece of eight a thread as far as 1024 threads go, so that the column sums
// and a row in flight stay within 128 registers and a CU holds 16 waves.
constexpr int kGradMaxH = 8192;
static int grad_threads(int H) { return H <= 512 ? 64 : H <= 1024 ? 128 : H <= 2048 ? 256 : H <= 4096 ? 512 : 1024; }

// Units (rows in flight, or runs of rows of one workgroup) of the gradient
// kernels: 1024 threads per CU, each unit leaving one row of partial column
// sums.
static int grad_units(int T, int H) {
  if (H > kGradMaxH) return std::min(T, 1024 / ((H + 2047) / 2048));
  const int nt = grad_threads(H), rw = nt == 64 ? 4 : 1;
  const int groups = std::min((T + rw - 1) / rw, 256 * 1024 / (nt * rw));
  return groups * rw;
}

// Workspace of the column sums: the rows' statistics, the units' sums.
static size_t grad_stats_bytes(int T, int H) { return H > kGradMaxH ? (size_t)T * sizeof(RowStats) : 0; }
static size_t grad_workspace(int T, int H) { return grad_stats_bytes(T, H) + (size_t)grad_units(T, H) * 3 * (size_t)H * 4; }

template <int TY, int TR, int NT, int CH>
static void launch_norm(const NormArgs &a, hipStream_t s) {
  constexpr int RW = norm_block(NT) / NT;
  hipLaunchKernelGGL((block_norm_kernel<TY, TR, NT, CH>), dim3((a.T + RW - 1) / RW), dim3(norm_block(NT)), 0, s, a);
}

template <int TY, int TR, int NT>
static void launch_grad(const NormArgs &a, hipStream_t s) {
  constexpr int RW = norm_block(NT) / NT;
  hipLaunchKernelGGL((block_norm_grad_kernel<TY, TR, NT>), dim3(grad_units(a.T, a.H) / RW), dim3(norm_block(NT)), 0, s, a);
}

template <int TY, int TR>
static void launch_grad_wide(const NormArgs &a, hipStream_t s) {
  hipLaunchKernelGGL((norm_stats_kernel<TY, TR>), dim3(a.T), dim3(1024), 0, s, a);
  if (a.stats)
    hipLaunchKernelGGL((norm_apply_kernel<TY, TR>), dim3((a.H + 2047) / 2048, grad_units(a.T, a.H)), dim3(256), 0, s, a);
}

template <int TY, int TR>
static void launch_norm_h(const NormArgs &a, bool grad, hipStream_t s) {
  if (grad) {
    if (a.H <= 512) launch_grad<TY, TR, 64>(a, s);
    else if (a.H <= 1024) launch_grad<TY, TR, 128>(a, s);
    else if (a.H <= 2048) launch_grad<TY, TR, 256>(a, s);
    else if (a.H <= 4096) launch_grad<TY, TR, 512>(a, s);
    else if (a.H <= kGradMaxH) launch_grad<TY, TR, 1024>(a, s);
    else launch_grad_wide<TY, TR>(a, s);
    return;
  }
  if (a.H <= 512) launch_norm<TY, TR, 64, 1>(a, s);
  else if (a.H <= 1024) launch_norm<TY, TR, 64, 2>(a, s);
  else if (a.H <= 2048) launch_norm<TY, TR, 256, 1>(a, s);
  else if (a.H <= 4096 && a.T <= 256) launch_norm<TY, TR, 512, 1>(a, s);   // (few rows: for latency)
  else if (a.H <= 4096) launch_norm<TY, TR, 256, 2>(a, s);
  else if (a.H <= 8192 && a.T <= 256) launch_norm<TY, TR, 1024, 1>(a, s);
  else if (a.H <= 8192) launch_norm<TY, TR, 512, 2>(a, s);
  else if (a.H <= 16384) launch_norm<TY, TR, 1024, 2>(a, s);
  else launch_norm<TY, TR, 1024, 4>(a, s);
}

static void launch_norm_types(const NormArgs &a, int ty, int tr, bool grad, hipStream_t s) {
  if (ty == MOEQ_F16 && tr == MOEQ_F16) launch_norm_h<MOEQ_F16, MOEQ_F16>(a, grad, s);
  else if (ty == MOEQ_F16) launch_norm_h<MOEQ_F16, MOEQ_F32>(a, grad, s);
  else if (ty == MOEQ_BF16 && tr == MOEQ_BF16) launch_norm_h<MOEQ_BF16, MOEQ_BF16>(a, grad, s);
  else if (ty == MOEQ_BF16) launch_norm_h<MOEQ_BF16, MOEQ_F32>(a, grad, s);
  else launch_norm_h<MOEQ_F32, MOEQ_F32>(a, grad, s);
}

static moeq_status check_norm(const char *who, const moeq_norm *d, const void *y) {
  if (!d) return fail(MOEQ_ERR_INVALID, "%s: null description", who);
  if (d->T < 0 || d->H < 1) return fail(MOEQ_ERR_INVALID, "%s: T=%d, H=%d", who, d->T, d->H);
  if (d->H > kNormMaxH) return fail(MOEQ_ERR_UNSUPPORTED, "%s: H=%d above %d", who, d->H, kNormMaxH);
  if (d->T > kNormMaxT) return fail(MOEQ_ERR_UNSUPPORTED, "%s: T=%d above %d", who, d->T, kNormMaxT);
  if (d->dtype != MOEQ_F16 && d->dtype != MOEQ_BF16 && d->dtype != MOEQ_F32)
    return fail(MOEQ_ERR_INVALID, "%s: bad dtype %d", who, d->dtype);
  if (d->res_dtype != d->dtype && d->res_dtype != MOEQ_F32)
    return fail(MOEQ_ERR_INVALID, "%s: bad res_dtype %d", who, d->res_dtype);
  if (d->post_norm != 0 && d->post_norm != 1) return fail(MOEQ_ERR_INVALID, "%s: post_norm=%d", who, d->post_norm);
  if (d->w_post && !d->post_norm) return fail(MOEQ_ERR_INVALID, "%s: w_post without post_norm", who);
  if (d->gate_per_token != 0 && d->gate_per_token != 1)
    return fail(MOEQ_ERR_INVALID, "%s: gate_per_token=%d", who, d->gate_per_token);
  if (d->T && !y && (d->w_post || d->gate)) return fail(MOEQ_ERR_INVALID, "%s: w_post or gate without y", who);
  if (!(d->eps > 0.f) || !(d->eps < 1e30f)) return fail(MOEQ_ERR_INVALID, "%s: eps must be positive and finite", who);
  if (!(__builtin_fabsf(d->alpha) < 1e30f)) return fail(MOEQ_ERR_INVALID, "%s: alpha must be finite", who);
  const uintptr_t m = d->dtype == MOEQ_F32 ? 3 : 1;
  if (((uintptr_t)d->w_pre | (uintptr_t)d->w_post | (uintptr_t)d->gate | (uintptr_t)y) & m)
    return fail(MOEQ_ERR_INVALID, "%s: an operand is not aligned to its elements", who);
  return MOEQ_OK;
}

// Row operands that the call needs: present and aligned.
static moeq_status need_rows(const char *who, const char *name, const void *p, int dtype) {
  if (!p) return fail(MOEQ_ERR_INVALID, "%s: null %s", who, name);
  if ((uintptr_t)p & (dtype == MOEQ_F32 ? 3 : 1)) return fail(MOEQ_ERR_INVALID, "%s: %s is not aligned to its elements", who, name);
  return MOEQ_OK;
}

static NormArgs norm_args(const moeq_norm *d, const void *res, const void *y) {
  NormArgs a{};
  a.res = res;
  a.y = y;
  a.w_pre = d->w_pre;
  a.w_post = d->w_post;
  a.gate = d->gate;
  a.ld_gate = d->gate_per_token ? d->H : 0;
  a.T = d->T;
  a.H = d->H;
  a.post = d->post_norm;
  a.alpha = d->alpha;
  a.eps = d->eps;
  return a;
}

}  // namespace moeq

using namespace moeq;

#define MOEQ_TRY(e) do { const moeq_status st_ = (e); if (st_ != MOEQ_OK) return st_; } while (0)

MOEQ_API moeq_status moeq_block_norm(const moeq_norm *d, const void *residual, const void *y, void *res_out, void *n,
                                     hipStream_t stream) {
  const char *who = "block_norm";
  MOEQ_TRY(check_norm(who, d, y));
  if (!d->T) return MOEQ_OK;
  MOEQ_TRY(need_rows(who, "residual", residual, d->res_dtype));
  MOEQ_TRY(need_rows(who, "n", n, d->dtype));
  if (y) MOEQ_TRY(need_rows(who, "res_out", res_out, d->res_dtype));
  NormArgs a = norm_args(d, residual, y);
  a.res_out = res_out;
  a.n = n;
  prof_begin("block_norm", stream);
  launch_norm_types(a, d->dtype, d->res_dtype, false, stream);
  prof_end("block_norm", stream);
  return check_launch("block_norm");
}

MOEQ_API moeq_status moeq_block_norm_grad_workspace_size(int32_t T, int32_t H, size_t *bytes) {
  const char *who = "block_norm_grad_workspace_size";
  if (!bytes) return fail(MOEQ_ERR_INVALID, "%s: null bytes", who);
  if (T < 0 || H < 1) return fail(MOEQ_ERR_INVALID, "%s: T=%d, H=%d", who, T, H);
  if (H > kNormMaxH) return fail(MOEQ_ERR_UNSUPPORTED, "%s: H=%d above %d", who, H, kNormMaxH);
  if (T > kNormMaxT) return fail(MOEQ_ERR_UNSUPPORTED, "%s: T=%d above %d", who, T, kNormMaxT);
  *bytes = grad_workspace(T, H);
  return MOEQ_OK;
}

MOEQ_API moeq_status moeq_block_norm_grad(const moeq_norm *d, const void *res, const void *y, const void *d_res,
                                          const void *d_n, void *d_residual, void *d_y, float *d_w_pre,
                                          float *d_w_post, void *d_gate, void *ws, size_t ws_bytes,
                                          hipStream_t stream) {
  const char *who = "block_norm_grad";
  MOEQ_TRY(check_norm(who, d, y));
  if (d->T) {
    MOEQ_TRY(need_rows(who, "res", res, d->res_dtype));
    MOEQ_TRY(need_rows(who, "d_n", d_n, d->dtype));
    MOEQ_TRY(need_rows(who, "d_residual", d_residual, d->res_dtype));
    if (y) MOEQ_TRY(need_rows(who, "d_y", d_y, d->dtype));
    if (d_res) MOEQ_TRY(need_rows(who, "d_res", d_res, d->res_dtype));
  }
  if (d->gate) {
    if (d->T || !d->gate_per_token) MOEQ_TRY(need_rows(who, "d_gate", d_gate, d->gate_per_token ? d->dtype : MOEQ_F32));
  } else if (d_gate) {
    return fail(MOEQ_ERR_INVALID, "%s: d_gate without gate", who);
  }
  if (d_w_post && (!d->post_norm || (d->T && !y))) return fail(MOEQ_ERR_INVALID, "%s: d_w_post without post norm", who);
  if (((uintptr_t)d_w_pre | (uintptr_t)d_w_post) & 3) return fail(MOEQ_ERR_INVALID, "%s: misaligned weight gradient", who);
  float *g_cols = d->gate && !d->gate_per_token ? (float *)d_gate : nullptr;
  const bool cols = d_w_pre || d_w_post || g_cols;
  const int units = grad_units(d->T, d->H);
  const size_t need = grad_workspace(d->T, d->H);
  float *part = (float *)((char *)ws + grad_stats_bytes(d->T, d->H));
  if (cols && need) {
    if (!ws || ((uintptr_t)ws & 15)) return fail(MOEQ_ERR_INVALID, "%s: null or misaligned workspace", who);
    if (ws_bytes < need) return fail(MOEQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, ws_bytes, need);
  }
  if (d->T) {
    NormArgs a = norm_args(d, res, y);
    a.d_res = d_res;
    a.d_n = d_n;
    a.d_r = d_residual;
    a.d_y = d_y;
    a.d_gate = d_gate;
    a.stats = cols && d->H > kGradMaxH ? (RowStats *)ws : nullptr;
    a.part = part;
    a.cols = cols;
    prof_begin("block_norm_grad", stream);
    launch_norm_types(a, d->dtype, d->res_dtype, true, stream);
    prof_end("block_norm_grad", stream);
    MOEQ_TRY(check_launch("block_norm_grad"));
  }
  if (cols) {
    prof_begin("norm_columns", stream);
    hipLaunchKernelGGL(norm_columns_kernel, dim3((d->H + 31) / 32, 3), dim3(1024), 0, stream, part, units,
                       d->H, d_w_pre, d_w_post, g_cols);
    prof_end("norm_columns", stream);
    MOEQ_TRY(check_launch("norm_columns"));
  }
  return MOEQ_OK;
}
