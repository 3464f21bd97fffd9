// Routing by softmax or sigmoid scores with a bias, groups and renormalised
// gates (the counting sort is that of route.hip), and its gradient.  One wave
// per token; lane l holds experts l + 64 s.
#include "check.hpp"
#include "route.hpp"
#include "vec8.hpp"

namespace moeq {

constexpr int kMaxGroups = 64;   // one lane each
constexpr int kScoreThreads = 256;

struct ScoreArgs {
  const void *logits;
  int64_t ld;
  const float *bias;   // [E] or null
  int T, E, k;
  int groups, top_groups, size;   // size: experts per group
  int sigmoid, top2, renorm;
  float scale;
};

// An expert, or a group, and what it is chosen by.
struct Cand64 {
  double v;
  int id;
};

__device__ __forceinline__ Cand64 better(Cand64 a, Cand64 b) {
  return (a.v > b.v || (a.v == b.v && a.id < b.id)) ? a : b;
}

__device__ __forceinline__ Cand64 wave_best(Cand64 c) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const Cand64 o{__shfl_xor(c.v, m, kWave), __shfl_xor(c.id, m, kWave)};
    c = better(c, o);
  }
  return c;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, m, kWave));
  return v;
}

// Logits of token t, expert lane + 64 s in v[s]; NaN and what lies beyond E
// as -infinity.
template <int TY>
__device__ __forceinline__ void load_row(const void *base, int64_t ld, int t, int E, float *v) {
  const int lane = threadIdx.x & 63;
  const uint8_t *row = (const uint8_t *)base + t * ld * Val<TY>::size;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int e = lane + s * kWave;
    float l = -__builtin_inff();
    if (e < E) {
      if constexpr (TY == MOEQ_F32) l = Val<TY>::get(gld<uint32_t>(row + 4 * e));
      else l = Val<TY>::get(gld<uint16_t>(row + 2 * e));
    }
    v[s] = l == l ? l : -__builtin_inff();
  }
}

// exp(l - m) for l <= m: 1 for l = m (both may be +infinity), 0 for l = -infinity.
__device__ __forceinline__ double exp_below(float l, float m) {
  return l == -__builtin_inff() ? 0.0 : l == m ? 1.0 : exp((double)l - (double)m);
}

__device__ __forceinline__ double sigmoid64(float l) {
  const double u = exp(-__builtin_fabs((double)l));
  return (l >= 0.f ? 1.0 : u) / (1.0 + u);
}

// Routing of token t by one wave: ids and gates of its k experts (and their
// counts and copies in LDS, where given).
__device__ __forceinline__ void score_token(const ScoreArgs &a, const float *l, int t, int32_t *__restrict__ ids,
                                            float *__restrict__ gates, int *s_hist, int *s_ids) {
  const int lane = threadIdx.x & 63;
  const double none = -__builtin_inf();
  const int E = a.E, k = a.k;
  double score[kSlots], c[kSlots];
  float m = l[0];
#pragma unroll
  for (int s = 1; s < kSlots; ++s) m = __builtin_fmaxf(m, l[s]);
  m = wave_max(m);
  double sum = 0.0;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    score[s] = a.sigmoid ? sigmoid64(l[s]) : exp_below(l[s], m);
    sum += score[s];
  }
  if (!a.sigmoid) {
    sum = wave_sum(sum);
#pragma unroll
    for (int s = 0; s < kSlots; ++s) score[s] = sum > 0.0 ? score[s] / sum : 0.0;
  }
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int e = lane + s * kWave;
    c[s] = a.bias && e < E ? score[s] + (double)a.bias[e] : (double)l[s];
    if (!(c[s] == c[s]) || l[s] == -__builtin_inff()) c[s] = none;
  }
  uint64_t kept = ~0ull;
  if (a.groups > 1) {
    double worth = none;
    for (int g = 0; g < a.groups; ++g) {
      double w = 0.0;
      int first = -1;
      for (int round = 0; round <= a.top2; ++round) {
        Cand64 b{none, 0x7fffffff};
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
          const int e = lane + s * kWave;
          if (e / a.size == g && e != first && e < E) {
            const double v = a.top2 && !a.bias && c[s] != none ? score[s] : c[s];
            b = better(b, Cand64{v, e});
          }
        }
        b = wave_best(b);
        w += b.v;
        first = b.id;
      }
      if (lane == g) worth = w == w ? w : none;
    }
    kept = 0;
    for (int i = 0; i < a.top_groups; ++i) {
      Cand64 b{none, 0x7fffffff};
      if (lane < a.groups && !((kept >> lane) & 1)) b = Cand64{worth, lane};
      kept |= 1ull << wave_best(b).id;
    }
  }
  uint32_t taken = 0;
  float sel[kSlots];   // logit of slot j kept by lane j % 64
  int sid[kSlots];     // its expert id
  float top = -__builtin_inff();
#pragma unroll
  for (int s = 0; s < kSlots; ++s) { sel[s] = -__builtin_inff(); sid[s] = 0; }
  for (int j = 0; j < k; ++j) {
    Cand64 b{none, 0x7fffffff};
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const int e = lane + s * kWave;
      if (e < E && !((taken >> s) & 1u) && (a.groups == 1 || ((kept >> (e / a.size)) & 1))) b = better(b, Cand64{c[s], e});
    }
    const int id = wave_best(b).id;
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if ((id >> 6) == s) v = __shfl(l[s], id & 63, kWave);
    if ((id & 63) == lane) taken |= 1u << (id >> 6);
    top = __builtin_fmaxf(top, v);
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (j == lane + s * kWave) { sel[s] = v; sid[s] = id; }
  }
  // gates from the chosen logits; a renormalised softmax needs no others
  double g[kSlots], total = 0.0;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    g[s] = 0.0;
    if (lane + s * kWave < k) {
      if (a.sigmoid) g[s] = sigmoid64(sel[s]);
      else if (a.renorm) g[s] = exp_below(sel[s], top);
      else g[s] = sum > 0.0 ? exp_below(sel[s], m) / sum : 0.0;
    }
    total += g[s];
  }
  if (a.renorm) total = wave_sum(total);
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = lane + s * kWave;
    if (j < k) {
      const double v = !a.renorm ? g[s] : total > 0.0 ? g[s] / total : 0.0;
      ids[(int64_t)t * k + j] = sid[s];
      gates[(int64_t)t * k + j] = (float)((double)a.scale * v);
      if (s_hist) atomicAdd(&s_hist[sid[s]], 1);
      if (s_ids) s_ids[t * k + j] = sid[s];
    }
  }
}

template <int TY>
__global__ void __launch_bounds__(kScoreThreads)
score_kernel(ScoreArgs a, int32_t *__restrict__ ids, float *__restrict__ gates) {
  const int t = blockIdx.x * (kScoreThreads / kWave) + (threadIdx.x >> 6);
  if (t >= a.T) return;
  float l[kSlots];
  load_row<TY>(a.logits, a.ld, t, a.E, l);
  score_token(a, l, t, ids, gates, nullptr, nullptr);
}

// Up to kRouteTokens tokens: choice and counting sort in one workgroup, a
// wave per token.
template <int TY>
__global__ void __launch_bounds__(kRouteTokens * kWave)
score_route_kernel(ScoreArgs a, RouteOut o) {
  constexpr int NTH = kRouteTokens * kWave;
  __shared__ RouteLds<kRouteTokens> s;
  const int t = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < kMaxE; e += NTH) { s.count[e] = 0; s.run[e] = 0; }
  __syncthreads();
  if (t < a.T) {
    float l[kSlots];
    load_row<TY>(a.logits, a.ld, t, a.E, l);
    score_token(a, l, t, o.ids, o.gates, s.count, s.ids);
  }
  __syncthreads();
  place_block<NTH>(o, a.T, a.E, a.k, s);
}

// Gradient of token t's logits.  The chosen experts' own factors are formed
// in lane j (slot j) in 64 bits, from the logits alone; with renorm the
// softmax's gradient is zero but for the chosen, s_e (v_e - 0).
template <int TY>
__global__ void __launch_bounds__(kScoreThreads)
score_grad_kernel(ScoreArgs a, const int32_t *__restrict__ ids, const float *__restrict__ d_gates, void *out,
                  int64_t ldd) {
  const int t = blockIdx.x * (kScoreThreads / kWave) + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= a.T) return;
  const int E = a.E, k = a.k;
  float l[kSlots];
  load_row<TY>(a.logits, a.ld, t, E, l);
  int id[kSlots];
  float sel[kSlots];
  double dg[kSlots], w[kSlots], rest[kSlots];
  float top = -__builtin_inff();
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = lane + s * kWave;
    id[s] = -1;
    dg[s] = 0.0;
    if (j < k) {
      id[s] = ids[(int64_t)t * k + j];
      dg[s] = d_gates[(int64_t)t * k + j];
    }
    if (id[s] < 0 || id[s] >= E) id[s] = -1;
    sel[s] = -__builtin_inff();
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
      const float v = __shfl(l[q], id[s] & 63, kWave);
      if (id[s] >= 0 && (id[s] >> 6) == q) sel[s] = v;
    }
    top = __builtin_fmaxf(top, sel[s]);
  }
  float m = l[0];
#pragma unroll
  for (int s = 1; s < kSlots; ++s) m = __builtin_fmaxf(m, l[s]);
  m = wave_max(m);
  top = wave_max(top);
  // w: the score, of a softmax up to a factor that cancels or follows; rest: 1 - s of a sigmoid
  double total = 0.0, sum = 0.0;
  float u[kSlots];
  const bool dense = !a.sigmoid && !a.renorm;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    w[s] = rest[s] = 0.0;
    u[s] = 0.f;
    if (id[s] >= 0) {
      if (a.sigmoid) {
        w[s] = sigmoid64(sel[s]);
        rest[s] = sigmoid64(-sel[s]);
      } else {
        w[s] = exp_below(sel[s], a.renorm ? top : m);
      }
      total += w[s];
    }
    if (dense) {
      u[s] = l[s] == -__builtin_inff() ? 0.f : l[s] == m ? 1.f : expf(l[s] - m);
      sum += u[s];
    }
  }
  double mean = 0.0;   // sum_i dg_i s_i
  if (a.renorm) total = wave_sum(total);
  if (dense) sum = wave_sum(sum);
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if (a.renorm) w[s] = total > 0.0 ? w[s] / total : 0.0;
    else if (dense) w[s] = sum > 0.0 ? w[s] / sum : 0.0;
    if (w[s] > 0.0) mean += dg[s] * w[s];
  }
  mean = wave_sum(mean);
  // what slot j adds to its expert: its share of the logit's gradient, or dg
  // itself where the softmax over all experts takes it further
  float add[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    double v = dense ? dg[s] : w[s] > 0.0 ? (dg[s] - (a.renorm ? mean : 0.0)) * w[s] : 0.0;
    if (a.sigmoid) v *= rest[s];
    add[s] = (float)((double)a.scale * v);
  }
  float d[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) d[s] = 0.f;
  for (int j = 0; j < k; ++j) {
    float v = 0.f;
    int e = -1;
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if ((j >> 6) == s) { v = __shfl(add[s], j & 63, kWave); e = __shfl(id[s], j & 63, kWave); }
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (e == lane + s * kWave) d[s] += v;
  }
  uint8_t *row = (uint8_t *)out + t * ldd * Val<TY>::size;
  const float inv = sum > 0.0 ? (float)(1.0 / sum) : 0.f, down = (float)((double)a.scale * mean);
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int e = lane + s * kWave;
    if (e >= E) continue;
    const float v = !dense ? d[s] : u[s] > 0.f ? u[s] * inv * (d[s] - down) : 0.f;
    if constexpr (TY == MOEQ_F32) ((uint32_t *)row)[e] = Val<TY>::put(v);
    else ((uint16_t *)row)[e] = (uint16_t)Val<TY>::put(v);
  }
}

static moeq_status check_scoring(const char *who, const moeq_scoring *d, const void *logits, int64_t ld, int32_t dtype,
                                 int32_t T, int32_t E, int32_t k) {
  if (!d) return fail(MOEQ_ERR_INVALID, "%s: null scoring", who);
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > E)
    return fail(MOEQ_ERR_INVALID, "%s: T=%d E=%d k=%d invalid (need 1 <= k <= E <= 256)", who, T, E, k);
  if (T > kMaxTokens || (int64_t)T * k > kMaxRows)
    return fail(MOEQ_ERR_UNSUPPORTED, "%s: T=%d above %d, or T*k above %d", who, T, kMaxTokens, kMaxRows);
  if (!okout(dtype)) return fail(MOEQ_ERR_INVALID, "%s: bad dtype %d", who, dtype);
  if (d->score != MOEQ_SCORE_SOFTMAX && d->score != MOEQ_SCORE_SIGMOID)
    return fail(MOEQ_ERR_INVALID, "%s: score=%d", who, d->score);
  if (d->renorm != 0 && d->renorm != 1) return fail(MOEQ_ERR_INVALID, "%s: renorm=%d", who, d->renorm);
  if (!(__builtin_fabsf(d->scale) < __builtin_inff())) return fail(MOEQ_ERR_INVALID, "%s: scale must be finite", who);
  if (T) MOEQ_TRY(check_matrix(who, "logits", logits, ld, E, dtype));
  return MOEQ_OK;
}

static ScoreArgs score_args(const moeq_scoring *d, const void *logits, int64_t ld, int T, int E, int k) {
  ScoreArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.bias = d->bias;
  a.T = T;
  a.E = E;
  a.k = k;
  a.groups = d->groups;
  a.top_groups = d->top_groups;
  a.size = d->groups > 0 ? E / d->groups : E;
  a.sigmoid = d->score == MOEQ_SCORE_SIGMOID;
  a.top2 = d->group_score == MOEQ_GROUP_TOP2;
  a.renorm = d->renorm;
  a.scale = d->scale;
  return a;
}

template <int TY>
static void launch_scored(const ScoreArgs &a, const moeq_routing *r, void *ws, hipStream_t stream) {
  if (a.T <= kRouteTokens) {
    const RouteOut o{nullptr, r->topk_ids, r->topk_gates, r->expert_offsets, r->sorted_pairs, r->pair_pos};
    hipLaunchKernelGGL((score_route_kernel<TY>), dim3(1), dim3(kRouteTokens * kWave), 0, stream, a, o);
    return;
  }
  constexpr int per = kScoreThreads / kWave;
  hipLaunchKernelGGL((score_kernel<TY>), dim3((a.T + per - 1) / per), dim3(kScoreThreads), 0, stream, a, r->topk_ids,
                     r->topk_gates);
  launch_place(r->topk_ids, a.T, a.E, a.k, r->expert_offsets, r->sorted_pairs, r->pair_pos, ws, stream);
}

template <int TY>
static void launch_scored_grad(const ScoreArgs &a, const int32_t *ids, const float *dg, void *out, int64_t ldd,
                               hipStream_t stream) {
  constexpr int per = kScoreThreads / kWave;
  hipLaunchKernelGGL((score_grad_kernel<TY>), dim3((a.T + per - 1) / per), dim3(kScoreThreads), 0, stream, a, ids, dg, out,
                     ldd);
}

}  // namespace moeq

using namespace moeq;

MOEQ_API moeq_status moeq_route_scored(const moeq_scoring *d, const void *logits, int64_t ld, int32_t dtype, int32_t T,
                                       int32_t E, int32_t k, const moeq_routing *out, void *ws, size_t ws_bytes,
                                       hipStream_t stream) {
  const char *who = "route_scored";
  MOEQ_TRY(check_scoring(who, d, logits, ld, dtype, T, E, k));
  if (d->groups < 1 || d->groups > kMaxGroups || E % d->groups)
    return fail(MOEQ_ERR_INVALID, "%s: groups=%d (1 to %d, dividing E=%d)", who, d->groups, kMaxGroups, E);
  if (d->top_groups < 1 || d->top_groups > d->groups || d->top_groups * (E / d->groups) < k)
    return fail(MOEQ_ERR_INVALID, "%s: top_groups=%d of %d groups of %d experts for k=%d", who, d->top_groups, d->groups,
                E / d->groups, k);
  if (d->groups > 1 && d->group_score != MOEQ_GROUP_MAX && d->group_score != MOEQ_GROUP_TOP2)
    return fail(MOEQ_ERR_INVALID, "%s: group_score=%d", who, d->group_score);
  if (d->groups > 1 && d->group_score == MOEQ_GROUP_TOP2 && E / d->groups < 2)
    return fail(MOEQ_ERR_INVALID, "%s: groups of one expert have no two largest", who);
  if ((uintptr_t)d->bias & 3) return fail(MOEQ_ERR_INVALID, "%s: misaligned bias", who);
  if (!out) return fail(MOEQ_ERR_INVALID, "%s: null routing output", who);
  if (!out->expert_offsets || (T > 0 && (!out->topk_ids || !out->topk_gates || !out->sorted_pairs || !out->pair_pos)))
    return fail(MOEQ_ERR_INVALID, "%s: null pointer", who);
  const size_t need = route_ws_bytes(T, E);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOEQ_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", who, ws_bytes, need);
  const ScoreArgs a = score_args(d, logits, ld, T, E, k);
  prof_begin("route_scored", stream);
  if (dtype == MOEQ_F16) launch_scored<MOEQ_F16>(a, out, ws, stream);
  else if (dtype == MOEQ_BF16) launch_scored<MOEQ_BF16>(a, out, ws, stream);
  else launch_scored<MOEQ_F32>(a, out, ws, stream);
  prof_end("route_scored", stream);
  return check_launch("route_scored");
}

MOEQ_API moeq_status moeq_route_scored_grad(const moeq_scoring *d, const void *logits, int64_t ld, int32_t dtype,
                                            int32_t T, int32_t E, int32_t k, const int32_t *ids, const float *d_gates,
                                            void *d_logits, int64_t ldd, hipStream_t stream) {
  const char *who = "route_scored_grad";
  MOEQ_TRY(check_scoring(who, d, logits, ld, dtype, T, E, k));
  if (!T) return MOEQ_OK;
  MOEQ_TRY(check_matrix(who, "d_logits", d_logits, ldd, E, dtype));
  if (!ids || !d_gates || (((uintptr_t)ids | (uintptr_t)d_gates) & 3))
    return fail(MOEQ_ERR_INVALID, "%s: null or misaligned ids or d_gates", who);
  const ScoreArgs a = score_args(d, logits, ld, T, E, k);
  prof_begin("route_scored_grad", stream);
  if (dtype == MOEQ_F16) launch_scored_grad<MOEQ_F16>(a, ids, d_gates, d_logits, ldd, stream);
  else if (dtype == MOEQ_BF16) launch_scored_grad<MOEQ_BF16>(a, ids, d_gates, d_logits, ldd, stream);
  else launch_scored_grad<MOEQ_F32>(a, ids, d_gates, d_logits, ldd, stream);
  prof_end("route_scored_grad", stream);
  return check_launch("route_scored_grad");
}
