// Routing by softmax or sigmoid scores with a bias, groups and renormalised
// gates (the counting sort is that of route.hip), and its gradient.
//
// Choices are defined in 64 bits, but few tokens have two experts that 32 bits
// cannot tell apart.  A wave therefore picks its token's experts by choices in
// fp32 and watches the distance of each from the next; where it is within what
// fp32 may be off (0.2 to 1.2 tokens in a hundred), the same code picks again in
// 64 bits.  (Choices without a bias are the logits themselves, and exact.)  That
// needs groups that fill a power of two of lanes, at 1, 2 or 4 experts a lane (up
// to 64, 128, 256 experts): any number of experts in one group, 256 in eight, but
// not 160 in eight, whose tokens are all picked in 64 bits, one group after the
// other.  So are tokens of which a group has infinite choices only to sum up.
//
// Up to 16 tokens one launch does all (16 tokens of 128 experts: 7 us); more are
// picked, scanned and placed.  8192 tokens of 256 experts in eight groups: the
// pick takes 20 us of 31.6 for 8.4 MB of logits, bound by its instructions, about
// 600 a token (k rounds of a maximum over the wave, the groups' ranks); picked in
// 64 bits throughout 58 us, by comparisons of floats with their index 38 us.  64,
// 512 and 4096 such tokens: 10.8, 14.5 and 28.9 us (each segment of the placement
// counts all pairs up to 4096); 8192 tokens of 160 experts in eight groups 69 us.
#include "check.hpp"
#include "route.hpp"
#include "vec8.hpp"
#include "wave.hpp"

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
  int lanes;           // lanes of a group in the fp32 pick (a power of two), 0: groups of another size
  int dtype;
  uint16_t *hist;      // [segments, E, 2] pairs of every half segment and expert, or null
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

__device__ __forceinline__ float logit(const void *row, int dtype, int e) {
  float l;
  if (dtype == MOEQ_F32) l = Val<MOEQ_F32>::get(gld<uint32_t>((const uint8_t *)row + 4 * e));
  else {
    const uint32_t bits = gld<uint16_t>((const uint8_t *)row + 2 * e);
    l = dtype == MOEQ_F16 ? Val<MOEQ_F16>::get(bits) : Val<MOEQ_BF16>::get(bits);
  }
  return l == l ? l : -__builtin_inff();
}

__device__ __forceinline__ const void *logit_row(const ScoreArgs &a, int t) {
  return (const uint8_t *)a.logits + t * a.ld * (a.dtype == MOEQ_F32 ? 4 : 2);
}

// Logits of token t, expert lane + 64 s in v[s]; NaN and what lies beyond E
// as -infinity.
__device__ __forceinline__ void load_row(const ScoreArgs &a, int t, float *v) {
  const int lane = threadIdx.x & 63;
  const void *row = logit_row(a, t);
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int e = lane + s * kWave;
    v[s] = e < a.E ? logit(row, a.dtype, e) : -__builtin_inff();
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

// The k experts of token t by one wave in 64 bits: slot j's id in lane j % 64,
// index j / 64; the largest logit and (softmax) the sum of the exponentials
// below it.
__device__ __forceinline__ void pick_exact(const ScoreArgs &a, int t, int *sid, float &m, float &total) {
  const int lane = threadIdx.x & 63;
  float l[kSlots];
  load_row(a, t, l);
  const double none = -__builtin_inf();
  const int E = a.E, k = a.k;
  double score[kSlots], c[kSlots];
  m = l[0];
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
#pragma unroll
  for (int s = 0; s < kSlots; ++s) sid[s] = 0;
  for (int j = 0; j < k; ++j) {
    Cand64 b{none, 0x7fffffff};
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const int e = lane + s * kWave;
      if (e < E && !((taken >> s) & 1u) && (a.groups == 1 || ((kept >> (e / a.size)) & 1))) b = better(b, Cand64{c[s], e});
    }
    const int id = wave_best(b).id;
    if ((id & 63) == lane) taken |= 1u << (id >> 6);
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (j == lane + s * kWave) sid[s] = id;
  }
  total = (float)sum;
}

// ---- the pick in registers: lane l holds experts NS l + s, so that a group of
// consecutive experts is a run of lanes.  V: float or double.

__device__ __forceinline__ float larger(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return __builtin_fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return __builtin_fmin(a, b); }

// Largest value over the wave, the same in every lane (as all_sum).
template <typename V>
__device__ __forceinline__ V all_max(V v) {
  v = larger(v, dpp<0xb1>(v));
  v = larger(v, dpp<0x4e>(v));
  v = larger(v, dpp<0x141>(v));
  v = larger(v, dpp<0x140>(v));
  v = larger(v, dpp_into<0x142, 0xa>(v, v));
  v = larger(v, dpp_into<0x143, 0xc>(v, v));
  return lane_value(v, 63);
}
// The two largest of two lanes' two largest.
template <typename V>
__device__ __forceinline__ void merge2(V &m1, V &m2, V o1, V o2) {
  m2 = larger(larger(m2, o2), smaller(m1, o1));
  m1 = larger(m1, o1);
}

// What fp32 choices may be off, for a choice of size v, in units of 2^-24: a
// sigmoid 4 (the exponential within 2 of an argument rounded to |l| of itself,
// where s (1 - s) |l| < 0.23; 1 for the sum, 2 for the reciprocal), a softmax
// 14 (2 of the exponential, 9 additions, 2 of the reciprocal, 1 of the product;
// what the arguments' rounding adds to both sides is below s |ln s| each), the
// bias's addition |v|.  Twice that, rounded up to 8 and 32.
__device__ __forceinline__ float choice_error(const ScoreArgs &a, float v) {
  return (a.sigmoid ? 0x1p-21f : 0x1p-19f) * (1.f + __builtin_fabsf(v));
}

template <int NS>
__device__ __forceinline__ void load_run(const ScoreArgs &a, int t, float (&l)[NS]) {
  const int lane = threadIdx.x & 63;
  const void *row = logit_row(a, t);
#pragma unroll
  for (int s = 0; s < NS; ++s) l[s] = lane * NS + s < a.E ? logit(row, a.dtype, lane * NS + s) : -__builtin_inff();
}

// As pick_exact, for k <= 64 (slot j in lane j).
template <int NS>
__device__ __forceinline__ void pick_wide(const ScoreArgs &a, int t, int &sid, float &m, float &total) {
  using V = double;
  float l[NS];
  load_run<NS>(a, t, l);
  const int lane = threadIdx.x & 63;
  const float out = -__builtin_inff();
  const V none = -(V)__builtin_inff();
  const bool by_logit = !a.bias;
  m = l[0];
#pragma unroll
  for (int s = 1; s < NS; ++s) m = __builtin_fmaxf(m, l[s]);
  m = all_max(m);
  V c[NS], score[NS];
  total = 0.f;
  if (!by_logit || (a.groups > 1 && a.top2) || (!a.sigmoid && !a.renorm)) {
    V sum = 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      score[s] = a.sigmoid ? sigmoid64(l[s]) : exp_below(l[s], m);
      sum += score[s];
    }
    if (!a.sigmoid) {
      sum = all_sum(sum);
      total = (float)sum;
#pragma unroll
      for (int s = 0; s < NS; ++s) score[s] = sum > 0.0 ? score[s] / sum : 0.0;
    }
  }
  uint32_t left = 0;   // experts of this lane that can be chosen
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int e = lane * NS + s;
    if (e < a.E) left |= 1u << s;
    c[s] = by_logit || e >= a.E ? (V)l[s] : score[s] + (V)a.bias[e];
    if (!(c[s] == c[s]) || l[s] == out) c[s] = none;
  }
  if (a.groups > 1) {
    V m1 = none, m2 = none;
#pragma unroll
    for (int s = 0; s < NS; ++s) merge2(m1, m2, a.top2 && by_logit && l[s] != out ? score[s] : c[s], none);
    if (a.lanes >= 2) merge2(m1, m2, dpp<0xb1>(m1), dpp<0xb1>(m2));
    if (a.lanes >= 4) merge2(m1, m2, dpp<0x4e>(m1), dpp<0x4e>(m2));
    if (a.lanes >= 8) merge2(m1, m2, dpp<0x141>(m1), dpp<0x141>(m2));
    if (a.lanes >= 16) merge2(m1, m2, dpp<0x140>(m1), dpp<0x140>(m2));
    if (a.lanes >= 32) merge2(m1, m2, __shfl_xor(m1, 16, kWave), __shfl_xor(m2, 16, kWave));
    V worth = a.top2 ? m1 + m2 : m1;
    if (!(worth == worth)) worth = none;
    const int mine = lane / a.lanes;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const V w = lane_value(worth, g * a.lanes);
      rank += w > worth || (w == worth && g < mine);
    }
    if (rank >= a.top_groups) left = 0;
  }
  V best;       // this lane's best choice left, and its index (-1: none left)
  int which;
  const auto look = [&]() {
    best = none;
    which = -1;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if ((left >> s & 1) && (which < 0 || c[s] > best)) { best = c[s]; which = s; }
  };
  look();
  sid = 0;
  for (int j = 0; j < a.k; ++j) {
    const V top = all_max(best);
    const int from = __builtin_ctzll(__ballot(which >= 0 && best == top));
    const int w = __builtin_amdgcn_readlane(which, from);
    if (lane == j) sid = from * NS + w;
    if (lane == from) left &= ~(1u << w);
    look();
  }
}

// ---- the same in fp32.  Choices are compared as integers in their order
// (maxima of integers take one instruction a step, and no NaN is in the way);
// kGone, below -infinity, for what cannot be chosen.
constexpr int kGone = (int)0x80000000;
__device__ __forceinline__ int key_of(float v) {   // (-0 counts as 0)
  const int b = __builtin_bit_cast(int, v + 0.f);
  return b ^ (b >> 31 & 0x7fffffff);
}
__device__ __forceinline__ float of_key(int k) { return __builtin_bit_cast(float, k ^ (k >> 31 & 0x7fffffff)); }
template <int CTRL>
__device__ __forceinline__ int max_dpp(int v) { return std::max(v, dpp_into<CTRL, 0xf>(v, kGone)); }
__device__ __forceinline__ int all_max(int v) {
  v = max_dpp<0xb1>(v);
  v = max_dpp<0x4e>(v);
  v = max_dpp<0x141>(v);
  v = max_dpp<0x140>(v);
  v = std::max(v, dpp_into<0x142, 0xa>(v, kGone));
  v = std::max(v, dpp_into<0x143, 0xc>(v, kGone));
  return __builtin_amdgcn_readlane(v, 63);
}
template <int CTRL>
__device__ __forceinline__ void merge2_dpp(int &m1, int &m2) {
  const int o1 = dpp_into<CTRL, 0xf>(m1, kGone), o2 = dpp_into<CTRL, 0xf>(m2, kGone);
  m2 = std::max(std::max(m2, o2), std::min(m1, o1));
  m1 = std::max(m1, o1);
}

// pick_wide's answer, or false where fp32 does not decide.  Each lane sorts
// its experts once, so that a round only moves the winner's up.
template <int NS>
__device__ __forceinline__ bool pick(const ScoreArgs &a, const float (&l)[NS], int &sid, float &m, float &total) {
  const int lane = threadIdx.x & 63;
  const float out = -__builtin_inff();
  const bool by_logit = !a.bias;
  bool sure = true;
  m = l[0];
#pragma unroll
  for (int s = 1; s < NS; ++s) m = __builtin_fmaxf(m, l[s]);
  if (!a.sigmoid) m = of_key(all_max(key_of(m)));
  float score[NS];
  total = 0.f;
  if (!by_logit || (a.groups > 1 && a.top2) || (!a.sigmoid && !a.renorm)) {
    if (a.sigmoid) {
#pragma unroll
      for (int s = 0; s < NS; ++s) score[s] = __builtin_amdgcn_rcpf(1.f + __expf(-l[s]));
    } else {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        score[s] = l[s] == out ? 0.f : l[s] == m ? 1.f : expf(l[s] - m);
        total += score[s];
      }
      total = all_sum(total);
      const float inv = __builtin_amdgcn_rcpf(total);
#pragma unroll
      for (int s = 0; s < NS; ++s) score[s] *= inv;
    }
  }
  int c[NS], id[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int e = id[s] = lane * NS + s;
    float v = l[s];
    if (!by_logit && e < a.E) {
      v = score[s] + a.bias[e];
      if (!(v == v) || l[s] == out) v = out;
    }
    c[s] = e < a.E ? key_of(v) : kGone;
  }
  if (a.groups > 1) {
    int m1 = kGone, m2 = kGone;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int k = a.top2 && by_logit ? key_of(l[s] == out ? out : score[s]) : c[s];
      m2 = std::max(m2, std::min(m1, k));
      m1 = std::max(m1, k);
    }
    if (a.lanes >= 2) merge2_dpp<0xb1>(m1, m2);
    if (a.lanes >= 4) merge2_dpp<0x4e>(m1, m2);
    if (a.lanes >= 8) merge2_dpp<0x141>(m1, m2);
    if (a.lanes >= 16) merge2_dpp<0x140>(m1, m2);
    if (a.lanes >= 32) {
      const int o1 = __shfl_xor(m1, 16, kWave), o2 = __shfl_xor(m2, 16, kWave);
      m2 = std::max(std::max(m2, o2), std::min(m1, o1));
      m1 = std::max(m1, o1);
    }
    const int mine = lane / a.lanes;
    int rank = 0;
    if (by_logit && !a.top2) {
      for (int g = 0; g < a.groups; ++g) {
        const int w = __builtin_amdgcn_readlane(m1, g * a.lanes);
        rank += w > m1 || (w == m1 && g < mine);
      }
    } else {
      const float worth = of_key(m1) + (a.top2 ? of_key(m2) : 0.f);
      // (a sum of two is off by what both are, on either side: from the largest
      // of any group, since they may cancel; no difference of infinities and
      // NaN is above that)
      const float size = __builtin_fabsf(of_key(m1)) + (a.top2 ? __builtin_fabsf(of_key(m2)) : 0.f);
      const float tol = 4.f * choice_error(a, of_key(all_max(mine < a.groups ? key_of(size) : kGone)));
      for (int g = 0; g < a.groups; ++g) {
        const float w = lane_value(worth, g * a.lanes);
        rank += w > worth;
        sure &= __builtin_fabsf(w - worth) > tol || g == mine;
      }
      sure |= mine >= a.groups;
    }
    if (rank >= a.top_groups) {
#pragma unroll
      for (int s = 0; s < NS; ++s) c[s] = kGone;
    }
  }
  // best first, equal ones by id
  const auto order = [&](int x, int y) {
    const bool turn = c[y] > c[x];
    const int k = turn ? c[y] : c[x], i = turn ? id[y] : id[x];
    c[y] = turn ? c[x] : c[y];
    id[y] = turn ? id[x] : id[y];
    c[x] = k;
    id[x] = i;
  };
#pragma unroll
  for (int n = 0; n < NS - 1; ++n)   // (neighbours only: equal ones keep their order)
#pragma unroll
    for (int s = 0; s < NS - 1 - n; ++s) order(s, s + 1);
  sid = 0;
  int last = 0x7fffffff;   // the smallest key that the last one is not surely above
  for (int j = 0; j < a.k; ++j) {
    const int top = all_max(c[0]);
    if (!by_logit) sure &= top < last;
    const int from = __builtin_ctzll(__ballot(c[0] == top));
    const int w = __builtin_amdgcn_readlane(id[0], from);
    if (lane == j) sid = w;
    const bool won = lane == from;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      c[s] = won ? s + 1 < NS ? c[s + 1 < NS ? s + 1 : s] : kGone : c[s];
      if (s + 1 < NS) id[s] = won ? id[s + 1 < NS ? s + 1 : s] : id[s];
    }
    const float v = of_key(top);
    last = key_of(v - 2.f * choice_error(a, v));
  }
  if (!by_logit) sure &= __ballot(c[0] >= last) == 0;
  return __ballot(!sure) == 0;
}

// Gates of the `items` slots (k of each token from t0 on) whose experts stand
// in sid: a thread each, in 64 bits, so that they are rounded once; but a softmax
// over all E divides by the fp32 sum of the pick, which is off by up to 16 steps
// of 2^-24.  A renormalised softmax needs no logits but the chosen.  (Every thread
// of the workgroup calls it; the tokens' largest logits and sums in m and total.)
template <int NTH>
__device__ __forceinline__ void put_gates(const ScoreArgs &a, int t0, int items, const int *sid, const float *m,
                                          const float *total, float *sel, double *g, int32_t *__restrict__ ids,
                                          float *__restrict__ gates) {
  for (int i = threadIdx.x; i < items; i += NTH) {
    const int t = i / a.k;
    const float l = logit(logit_row(a, t0 + t), a.dtype, sid[i]);
    sel[i] = l;
    if (a.sigmoid) g[i] = sigmoid64(l);
    else if (!a.renorm) g[i] = exp_below(l, m[t]);
  }
  if (a.renorm) __syncthreads();
  if (a.renorm && !a.sigmoid) {
    for (int i = threadIdx.x; i < items; i += NTH) {
      const int t = i / a.k;
      float top = sel[t * a.k];
      for (int j = 1; j < a.k; ++j) top = __builtin_fmaxf(top, sel[t * a.k + j]);
      g[i] = exp_below(sel[i], top);
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < items; i += NTH) {
    const int t = i / a.k;
    double div = a.sigmoid ? 1.0 : (double)total[t];
    if (a.renorm) {
      div = 0.0;
      for (int j = 0; j < a.k; ++j) div += g[t * a.k + j];
    }
    ids[i] = sid[i];
    gates[i] = div > 0.0 ? (float)((double)a.scale * (g[i] / div)) : 0.f;
  }
}

constexpr int kPickMost = 64;   // slots of a token that go through LDS

// The experts and gates of tokens t0 .. t0 + NW TW - 1 by a workgroup of NW
// waves, TW tokens each; the pairs also into s_hist and s_ids, where given.
template <int NS, int NW, int TW>
struct PickLds {
  float sel[NW * TW * kPickMost], m[NW * TW], total[NW * TW];
  int sid[NW * TW * kPickMost];
  double g[NW * TW * kPickMost];
};
template <int NS, int NW, int TW>
__device__ __forceinline__ void pick_tokens(const ScoreArgs &a, int t0, int32_t *__restrict__ ids, float *__restrict__ gates,
                                            PickLds<NS, NW, TW> &s, int *s_hist, int *s_ids) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = std::min(NW * TW, a.T - t0);
  float next[NS];
  if (t0 + wave * TW < a.T) load_run<NS>(a, t0 + wave * TW, next);
#pragma unroll 1
  for (int i = 0; i < TW; ++i) {
    const int at = wave * TW + i;
    if (t0 + at >= a.T) break;
    float l[NS], m, total;
    int sid[kSlots];
#pragma unroll
    for (int q = 0; q < NS; ++q) l[q] = next[q];
    if (i + 1 < TW && t0 + at + 1 < a.T) load_run<NS>(a, t0 + at + 1, next);
    if (!a.lanes) pick_exact(a, t0 + at, sid, m, total);
    else if (!pick<NS>(a, l, sid[0], m, total)) pick_wide<NS>(a, t0 + at, sid[0], m, total);
    if (lane < a.k) {
      s.sid[at * a.k + lane] = sid[0];
      if (s_hist) atomicAdd(&s_hist[sid[0]], 1);
      if (s_ids) s_ids[at * a.k + lane] = sid[0];
    }
    if (lane == 0) {
      s.m[at] = m;
      s.total[at] = total;
    }
  }
  __syncthreads();
  const int64_t p = (int64_t)t0 * a.k;
  put_gates<NW * kWave>(a, t0, n * a.k, s.sid, s.m, s.total, s.sel, s.g, ids + p, gates + p);
}

// Many tokens.  With hist, a workgroup's NW TW tokens are half a segment of the
// counting sort, whose pairs it counts (an expert at most once per token) into
// its half of the segment's words.
template <int NS, int NW, int TW>
__global__ void __launch_bounds__(NW *kWave)
score_kernel(ScoreArgs a, int32_t *__restrict__ ids, float *__restrict__ gates) {
  __shared__ PickLds<NS, NW, TW> s;
  __shared__ int s_hist[kMaxE];
  if (a.hist) {
    for (int e = threadIdx.x; e < a.E; e += NW * kWave) s_hist[e] = 0;
    __syncthreads();
  }
  pick_tokens<NS, NW, TW>(a, blockIdx.x * (NW * TW), ids, gates, s, a.hist ? s_hist : nullptr, nullptr);
  if (a.hist)   // (pick_tokens has synchronised after the counts)
    for (int e = threadIdx.x; e < a.E; e += NW * kWave)
      a.hist[((int64_t)(blockIdx.x >> 1) * a.E + e) * 2 + (blockIdx.x & 1)] = (uint16_t)s_hist[e];
}

// Up to kRouteTokens tokens: choice and counting sort in one workgroup, a
// wave per token.
template <int NS>
__global__ void __launch_bounds__(kRouteTokens * kWave)
score_route_kernel(ScoreArgs a, RouteOut o) {
  constexpr int NTH = kRouteTokens * kWave;
  __shared__ RouteLds<kRouteTokens> r;
  __shared__ PickLds<NS, kRouteTokens, 1> s;
  for (int e = threadIdx.x; e < kMaxE; e += NTH) { r.count[e] = 0; r.run[e] = 0; }
  __syncthreads();
  pick_tokens<NS, kRouteTokens, 1>(a, 0, o.ids, o.gates, s, r.count, r.ids);
  place_block<NTH>(o, a.T, a.E, a.k, r);
}

// More than kPickMost slots: a wave per token, all in 64 bits.
__global__ void __launch_bounds__(kScoreThreads)
score_wide_kernel(ScoreArgs a, int32_t *__restrict__ ids, float *__restrict__ gates) {
  const int lane = threadIdx.x & 63, t = blockIdx.x * (kScoreThreads / kWave) + (threadIdx.x >> 6), k = a.k;
  if (t >= a.T) return;
  float sel[kSlots], m, sum;
  int sid[kSlots];
  pick_exact(a, t, sid, m, sum);
  float top = -__builtin_inff();
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    sel[s] = lane + s * kWave < k ? logit(logit_row(a, t), a.dtype, sid[s]) : -__builtin_inff();
    top = __builtin_fmaxf(top, sel[s]);
  }
  top = wave_max(top);
  double g[kSlots], total = 0.0;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    g[s] = 0.0;
    if (lane + s * kWave < k) g[s] = a.sigmoid ? sigmoid64(sel[s]) : exp_below(sel[s], a.renorm ? top : m);
    total += g[s];
  }
  const double div = a.renorm ? wave_sum(total) : a.sigmoid ? 1.0 : (double)sum;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = lane + s * kWave;
    if (j < k) {
      ids[(int64_t)t * k + j] = sid[s];
      gates[(int64_t)t * k + j] = div > 0.0 ? (float)((double)a.scale * (g[s] / div)) : 0.f;
    }
  }
}

// Gradient of the logits of four tokens by a workgroup of four waves.  What a
// chosen expert gets is formed by one thread per (token, slot) in 64 bits and
// put into the token's row in LDS; the rows leave along their length.  Only a
// softmax over all E without renorm reads (and gives a gradient to) the other
// logits.
//
// Where one expert has nearly all the weight, v_e - sum_i v_i s_i is what is
// left of two nearly equal numbers.  What the experts bring is therefore taken
// relative to c, what the one of the largest weight brings (0 if that is not a
// chosen one), so that no term is larger than the differences that count:
//   renorm:  d_j = scale (x_j - sum_i w_i x_i / S) w_j / S,  x_j = dg_j - c, S = sum_i w_i
//   over all E (x_e: sum of dg_j over e's slots, less c; S: sum of all weights, R: of those not chosen):
//            d_l_e = scale (x_e - (sum_i w_i x_i - R c) / S) w_e / S
// with R summed by itself: an entry is off by what its terms are, however small
// it is beside them.  The others' entries are products in fp32.
//
// 16384 tokens of 256 experts, top-8: 10.6 us (sigmoid 11.1) with renorm for 17
// MB out and 8 MB of lines of chosen logits in, 16.5 us over all E (34 MB and an
// exponential per expert).  That is 2.0 to 2.4 TB/s: bound by the latency of
// the phases between four barriers, in which a token's k slots keep few lanes
// busy, not by bytes.
constexpr int kGradTokens = 4;
struct GradLds {
  static constexpr int NT = kGradTokens;
  int id[NT * kPickMost];
  float l[NT * kPickMost], dg[NT * kPickMost], add[NT * kPickMost], m[NT], rest[NT], down[NT], inv[NT];
  double w[NT * kPickMost], wx[NT * kPickMost];
  __attribute__((aligned(16))) float d[NT][kMaxE];
};
static_assert(kGradTokens * kPickMost <= kScoreThreads, "a thread per slot");

__global__ void __launch_bounds__(kScoreThreads)
score_grad_kernel(ScoreArgs a, const int32_t *__restrict__ ids, const float *__restrict__ d_gates, void *out, int64_t ldd) {
  constexpr int NT = kGradTokens, TW = NT / (kScoreThreads / kWave);
  __shared__ GradLds s;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.x * NT, k = a.k, E = a.E;
  const bool dense = !a.sigmoid && !a.renorm, slot = tid < std::min(NT, a.T - t0) * k;
  const int st = tid / k, s0 = st * k;   // this thread's slot: its token, and that token's first
  int id = -1;
  float l = -__builtin_inff(), dg = 0.f;
  if (slot) {
    const int64_t p = (int64_t)t0 * k + tid;
    id = ids[p];
    dg = d_gates[p];
    if ((uint32_t)id < (uint32_t)E) l = logit(logit_row(a, t0 + st), a.dtype, id);
    else id = -1;
    s.id[tid] = id;
    s.dg[tid] = dg;
    s.l[tid] = l;
  }
#pragma unroll
  for (int i = 0; i < NT * kMaxE / 4 / kScoreThreads; ++i) *(f32x4 *)&s.d[0][(i * kScoreThreads + tid) * 4] = f32x4{0.f, 0.f, 0.f, 0.f};
  float u[TW][4];   // dense: exponentials of experts 4 lane .., then -1 for chosen ones
  if (dense) {
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const int t = wave * TW + i;
      if (t0 + t >= a.T) continue;
      load_run<4>(a, t0 + t, u[i]);
      const float m = of_key(all_max(key_of(__builtin_fmaxf(__builtin_fmaxf(u[i][0], u[i][1]), __builtin_fmaxf(u[i][2], u[i][3])))));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v = u[i][q];
        u[i][q] = v == -__builtin_inff() ? 0.f : v == m ? 1.f : expf(v - m);
      }
      if (lane == 0) s.m[t] = m;
    }
  }
  __syncthreads();
  // w: a slot's weight, of a softmax up to a factor; dense: of an expert's
  // first slot, 0 for its others
  bool first = id >= 0;
  double w = 0.0, x = dg, c = 0.0;
  if (slot && (a.renorm || dense)) {
    float top = s.l[s0];
    int at = s0;
    for (int j = s0 + 1; j < s0 + k; ++j)
      if (s.l[j] > top) {
        top = s.l[j];
        at = j;
      }
    if (dense) {
      const int lead = top == s.m[st] ? s.id[at] : -2;
      double mine = 0.0;
      for (int j = s0; j < s0 + k; ++j) {
        const int o = s.id[j];
        const double b = s.dg[j];
        mine += o == id ? b : 0.0;
        c += o == lead ? b : 0.0;
        first &= o != id || j >= tid;
      }
      x = mine - c;
      if (first) w = exp_below(l, s.m[st]);
      if (id >= 0) s.d[st][id] = 1.f;
    } else {
      x = (double)dg - (double)s.dg[at];
      if (id >= 0) w = a.sigmoid ? sigmoid64(l) : exp_below(l, top);
    }
    s.w[tid] = w;
    s.wx[tid] = w > 0.0 ? w * x : 0.0;
  } else if (first) {
    w = sigmoid64(l);
  }
  if (dense) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const int t = wave * TW + i;
      if (t0 + t >= a.T) continue;
      const f32x4 chosen = *(const f32x4 *)&s.d[t][lane * 4];
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (chosen[q] != 0.f) u[i][q] = -1.f;
        else sum += u[i][q];
      }
      sum = all_sum(sum);
      if (lane == 0) s.rest[t] = sum;
    }
  }
  if (a.renorm || dense) __syncthreads();
  if (slot) {
    double d = w > 0.0 ? x * w : 0.0;
    if (a.renorm || dense) {
      const double rest = dense ? (double)s.rest[st] : 0.0;
      double chosen = 0.0, mean = 0.0;
      for (int j = s0; j < s0 + k; ++j) {
        chosen += s.w[j];
        mean += s.wx[j];
      }
      const double total = chosen + rest;
      if (dense && tid == s0) {
        s.down[st] = total > 0.0 ? (float)((double)a.scale * ((mean + c * chosen) / total)) : 0.f;
        s.inv[st] = total > 0.0 ? (float)(1.0 / total) : 0.f;
      }
      d = w > 0.0 ? (x - (mean - rest * c) / total) * (w / total) : 0.0;
    }
    if (a.sigmoid && w > 0.0) d *= sigmoid64(-l);
    const float v = (float)((double)a.scale * d);
    if (!dense) s.add[tid] = v;
    else if (first) s.d[st][id] = v;
  }
  __syncthreads();
  if (!dense) {
    if (id >= 0) {   // an expert's first slot adds up all that are its
      float sum = 0.f;
      for (int j = s0; j < s0 + k; ++j) {
        if (s.id[j] != id) continue;
        sum += s.add[j];
        first &= j >= tid;
      }
      if (first) s.d[st][id] = sum;
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < TW; ++i) {
    const int t = wave * TW + i, n = E - lane * 4;
    if (t0 + t >= a.T || n <= 0) continue;
    f32x4 d = *(const f32x4 *)&s.d[t][lane * 4];
    if (dense) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (u[i][q] >= 0.f) d[q] = u[i][q] > 0.f ? u[i][q] * s.inv[t] * (0.f - s.down[t]) : 0.f;
    }
    const int64_t at = (int64_t)(t0 + t) * ldd + lane * 4;
    if (a.dtype == MOEQ_F32) {
      float *o = (float *)out + at;
      if (n >= 4) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, d), (u32x4_a4 *)o);
      else
        for (int q = 0; q < n; ++q) o[q] = q == 0 ? d[0] : q == 1 ? d[1] : d[2];
    } else {
      uint16_t *o = (uint16_t *)out + at;
      uint32_t b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) b[q] = a.dtype == MOEQ_F16 ? Val<MOEQ_F16>::put(d[q]) : Val<MOEQ_BF16>::put(d[q]);
      typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
      if (n >= 4) __builtin_nontemporal_store(u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16}, (u32x2_a2 *)o);
      else
        for (int q = 0; q < n; ++q) o[q] = (uint16_t)(q == 0 ? b[0] : q == 1 ? b[1] : b[2]);
    }
  }
}

// More than kPickMost slots: a wave per token, expert e in lane e % 64 (4096
// tokens of 256 experts, 100 slots: 9.2 us with renorm, 9.8 us over all E).
template <int TY>
__global__ void __launch_bounds__(kScoreThreads)
score_grad_wide_kernel(ScoreArgs a, const int32_t *__restrict__ ids, const float *__restrict__ d_gates, void *out,
                  int64_t ldd) {
  __shared__ int s_n[kScoreThreads / kWave][kMaxE];
  __shared__ float s_v[kScoreThreads / kWave][kMaxE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * (kScoreThreads / kWave) + wave;
  if (t >= a.T) return;   // (a wave works in its own part of LDS)
  const int E = a.E, k = a.k;
  const bool dense = !a.sigmoid && !a.renorm;
  float l[kSlots];
  load_row(a, t, l);
  int id[kSlots];
  float dg[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int j = lane + s * kWave;
    id[s] = j < k ? ids[(int64_t)t * k + j] : -1;
    dg[s] = j < k ? d_gates[(int64_t)t * k + j] : 0.f;
    if (id[s] >= E) id[s] = -1;
  }
  // an expert's slots, and the sum of what they bring: through LDS, and where
  // one has several, in slot order
  int n[kSlots];
  double v[kSlots];
  bool several = false;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) s_n[wave][lane + s * kWave] = 0;
  lds_order();
#pragma unroll
  for (int s = 0; s < kSlots; ++s)
    if (id[s] >= 0) {
      atomicAdd(&s_n[wave][id[s]], 1);
      s_v[wave][id[s]] = dg[s];
    }
  lds_order();
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    n[s] = s_n[wave][lane + s * kWave];
    v[s] = n[s] ? s_v[wave][lane + s * kWave] : 0.f;
    several |= n[s] > 1;
  }
  if (__ballot(several)) {
#pragma unroll
    for (int s = 0; s < kSlots; ++s) v[s] = 0.0;
#pragma unroll
    for (int b = 0; b < kSlots; ++b)
      for (int j = b * kWave; j < std::min(k, (b + 1) * kWave); ++j) {
        const int e = __builtin_amdgcn_readlane(id[b], j & 63);
        const float g = lane_value(dg[b], j & 63);
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
          if (e == lane + s * kWave) v[s] += g;
      }
  }
  float m = l[0], top = -__builtin_inff();
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    m = __builtin_fmaxf(m, l[s]);
    if (n[s]) top = __builtin_fmaxf(top, l[s]);
  }
  m = wave_max(m);
  top = wave_max(top);
  // c: what a slot of the expert of the largest weight brings (dense: all its
  // slots, 0 if it is not chosen)
  double c = 0.0;
  if (a.renorm || (dense && top == m)) {
    bool found = false;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const uint64_t is = __ballot(n[s] && l[s] == top);
      if (!found && is) {
        const int from = __builtin_ctzll(is);
        c = lane_value(v[s], from) / (dense ? 1 : __builtin_amdgcn_readlane(n[s], from));
        found = true;
      }
    }
  }
  // w: a chosen expert's score, of a softmax up to a factor; u: the others' exponentials
  double w[kSlots], chosen = 0.0, rest = 0.0, mean = 0.0;
  float u[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    w[s] = 0.0;
    u[s] = 0.f;
    if (n[s]) {
      w[s] = a.sigmoid ? sigmoid64(l[s]) : exp_below(l[s], a.renorm ? top : m);
      chosen += dense ? w[s] : n[s] * w[s];
      v[s] -= (dense ? 1 : n[s]) * c;
      if (w[s] > 0.0) mean += v[s] * w[s];
    } else if (dense) {
      u[s] = l[s] == -__builtin_inff() ? 0.f : l[s] == m ? 1.f : expf(l[s] - m);
      rest += u[s];
    }
  }
  rest = wave_sum(rest);
  chosen = wave_sum(chosen);
  mean = wave_sum(mean);
  const double total = chosen + rest;
  uint8_t *row = (uint8_t *)out + t * ldd * Val<TY>::size;
  const float inv = total > 0.0 ? (float)(1.0 / total) : 0.f, down = total > 0.0 ? (float)((double)a.scale * ((mean + c * chosen) / total)) : 0.f;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int e = lane + s * kWave;
    if (e >= E) continue;
    float g = 0.f;
    if (w[s] > 0.0) {
      double x = v[s] * w[s];
      if (a.renorm || dense) x = (v[s] - (dense ? 1 : n[s]) * (mean - rest * c) / total) * (w[s] / total);
      if (a.sigmoid) x *= sigmoid64(-l[s]);
      g = (float)((double)a.scale * x);
    } else if (u[s] > 0.f) {
      g = u[s] * inv * (0.f - down);
    }
    if constexpr (TY == MOEQ_F32) ((uint32_t *)row)[e] = Val<TY>::put(g);
    else ((uint16_t *)row)[e] = (uint16_t)Val<TY>::put(g);
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

static ScoreArgs score_args(const moeq_scoring *d, const void *logits, int64_t ld, int32_t dtype, int T, int E, int k) {
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
  a.dtype = dtype;
  const int per = E <= 64 ? 1 : E <= 128 ? 2 : 4, lanes = a.size / per;   // experts of a lane in the fp32 pick
  a.lanes = a.groups <= 1 ? 64 : a.size % per || (lanes & (lanes - 1)) || lanes > 32 ? 0 : lanes;
  return a;
}

template <int NS>
static void launch_scored(const ScoreArgs &a, const moeq_routing *r, void *ws, hipStream_t stream) {
  if (a.T <= kRouteTokens && a.k <= kPickMost) {
    const RouteOut o{nullptr, r->topk_ids, r->topk_gates, r->expert_offsets, r->sorted_pairs, r->pair_pos};
    hipLaunchKernelGGL((score_route_kernel<NS>), dim3(1), dim3(kRouteTokens * kWave), 0, stream, a, o);
    return;
  }
  bool counted = false;
  if (a.k > kPickMost) {
    constexpr int per = kScoreThreads / kWave;
    if (a.T)
      hipLaunchKernelGGL(score_wide_kernel, dim3((a.T + per - 1) / per), dim3(kScoreThreads), 0, stream, a, r->topk_ids,
                         r->topk_gates);
  } else if (route_ws_bytes(a.T, a.E)) {   // the segments' counts go through the workspace
    ScoreArgs b = a;
    b.hist = (uint16_t *)ws;
    counted = true;
    hipLaunchKernelGGL((score_kernel<NS, 16, kSegTokens / 32>), dim3(2 * route_segments(a.T)), dim3(1024), 0, stream, b,
                       r->topk_ids, r->topk_gates);
  } else {
    hipLaunchKernelGGL((score_kernel<NS, 4, 1>), dim3((a.T + 3) / 4), dim3(256), 0, stream, a, r->topk_ids, r->topk_gates);
  }
  launch_place(r->topk_ids, a.T, a.E, a.k, r->expert_offsets, r->sorted_pairs, r->pair_pos, ws, counted, stream);
}

template <int TY>
static void launch_scored_grad(const ScoreArgs &a, const int32_t *ids, const float *dg, void *out, int64_t ldd,
                               hipStream_t stream) {
  constexpr int per = kScoreThreads / kWave;
  hipLaunchKernelGGL((score_grad_wide_kernel<TY>), dim3((a.T + per - 1) / per), dim3(kScoreThreads), 0, stream, a, ids, dg,
                     out, ldd);
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
  const ScoreArgs a = score_args(d, logits, ld, dtype, T, E, k);
  prof_begin("route_scored", stream);
  if (E <= 64) launch_scored<1>(a, out, ws, stream);
  else if (E <= 128) launch_scored<2>(a, out, ws, stream);
  else launch_scored<4>(a, out, ws, stream);
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
  const ScoreArgs a = score_args(d, logits, ld, dtype, T, E, k);
  prof_begin("route_scored_grad", stream);
  if (k <= kPickMost)
    hipLaunchKernelGGL(score_grad_kernel, dim3((T + kGradTokens - 1) / kGradTokens), dim3(kScoreThreads), 0, stream, a, ids,
                       d_gates, d_logits, ldd);
  else if (dtype == MOEQ_F16) launch_scored_grad<MOEQ_F16>(a, ids, d_gates, d_logits, ldd, stream);
  else if (dtype == MOEQ_BF16) launch_scored_grad<MOEQ_BF16>(a, ids, d_gates, d_logits, ldd, stream);
  else launch_scored_grad<MOEQ_F32>(a, ids, d_gates, d_logits, ldd, stream);
  prof_end("route_scored_grad", stream);
  return check_launch("route_scored_grad");
}
