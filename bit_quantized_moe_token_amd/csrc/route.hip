// Top-k routing and the token -> expert counting sort: in one workgroup for
// up to 16 tokens; else top-k in workgroups of 4 tokens, then placement in
// 64-token segments.  Up to 4096 tokens each segment counts every pair's
// expert itself (no workspace, no grid-wide step); beyond, per-segment
// histograms and one scan over the segments go through a workspace, so the
// work stays linear in the batch.
//
// Top-k with softmax gates over the selected logits (router-guided top-n
// compensation, "Bandwidth-Efficient Adaptive Mixture-of-Experts via
// Low-Rank Compensation", abstract, presupposes a per-token top-k list) and a
// stable counting sort of the (token, slot) pairs by expert with prefix-sum
// offsets (MxMoE abstract: uneven expert activation makes per-expert work
// heterogeneous, so experts get contiguous, variable-length row ranges).
//
// The single-workgroup routing (route_block in route.hpp) runs one wave
// per token; ties in the top-k order go to the lower expert id.
#include "route.hpp"

namespace moeq {

constexpr int kRouteThreads = 1024;

__global__ void __launch_bounds__(kRouteThreads)
route_kernel(RouteOut o, int T, int E, int k) {
  __shared__ RouteLds<kRouteThreads / kWave> s;
  route_block<kRouteThreads>(o, T, E, k, s);
}


// ---- many tokens: two kernels.  Top-k spread over workgroups of
// kTopkWaves tokens (one wave per token, one wave per SIMD), so the
// rounds of many tokens run on many CUs; then placement in segments of
// kSegTokens tokens.
constexpr int kTopkThreads = 256;
constexpr int kTopkWaves = kTopkThreads / kWave;
constexpr int kSegThreads = 256;
constexpr int kSegWaves = kSegThreads / kWave;

__global__ void __launch_bounds__(kTopkThreads)
route_topk_kernel(const float *__restrict__ logits, int T, int E, int k, int32_t *__restrict__ ids,
                  float *__restrict__ gates) {
  const int t = blockIdx.x * kTopkWaves + (threadIdx.x >> 6);
  topk_tokens<1>(logits, t, T, kTopkWaves, E, k, ids, gates, nullptr);
}

// Per-expert totals (s_tot) and counts of the pairs before p0 (s_base) of
// all P expert ids, then the offsets (s_off) by an exclusive scan; every
// thread of the workgroup takes part.
__device__ __forceinline__ void count_before(const int32_t *__restrict__ ids, int P, int p0, int E, int *s_tot,
                                             int *s_base, int *s_off) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // ids in batches of 16 per thread: a batch's loads are all requested
  // before its first counter update, so it waits for memory once
  constexpr int kCountBatch = 16;
  for (int q = 0; q < P; q += kCountBatch * kSegThreads) {
    int ev[kCountBatch];
#pragma unroll
    for (int u = 0; u < kCountBatch; ++u) {
      const int p = q + u * kSegThreads + tid;
      ev[u] = p < P ? ids[p] : -1;
    }
#pragma unroll
    for (int u = 0; u < kCountBatch; ++u) {
      const int p = q + u * kSegThreads + tid;
      if (ev[u] >= 0) {
        atomicAdd(&s_tot[ev[u]], 1);
        if (p < p0) atomicAdd(&s_base[ev[u]], 1);
      }
    }
  }
  __syncthreads();
  if (wave == 0) {
    int carry = 0;
    for (int base = 0; base < E; base += kWave) {
      const int e = base + lane;
      const int c = e < E ? s_tot[e] : 0;
      int incl = c;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int o = __shfl_up(incl, off, kWave);
        if (lane >= off) incl += o;
      }
      if (e < E) s_off[e] = carry + incl - c;
      carry += __shfl(incl, kWave - 1, kWave);
    }
    if (lane == 0) s_off[E] = carry;
  }
  __syncthreads();
}

// Segment blockIdx.x: per-expert pair totals and the counts of the pairs
// before the segment, from all T*k expert ids (LDS counters); expert
// offsets by an exclusive scan (segment 0 writes them); then the stable
// placement of the segment's pairs in ascending pair id (ballot peer masks
// inside a wave, per-wave counts across waves and chunks).
// seg_base (long batches, see route_scan_kernel): the segment's first
// position per expert, computed beforehand; the kernel then only places.
__global__ void __launch_bounds__(kSegThreads)
route_place_kernel(const int32_t *__restrict__ ids, int T, int E, int k, int32_t *__restrict__ offsets,
                   int32_t *__restrict__ sorted_pairs, int32_t *__restrict__ pair_pos,
                   const int32_t *__restrict__ seg_base) {
  __shared__ int s_tot[kMaxE];
  __shared__ int s_base[kMaxE];
  __shared__ int s_off[kMaxE + 1];
  __shared__ int s_run[kMaxE];
  __shared__ int s_wave[kSegWaves][kMaxE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int seg = blockIdx.x;
  const int P = T * k;
  const int p0 = seg * kSegTokens * k, p1 = std::min(T, (seg + 1) * kSegTokens) * k;
  for (int e = tid; e < E; e += kSegThreads) { s_tot[e] = 0; s_base[e] = 0; s_run[e] = 0; }
  if (seg_base) {
    for (int e = tid; e < E; e += kSegThreads) s_base[e] = seg_base[(int64_t)seg * E + e];
    __syncthreads();
  } else {
    __syncthreads();
    count_before(ids, P, p0, E, s_tot, s_base, s_off);
    if (seg == 0)
      for (int e = tid; e <= E; e += kSegThreads) offsets[e] = s_off[e];
    for (int e = tid; e < E; e += kSegThreads) s_base[e] += s_off[e];
    __syncthreads();
  }
  for (int base = p0; base < p1; base += kSegThreads) {
    const int p = base + tid;
    const bool valid = p < p1;
    const int e = valid ? ids[p] : 0;
    uint64_t peers = __ballot(valid);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint64_t bal = __ballot(valid && ((e >> b) & 1));
      peers &= ((e >> b) & 1) ? bal : ~bal;
    }
    const uint64_t below = (lane == 0) ? 0ull : (~0ull >> (64 - lane));
    const int rank = __popcll(peers & below);
    const bool leader = valid && (peers & below) == 0;
    for (int x = tid; x < kSegWaves * kMaxE; x += kSegThreads) (&s_wave[0][0])[x] = 0;
    __syncthreads();
    if (leader) s_wave[wave][e] = __popcll(peers);
    __syncthreads();
    if (valid) {
      int before = s_run[e];
      for (int w = 0; w < wave; ++w) before += s_wave[w][e];
      const int pos = s_base[e] + before + rank;
      sorted_pairs[pos] = p;
      pair_pos[p] = pos;
    }
    __syncthreads();
    for (int x = tid; x < E; x += kSegThreads) {
      int add = 0;
      for (int w = 0; w < kSegWaves; ++w) add += s_wave[w][x];
      s_run[x] += add;
    }
    __syncthreads();
  }
}

// ---- long batches: the placement above counts every pair in every
// segment (T^2 k / 64 counter updates in all).  Beyond kScanMinTokens the
// counts go through a workspace instead: each segment's per-expert
// histogram (route_count_kernel), then one workgroup turns them into each
// segment's first position per expert and the expert offsets
// (route_scan_kernel), and the placement starts from those.
constexpr int kScanMinTokens = 4096;

__global__ void __launch_bounds__(kSegThreads)
route_count_kernel(const int32_t *__restrict__ ids, int T, int E, int k, int32_t *__restrict__ hist) {
  __shared__ int s_cnt[kMaxE];
  const int tid = threadIdx.x, seg = blockIdx.x;
  const int p0 = seg * kSegTokens * k, p1 = std::min(T, (seg + 1) * kSegTokens) * k;
  for (int e = tid; e < E; e += kSegThreads) s_cnt[e] = 0;
  __syncthreads();
  for (int p = p0 + tid; p < p1; p += kSegThreads) atomicAdd(&s_cnt[ids[p]], 1);
  __syncthreads();
  for (int e = tid; e < E; e += kSegThreads) hist[(int64_t)seg * E + e] = s_cnt[e];
}

// One workgroup: every expert's segments in kScanParts parts of consecutive
// ones, a thread per expert and part.  The parts' sums and the experts' totals
// give each part's first position, the offsets are the exclusive scan of the
// totals; then each segment's first position per expert is written over its
// histogram.  Loads in batches of 16 segments, so that a batch waits for
// memory once; what a thread has loaded last it does not load again (8192
// tokens, 256 experts: 24 us with one part and a second pass over all, now
// 8 us).
constexpr int kScanParts = 4;
constexpr int kScanThreads = kMaxE * kScanParts;
constexpr int kScanBatch = 16;

__global__ void __launch_bounds__(kScanThreads)
route_scan_kernel(int nseg, int E, int32_t *__restrict__ hist, int32_t *__restrict__ offsets, int halves) {
  // (halves: a word holds the counts of its segment's halves, 16 bits each)
  const auto count = [&](int v) { return halves ? (v & 0xffff) + (v >> 16) : v; };
  __shared__ int s_part[kScanParts][kMaxE];
  __shared__ int s_off[kMaxE + 1];
  const int e = threadIdx.x % kMaxE, part = threadIdx.x / kMaxE, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (nseg + kScanParts - 1) / kScanParts, s0 = std::min(nseg, part * per), s1 = std::min(nseg, s0 + per);
  int c[2 * kScanBatch];   // the first segments' counts
  int sum = 0;
#pragma unroll
  for (int u = 0; u < 2 * kScanBatch; ++u) c[u] = e < E && s0 + u < s1 ? hist[(int64_t)(s0 + u) * E + e] : 0;
#pragma unroll
  for (int u = 0; u < 2 * kScanBatch; ++u) sum += c[u] = count(c[u]);
  for (int s = s0 + 2 * kScanBatch; s < s1; s += kScanBatch) {
    int d[kScanBatch];
#pragma unroll
    for (int u = 0; u < kScanBatch; ++u) d[u] = e < E && s + u < s1 ? hist[(int64_t)(s + u) * E + e] : 0;
#pragma unroll
    for (int u = 0; u < kScanBatch; ++u) sum += count(d[u]);
  }
  s_part[part][e] = sum;
  __syncthreads();
  if (wave == 0) {
    int carry = 0;
    for (int base = 0; base < E; base += kWave) {
      const int x = base + lane;
      int cnt = 0;
      if (x < E)
        for (int q = 0; q < kScanParts; ++q) cnt += s_part[q][x];
      int incl = cnt;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int o = __shfl_up(incl, off, kWave);
        if (lane >= off) incl += o;
      }
      if (x < E) s_off[x] = carry + incl - cnt;
      carry += __shfl(incl, kWave - 1, kWave);
    }
    if (lane == 0) s_off[E] = carry;
  }
  __syncthreads();
  for (int x = threadIdx.x; x <= E; x += kScanThreads) offsets[x] = s_off[x];
  if (e >= E) return;
  int run = s_off[e];
  for (int q = 0; q < part; ++q) run += s_part[q][e];
#pragma unroll
  for (int u = 0; u < 2 * kScanBatch; ++u) {
    if (s0 + u < s1) hist[(int64_t)(s0 + u) * E + e] = run;
    run += c[u];
  }
  for (int s = s0 + 2 * kScanBatch; s < s1; s += kScanBatch) {
    int d[kScanBatch];
#pragma unroll
    for (int u = 0; u < kScanBatch; ++u) d[u] = s + u < s1 ? hist[(int64_t)(s + u) * E + e] : 0;
#pragma unroll
    for (int u = 0; u < kScanBatch; ++u) {
      if (s + u < s1) hist[(int64_t)(s + u) * E + e] = run;
      run += count(d[u]);
    }
  }
}

// Routing mass (PagedWeight review summary: routing-mass buckets protect
// frequently used experts): m_e = sum of the gates of expert e's pairs.
// One wave per expert: lane-strided partial sums over the expert's sorted
// pairs, then a fixed xor-shuffle tree, so the result is deterministic.
// bucket_e = number of edges <= m_e.
constexpr int kMaxEdges = 8;
struct MassEdges {
  float v[kMaxEdges];
  int n;
};

__global__ void __launch_bounds__(256)
route_mass_kernel(const float *__restrict__ gates, const int32_t *__restrict__ offsets,
                  const int32_t *__restrict__ sorted_pairs, int E, MassEdges ed, float *__restrict__ mass,
                  int32_t *__restrict__ bucket) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (e >= E) return;
  const int lo = offsets[e], hi = offsets[e + 1];
  float acc = 0.f;
  for (int pos = lo + lane; pos < hi; pos += kWave) acc += gates[sorted_pairs[pos]];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) acc += __shfl_xor(acc, off, kWave);
  if (lane == 0) {
    mass[e] = acc;
    if (bucket) {
      int b = 0;
      for (int i = 0; i < ed.n; ++i) b += ed.v[i] <= acc ? 1 : 0;
      bucket[e] = b;
    }
  }
}

size_t route_ws_bytes(int T, int E) { return T > kScanMinTokens ? (size_t)route_segments(T) * E * 4 : 0; }

void launch_place(const int32_t *ids, int T, int E, int k, int32_t *offsets, int32_t *sorted_pairs, int32_t *pair_pos,
                  void *ws, bool halves, hipStream_t stream) {
  const int nseg = std::max(1, route_segments(T));   // (no tokens: the offsets alone)
  int32_t *hist = nullptr;
  if (T > kScanMinTokens) {
    hist = static_cast<int32_t *>(ws);
    if (!halves)
      hipLaunchKernelGGL(route_count_kernel, dim3(nseg), dim3(kSegThreads), 0, stream, ids, T, E, k, hist);
    hipLaunchKernelGGL(route_scan_kernel, dim3(1), dim3(kScanThreads), 0, stream, nseg, E, hist, offsets, (int)halves);
  }
  hipLaunchKernelGGL(route_place_kernel, dim3(nseg), dim3(kSegThreads), 0, stream, ids, T, E, k, offsets, sorted_pairs,
                     pair_pos, (const int32_t *)hist);
}

}  // namespace moeq

using namespace moeq;

// Up to kRouteSingleMax tokens: the single-workgroup kernel (one launch,
// one wave per token); more: the top-k and placement kernels (measured:
// 9.7 against 11.9 us at 64 tokens, 9.4 against 7.8 us at 16).  The
// workspace is needed only beyond kScanMinTokens tokens.
constexpr int kRouteSingleMax = kRouteTokens;
static inline bool route_single(int T) { return T <= kRouteSingleMax; }

MOEQ_API moeq_status moeq_route_workspace_size(int32_t T, int32_t E, int32_t k, size_t *bytes) {
  if (!bytes) return fail(MOEQ_ERR_INVALID, "route_workspace_size: null output");
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > E)
    return fail(MOEQ_ERR_INVALID, "route_workspace_size: T=%d E=%d k=%d invalid", T, E, k);
  *bytes = route_ws_bytes(T, E);
  return MOEQ_OK;
}

MOEQ_API moeq_status moeq_route(const float *logits, int32_t T, int32_t E, int32_t k,
                                const moeq_routing *out, void *ws, size_t ws_bytes,
                                hipStream_t stream) {
  if (!out) return fail(MOEQ_ERR_INVALID, "route: null routing output");
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > E)
    return fail(MOEQ_ERR_INVALID, "route: T=%d E=%d k=%d invalid (need 1 <= k <= E <= 256)", T, E, k);
  if ((int64_t)T * k > (int64_t)0x7fffffff) return fail(MOEQ_ERR_UNSUPPORTED, "route: T*k too large");
  if (!out->expert_offsets || (T > 0 && (!logits || !out->topk_ids || !out->topk_gates ||
                                         !out->sorted_pairs || !out->pair_pos)))
    return fail(MOEQ_ERR_INVALID, "route: null pointer");
  const size_t need = route_ws_bytes(T, E);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOEQ_ERR_WORKSPACE, "route: workspace has %zu bytes, needs %zu", ws_bytes, need);
  prof_begin("route", stream);
  if (route_single(T)) {
    const RouteOut o{logits, out->topk_ids, out->topk_gates, out->expert_offsets, out->sorted_pairs, out->pair_pos};
    hipLaunchKernelGGL(route_kernel, dim3(1), dim3(kRouteThreads), 0, stream, o, T, E, k);
  } else {
    hipLaunchKernelGGL(route_topk_kernel, dim3((T + kTopkWaves - 1) / kTopkWaves), dim3(kTopkThreads), 0, stream,
                       logits, T, E, k, out->topk_ids, out->topk_gates);
    launch_place(out->topk_ids, T, E, k, out->expert_offsets, out->sorted_pairs, out->pair_pos, ws, false, stream);
  }
  prof_end("route", stream);
  return check_launch("route");
}

MOEQ_API moeq_status moeq_route_mass(const moeq_routing *r, int32_t T, int32_t E, int32_t k, const float *edges,
                                     int32_t n_edges, float *mass, int32_t *bucket, hipStream_t stream) {
  if (!r) return fail(MOEQ_ERR_INVALID, "route_mass: null routing");
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > E)
    return fail(MOEQ_ERR_INVALID, "route_mass: T=%d E=%d k=%d invalid", T, E, k);
  if (n_edges < 0 || n_edges > kMaxEdges || (n_edges > 0 && !edges))
    return fail(MOEQ_ERR_INVALID, "route_mass: n_edges=%d not in 0..%d (or null edges)", n_edges, kMaxEdges);
  MassEdges ed{};
  ed.n = n_edges;
  for (int i = 0; i < n_edges; ++i) {
    if (!(edges[i] == edges[i]) || (i > 0 && edges[i] < edges[i - 1]))
      return fail(MOEQ_ERR_INVALID, "route_mass: edges must be ascending and not NaN");
    ed.v[i] = edges[i];
  }
  if (!mass || !r->expert_offsets || (T > 0 && (!r->topk_gates || !r->sorted_pairs)))
    return fail(MOEQ_ERR_INVALID, "route_mass: null pointer");
  prof_begin("route_mass", stream);
  hipLaunchKernelGGL(route_mass_kernel, dim3((E + 3) / 4), dim3(256), 0, stream, r->topk_gates, r->expert_offsets,
                     r->sorted_pairs, E, ed, mass, bucket);
  prof_end("route_mass", stream);
  return check_launch("route_mass");
}
