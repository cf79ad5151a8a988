// Router of the mixture of experts: from the gate's fp16 logits [T, E] to the
// top-k experts of every token, their combine weights, and the expert-grouped
// row layout that the dispatch quantizer, the grouped linears and the combine
// read -- all on the device, so a step needs no host round trip.
//
// Selection: the k largest logits, ties to the lower expert.  A logit becomes a
// 32-bit key whose unsigned order is that rule: the order-preserving 16-bit
// image of the fp16 value (-0 as +0, NaN below -inf) over the complemented
// expert index, so one redux.sync maximum per choice finds value and expert.
// Weights (fp32): exp(l_j - l_max) over the sum of the same over the chosen
// experts, or over all of them; the maximum itself counts as 1, so a token whose
// largest logit is +inf shares its weight among the experts that have it, and a
// token without any logit above -inf gets weight 0 everywhere.
// Grouping: rows ordered by (expert, token): a counting sort.  Every warp takes
// a run of consecutive tokens and counts its rows per expert in a table of its
// own; prefix sums over warps, chunks of tokens and experts turn the counts into
// first rows, and the second walk over the same tokens hands the rows out in
// order.  No atomic's order reaches a result.
//
// Bound: launches and latency.  Up to 64 tokens one CTA; up to 1024 one cluster, whose
// CTAs read each other's counts from shared memory; both one launch.  Above, two
// launches over up to 128 CTAs, the counts of all chunks in between: there the choices'
// instructions want all SMs.  Measured on B200 (graph): 1 token 2.7 us; 256 tokens, 64
// experts 5.0 us (two launches 6.4); 1000 tokens, 160 experts, 6 choices 10.6 us (8.9,
// but called from Python, where a launch is what costs, 17.8 against 20.4); 8192
// tokens, 64 experts 8.5 us (one cluster 22.7).  With hundreds of experts and many
// choices it is bound by the instructions of the choices, two per key and choice: 4096
// tokens with 8 choices of 256 experts 16.5 us, of 1024 45.6.  Weights over all experts:
// 1000 tokens, 160 experts 12.1 us.
#pragma once

#include "ptx.cuh"

namespace fp8q {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 8;
constexpr int kRouteOneCtaTokens = 64;    // at most: one CTA, one launch
constexpr int kRouteClusterTokens = 1024;  // at most: one cluster
constexpr int kRouteMaxCluster = 16;
constexpr int kRouteMaxChunks = 128;      // CTAs of the two-launch form

struct RouteParams {
  const __half* logits;   // [T, E]
  int T, E, topk;
  int renormalize;        // 1: weights sum to 1 over the chosen experts; 0: softmax over all experts
  int chunk;              // tokens per CTA
  int chunks;             // CTAs
  int32_t* experts;       // [T, topk]
  float* weights;         // [T, topk]
  int32_t* offsets;       // [E + 1]
  int32_t* row_token;     // [T * topk]
  float* row_weight;      // [T * topk]
  int32_t* token_rows;    // [T, topk]
  int32_t* counts;        // [chunks, E] workspace of the two-launch form
};

// Tokens of a CTA of the two-launch form.
inline int route_chunk(int64_t T) {
  const int64_t c = (T + kRouteMaxChunks - 1) / kRouteMaxChunks;
  return static_cast<int>(c < 32 ? 32 : c);
}

// fp16 bits -> 16-bit unsigned of the same order; NaN -> 0, -0 -> +0.
__device__ __forceinline__ uint32_t route_order(uint32_t h) {
  if ((h & 0x7fffu) > 0x7c00u) return 0u;
  if (h == 0x8000u) h = 0u;
  return (h & 0x8000u) ? (~h & 0xffffu) : (h | 0x8000u);
}
// The logit of a key (NaN: -inf, which weighs nothing).
__device__ __forceinline__ float route_logit(uint32_t key) {
  const uint32_t o = key >> 16;
  const uint32_t h = o == 0u ? 0xfc00u : (o & 0x8000u) ? (o & 0x7fffu) : (~o & 0xffffu);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}
// exp(l - m) of the softmax; m is the token's largest logit.
__device__ __forceinline__ float route_exp(float l, float m) {
  if (m == -INFINITY) return 0.0f;
  return l == m ? 1.0f : expf(l - m);
}

// Tokens [first, last) of this warp within its CTA's chunk.
struct RouteSpan {
  int first, last;
};
__device__ __forceinline__ RouteSpan route_span(const RouteParams& p, int warp, int warps) {
  const int c0 = static_cast<int>(blockIdx.x) * p.chunk;
  const int n = max(0, min(p.chunk, p.T - c0));
  const int per = (n + warps - 1) / warps;
  RouteSpan s;
  s.first = c0 + min(n, warp * per);
  s.last = c0 + min(n, (warp + 1) * per);
  return s;
}

// Choose the experts of this warp's tokens; count them per expert in `hist`.
template <int KPL>
__device__ __forceinline__ void route_choose(const RouteParams& p, const RouteSpan& s, uint16_t* hist, int lane) {
  unsigned short raw[KPL];   // the next token's logits, loaded while one is worked on
  auto fetch = [&](int t) {
    const unsigned short* src = reinterpret_cast<const unsigned short*>(p.logits + static_cast<int64_t>(t) * p.E);
#pragma unroll
    for (int i = 0; i < KPL; ++i) raw[i] = lane + 32 * i < p.E ? __ldg(src + lane + 32 * i) : 0;
  };
  if (s.first < s.last) fetch(s.first);
  for (int t = s.first; t < s.last; ++t) {
    uint32_t key[KPL];
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int e = lane + 32 * i;
      key[i] = e < p.E ? (route_order(raw[i]) << 16) | (0xffffu - static_cast<uint32_t>(e)) : 0u;
    }
    if (t + 1 < s.last) fetch(t + 1);
    float all = 0.0f, m = 0.0f;
    uint32_t mine = 0;   // lane j: the j-th choice
    for (int j = 0; j < p.topk; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < KPL; ++i) best = max(best, key[i]);
      best = __reduce_max_sync(0xffffffffu, best);
      if (j == 0) {
        m = route_logit(best);
        if (!p.renormalize) {
#pragma unroll
          for (int i = 0; i < KPL; ++i)
            if (key[i] != 0u) all += route_exp(route_logit(key[i]), m);
        }
      }
      if (lane == j) mine = best;
#pragma unroll
      for (int i = 0; i < KPL; ++i)
        if (key[i] == best) key[i] = 0u;
    }
    const bool have = lane < p.topk;
    const float z = have ? route_exp(route_logit(mine), m) : 0.0f;
    float sum = p.renormalize ? z : all;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (have) {
      const int e = static_cast<int>(0xffffu - (mine & 0xffffu));
      const int64_t at = static_cast<int64_t>(t) * p.topk + lane;
      p.experts[at] = e;
      p.weights[at] = sum > 0.0f ? __fdiv_rn(z, sum) : 0.0f;
      ++hist[e];   // a token's experts are distinct: no two lanes share a counter
    }
    __syncwarp();
  }
}

// hist[w][e] -> rows of expert e in the warps before w; returns their sum.
template <int WARPS>
__device__ __forceinline__ int route_warp_prefix(uint16_t* hist, int E, int e) {
  int acc = 0;
#pragma unroll
  for (int w0 = 0; w0 < WARPS; w0 += 8) {   // eight reads in flight
    int c[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) c[u] = hist[(w0 + u) * E + e];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      hist[(w0 + u) * E + e] = static_cast<uint16_t>(acc);
      acc += c[u];
    }
  }
  return acc;
}

// Exclusive prefix sum over the experts by one warp: first[e] and, at [E], the sum.
__device__ __forceinline__ void route_expert_prefix(int E, const int* total, int* first, int lane) {
  const int per = (E + 31) / 32;
  const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) sum += total[e];
  int acc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, acc, o);
    if (lane >= o) acc += v;
  }
  int at = acc - sum;
  for (int e = e0; e < e1; ++e) {
    const int c = total[e];   // (total may be first)
    first[e] = at;
    at += c;
  }
  if (lane == 31) first[E] = acc;
}

// The rows (token, choice) of this warp's tokens, 32 at a time in their order: f(row's
// position in [T, topk], its expert, its rank among the rows of that expert so far).
// `hist` counts them per expert.
template <typename F>
__device__ __forceinline__ void route_walk(const RouteParams& p, const RouteSpan& s, uint16_t* hist, int lane, F f) {
  const int64_t last = static_cast<int64_t>(s.last) * p.topk;
  for (int64_t at0 = static_cast<int64_t>(s.first) * p.topk; at0 < last; at0 += 32) {
    const int64_t at = at0 + lane;
    const int e = at < last ? p.experts[at] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);   // lanes with the same expert
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int before = e >= 0 ? hist[e] : 0;
    __syncwarp();
    if (e >= 0) {
      if (rank == 0) hist[e] = static_cast<uint16_t>(before + __popc(same));
      f(at, e, before + rank);
    }
    __syncwarp();
  }
}

// Hand out the rows.  base[e]: the first row of expert e in this chunk; hist[e]: this
// warp's next row within it.
__device__ __forceinline__ void route_place(const RouteParams& p, const RouteSpan& s, uint16_t* hist, const int* base,
                                            int lane) {
  route_walk(p, s, hist, lane, [&](int64_t at, int e, int place) {
    const int row = base[e] + place;
    p.token_rows[at] = row;
    p.row_token[row] = static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(p.topk));
    p.row_weight[row] = p.weights[at];
  });
}

// Shared memory: per-warp counters [warps][E] uint16, then three int tables [E + 1].
inline size_t route_smem(int E, int warps) {
  return ((static_cast<size_t>(warps) * E * 2 + 15) & ~size_t(15)) + 3 * static_cast<size_t>(E + 1) * 4;
}
struct RouteTables {
  uint16_t* hist;
  int* total;
  int* first;
  int* all;
};
__device__ __forceinline__ RouteTables route_tables(uint8_t* smem, int E, int warps) {
  RouteTables r;
  r.hist = reinterpret_cast<uint16_t*>(smem);
  r.total = reinterpret_cast<int*>(smem + ((static_cast<size_t>(warps) * E * 2 + 15) & ~size_t(15)));
  r.first = r.total + (E + 1);
  r.all = r.first + (E + 1);
  return r;
}

// First launch: choices and counts.  One CTA alone goes on to place the rows; so do
// the CTAs of a cluster (kCluster: the grid is one), each reading the others'
// counts from their shared memory.
template <int KPL, int THREADS, bool kCluster>
__global__ void __launch_bounds__(THREADS) route_choose_kernel(const RouteParams p) {
  extern __shared__ __align__(16) uint8_t route_smem_raw[];
  constexpr int kWarps = THREADS / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RouteTables tb = route_tables(route_smem_raw, p.E, kWarps);
  for (int i = threadIdx.x; i < kWarps * p.E; i += THREADS) tb.hist[i] = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const RouteSpan s = route_span(p, warp, kWarps);
  uint16_t* hist = tb.hist + warp * p.E;
  route_choose<KPL>(p, s, hist, lane);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += THREADS) tb.total[e] = route_warp_prefix<kWarps>(tb.hist, p.E, e);
  __syncthreads();
  if (kCluster) {
    cluster_arrive();
    cluster_wait();
    const int rank = static_cast<int>(cluster_ctarank()), n = static_cast<int>(cluster_nctarank());
    for (int e = threadIdx.x; e < p.E; e += THREADS) {
      const uint32_t at = smem_u32(tb.total + e);
      int before = 0, sum = 0;
      for (int c0 = 0; c0 < n; c0 += 8) {   // (n is 8 or 16)
        int v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = ld_dsmem_i32(mapa_shared(at, static_cast<uint32_t>(c0 + u)));
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          sum += v[u];
          if (c0 + u < rank) before += v[u];
        }
      }
      tb.all[e] = sum;
      tb.first[e] = before;
    }
    __syncthreads();
    cluster_arrive();   // no CTA leaves while another reads its counts
    if (warp == 0) route_expert_prefix(p.E, tb.all, tb.all, lane);   // all[e] -> first row of expert e
    __syncthreads();
    if (rank == 0)
      for (int e = threadIdx.x; e <= p.E; e += THREADS) p.offsets[e] = tb.all[e];
    for (int e = threadIdx.x; e < p.E; e += THREADS) tb.first[e] += tb.all[e];
    __syncthreads();
    route_place(p, s, hist, tb.first, lane);
    cluster_wait();
    return;
  }
  if (p.chunks > 1) {
    for (int e = threadIdx.x; e < p.E; e += THREADS)
      p.counts[static_cast<int64_t>(blockIdx.x) * p.E + e] = tb.total[e];
    return;
  }
  if (warp == 0) route_expert_prefix(p.E, tb.total, tb.first, lane);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += THREADS) p.offsets[e] = tb.first[e];
  route_place(p, s, hist, tb.first, lane);
}

// Second launch: the first row of every (chunk, expert) from the counts of all
// chunks, then the rows of this chunk.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) route_place_kernel(const RouteParams p) {
  extern __shared__ __align__(16) uint8_t route_smem_raw[];
  constexpr int kWarps = THREADS / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RouteTables tb = route_tables(route_smem_raw, p.E, kWarps);
  for (int i = threadIdx.x; i < kWarps * p.E; i += THREADS) tb.hist[i] = 0;
  for (int e = threadIdx.x; e <= p.E; e += THREADS) tb.total[e] = tb.first[e] = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  // rows of each expert in the chunks before this one (first) and in all (total)
  const int parts = max(1, THREADS / p.E);
  for (int i = threadIdx.x; i < parts * p.E; i += THREADS) {
    const int e = i % p.E;
    int before = 0, sum = 0;
    for (int c0 = i / p.E; c0 < p.chunks; c0 += 8 * parts) {   // eight loads in flight
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = c0 + u * parts < p.chunks ? p.counts[static_cast<int64_t>(c0 + u * parts) * p.E + e] : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        sum += v[u];
        if (c0 + u * parts < static_cast<int>(blockIdx.x)) before += v[u];
      }
    }
    atomicAdd(&tb.total[e], sum);      // integers: the order does not matter
    atomicAdd(&tb.first[e], before);
  }
  // this warp's rows per expert
  const RouteSpan s = route_span(p, warp, kWarps);
  uint16_t* hist = tb.hist + warp * p.E;
  route_walk(p, s, hist, lane, [](int64_t, int, int) {});
  __syncthreads();
  if (warp == 0) route_expert_prefix(p.E, tb.total, tb.total, lane);   // total[e] -> first row of expert e
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= p.E; e += THREADS) p.offsets[e] = tb.total[e];
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
    tb.first[e] += tb.total[e];
    route_warp_prefix<kWarps>(tb.hist, p.E, e);
  }
  __syncthreads();
  route_place(p, s, hist, tb.first, lane);
}

}  // namespace fp8q
