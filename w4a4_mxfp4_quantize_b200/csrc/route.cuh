// Routing of a mixture-of-experts layer: the k largest logits of each token (ties to
// the lowest index), their weights, and the (token, choice) pairs sorted by expert.
//
// The lanes that share a token hold its logits as order-preserving 32-bit keys and take
// the largest k times.  Logits are read past L1: in the layer's second kernel they may
// have been written since this SM's L1 last saw them.  Selection compares the logits themselves, so it
// is exact: softmax and sigmoid are both increasing.  A NaN ranks as -infinity.
#pragma once
#include <type_traits>

#include "mx.cuh"
#include "ptx.cuh"

namespace macaq {

constexpr int kMaxChoices = 32;

struct RouteRule {
  const void* logits;  // [T, E], bf16 or fp32
  int logits_f32;
  int E, k;
  int sigmoid;   // score: 0 softmax over the E logits, 1 sigmoid of each
  int renorm;    // the k weights divided by their sum
  float scale;   // multiplies every weight
};

// Order-preserving unsigned key of a logit; -0 counts as +0 and NaN as -infinity.
// No logit has key 0: it marks an expert that is taken (or past E).
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (isnan(v)) v = -INFINITY;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return (key & 0x80000000u) ? __uint_as_float(key & 0x7FFFFFFFu) : __uint_as_float(~key);
}
__device__ __forceinline__ float load_logit(const RouteRule& r, int64_t at) {
  if (r.logits_f32) return __ldcg(static_cast<const float*>(r.logits) + at);
  return bf16lo(__ldcg(static_cast<const unsigned short*>(r.logits) + at));
}

// Reductions over the G lanes that share a token.
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (G == 32) {
    v = __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}
template <int G, typename V>
__device__ __forceinline__ V group_sum(V v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp chooses for 32 / G tokens at a time, G lanes to a token, lane g of them holding
// experts g L .. g L + L - 1 (G L >= E).  A round is a chain of steps that wait for one
// another: local maximum, maximum of the lanes, removal of the largest.  One token over
// 32 lanes takes 92 to 117 cycles a round (one warp-wide maximum instruction), four tokens
// over 8 lanes each about 150 (three exchanges): the first where every warp has a token
// at most, the second where there are more.
template <int G_, int L_>
struct Spread {
  static constexpr int G = G_, L = L_, kTokens = 32 / G_, kSlots = 32 / G_;  // choices per lane: k <= 32
};
template <int kMaxE, typename F>
__device__ __forceinline__ void for_spread(int E, bool few, F&& f) {
  if (few && E <= 128) f(Spread<32, 4>());
  else if (E <= 64) f(Spread<8, 8>());
  else if (E <= 128) f(Spread<8, 16>());
  else if (E <= 256) f(Spread<16, 16>());
  else if (kMaxE <= 512 || E <= 512) f(Spread<32, 16>());
  else f(Spread<32, 32>());
}

// One warp, up to kTokens tokens: token t0 + (lane / G) step.  Calls f(token, j, expert,
// weight) for each choice j < k of each token below t1, from the lane that holds it.
// `ids`: 32 kTokens words of shared memory of the warp's own.
//   softmax: exp(l_j - max) / sum, over all E or (renorm) the chosen
//   sigmoid: 1 / (1 + exp(-l_j)), divided (renorm) by the sum of the chosen
// A logit of -infinity has weight zero, also where all are -infinity (a sigmoid
// below 2^-126 is zero too).  A NaN logit makes the weights of its token NaN where
// it is chosen or enters the sum.
// A round takes every expert of the largest key.  Where that took more than k in the
// end, or left the last round nothing, some were equal: the rounds run once more, one
// expert a round, the lowest of the lowest lane.
template <typename S, typename F>
__device__ __forceinline__ void choose_experts(const RouteRule& r, int64_t t0, int64_t t1, int64_t step, int* ids, F&& f) {
  constexpr int G = S::G, L = S::L;
  const int lane = threadIdx.x & 31, g = lane % G, first = g * L;
  const int64_t mine = t0 + (lane / G) * step;
  const int64_t token = mine < t1 ? mine : t0;  // lanes without a token repeat the first
  const int64_t base = token * r.E + first;
  ids += lane / G * 32;
  uint32_t key[L];
  bool nan = false;
  const bool vec = r.E % 4 == 0;  // rows and lanes start on four logits
  if (r.logits_f32) {
    const float* p = static_cast<const float*>(r.logits) + base;
    if (vec) {
#pragma unroll
      for (int i = 0; i < L; i += 4) {
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (first + i < r.E) v = __ldcg(reinterpret_cast<const float4*>(p + i));
        key[i] = __float_as_uint(v.x);
        key[i + 1] = __float_as_uint(v.y);
        key[i + 2] = __float_as_uint(v.z);
        key[i + 3] = __float_as_uint(v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i) key[i] = first + i < r.E ? __float_as_uint(__ldcg(p + i)) : 0xFF800000u;
    }
  } else {
    const unsigned short* p = static_cast<const unsigned short*>(r.logits) + base;
    if (vec) {
#pragma unroll
      for (int i = 0; i < L; i += 4) {
        uint2 v = make_uint2(0xFF80FF80u, 0xFF80FF80u);
        if (first + i < r.E) v = __ldcg(reinterpret_cast<const uint2*>(p + i));
        key[i] = v.x << 16;
        key[i + 1] = v.x & 0xFFFF0000u;
        key[i + 2] = v.y << 16;
        key[i + 3] = v.y & 0xFFFF0000u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i) key[i] = first + i < r.E ? static_cast<uint32_t>(__ldcg(p + i)) << 16 : 0xFF800000u;
    }
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    nan = nan || isnan(__uint_as_float(key[i]));
    key[i] = first + i < r.E ? logit_key(__uint_as_float(key[i])) : 0u;
  }
  const uint32_t any_nan = __ballot_sync(0xffffffffu, nan) >> (lane / G * G);
  nan = (any_nan & (0xffffffffu >> (32 - G))) != 0;  // of this token
  auto local_max = [&] {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < L; ++i) m = max(m, key[i]);
    return m;
  };
  float all = 0.f;  // softmax over all E: its sum
  if (!r.sigmoid && !r.renorm) {
    const float mx = key_logit(group_max<G>(local_max()));
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const float v = key_logit(key[i]);
      all += key[i] == 0u || v == -INFINITY ? 0.f : __expf(v - mx);
    }
    all = group_sum<G>(all);
    if (nan) all = __int_as_float(0x7FFFFFFF);
  }
  uint32_t chosen[S::kSlots];  // keys of choices g, g + G, ...
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i) chosen[i] = 0u;
  uint32_t top = 0u, last = 0u;
#pragma unroll 1
  for (int j = 0; j < r.k; ++j) {
    const uint32_t m = group_max<G>(local_max());
    int hit = -1;
#pragma unroll
    for (int i = L - 1; i >= 0; --i) {
      const bool take = key[i] == m;
      hit = take ? first + i : hit;
      key[i] = take ? 0u : key[i];
    }
    if (hit >= 0) ids[j] = hit;
#pragma unroll
    for (int i = 0; i < S::kSlots; ++i) chosen[i] = j == g + i * G ? m : chosen[i];
    top = j == 0 ? m : top;
    last = m;
  }
  int taken = 0;
#pragma unroll
  for (int i = 0; i < L; ++i) taken += key[i] == 0u && first + i < r.E ? 1 : 0;
  const bool again = group_sum<G>(taken) != r.k || last == 0u;
  if (__any_sync(0xffffffffu, again)) {
#pragma unroll
    for (int i = 0; i < L; ++i) key[i] = first + i < r.E ? logit_key(load_logit(r, base + i)) : 0u;
#pragma unroll 1
    for (int j = 0; j < r.k; ++j) {
      const uint32_t best = local_max(), m = group_max<G>(best);
      const uint32_t who = __ballot_sync(0xffffffffu, best == m) >> (lane / G * G);
      bool own = g == __ffs(who) - 1;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        if (own && key[i] == m) {
          ids[j] = first + i;
          key[i] = 0u;
          own = false;
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < S::kSlots; ++i) chosen[i] = j == g + i * G ? m : chosen[i];
    }
  }
  __syncwarp();
  const float mx = key_logit(top);
  float w[S::kSlots], sum = 0.f;
  int e[S::kSlots];
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i) {
    const bool in = g + i * G < r.k;
    e[i] = in ? ids[g + i * G] : 0;
    float l = key_logit(chosen[i]);
    if (nan && in) {  // a NaN's key says -infinity
      l = load_logit(r, token * r.E + e[i]);
    }
    const float x = __expf(r.sigmoid ? -l : l - mx);
    w[i] = r.sigmoid ? __fdividef(1.0f, 1.0f + x) : x;
    w[i] = !in || l == -INFINITY ? 0.f : w[i];  // also where the largest logit is -infinity itself
    sum += w[i];
  }
  if (r.renorm || !r.sigmoid) {
    sum = r.renorm ? group_sum<G>(sum) : all;
#pragma unroll
    for (int i = 0; i < S::kSlots; ++i) w[i] = sum == 0.f ? 0.f : __fdividef(w[i], sum);
  }
  if (mine < t1) {
#pragma unroll
    for (int i = 0; i < S::kSlots; ++i)
      if (g + i * G < r.k) f(mine, g + i * G, e[i], w[i] * r.scale);
  }
  __syncwarp();  // `ids` may be written again
}

// ============================================================================
// Sorting the choices by expert
// ============================================================================
// Stable and without a sort: within a run of 64 tokens a token picks an expert at
// most once, so "how many earlier tokens of the run picked e" is a population count
// of a 64-bit mask per expert.  CTA b of kernel one handles tokens [b q, (b + 1) q),
// chooses their experts and counts them; kernel two adds up the counts of the CTAs
// before it (and of the experts before each), then places its own tokens 64 at a
// time.  At most kRouteCtas CTAs, so that adding up stays short.  One CTA alone does
// both parts in kernel one.
constexpr int kRouteThreads = 512;
constexpr int kRouteCtas = 148;
constexpr int kRouteRun = 64;
constexpr int kRouteMaxE = 1024;

struct RouteParams {
  RouteRule rule;
  int64_t T;
  int per_cta;       // q
  int32_t* ids;      // [T, k]
  float* weights;    // [T, k]
  int64_t* counts;   // [E] or nullptr (no sorting)
  int32_t* order;    // [T k]
  int32_t* hist;     // [gridDim.x, E] (more than one CTA)
};

struct RouteTables {
  int base[kRouteMaxE];                  // row that the next choice of expert e gets
  unsigned long long picked[kRouteMaxE]; // tokens of this run that picked e
  int warp_total[kRouteThreads / 32];
};

// base[e] (0 <= e < E, counts on entry) becomes the sum of the counts before e.
__device__ __forceinline__ void exclusive_prefix(RouteTables& s, int E) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += kRouteThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int c = e < E ? s.base[e] : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) s.warp_total[warp] = inc;
    __syncthreads();
    int before = carry, total = 0;
    for (int w = 0; w < kRouteThreads / 32; ++w) {
      if (w < warp) before += s.warp_total[w];
      total += s.warp_total[w];
    }
    if (e < E) s.base[e] = before + inc - c;
    carry += total;
    __syncthreads();
  }
}

// Places the choices of tokens [t0, t1), base[] holding the first free row of each expert.
__device__ __forceinline__ void place_choices(const RouteParams& p, RouteTables& s, int64_t t0, int64_t t1) {
  const int k = p.rule.k, E = p.rule.E;
  for (int e = threadIdx.x; e < E; e += kRouteThreads) s.picked[e] = 0ull;
  __syncthreads();
  for (int64_t r0 = t0; r0 < t1; r0 += kRouteRun) {
    const int n = static_cast<int>(min(static_cast<int64_t>(kRouteRun), t1 - r0)) * k;
    for (int i = threadIdx.x; i < n; i += kRouteThreads)
      atomicOr(&s.picked[p.ids[r0 * k + i]], 1ull << (i / k));
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kRouteThreads) {
      const int e = p.ids[r0 * k + i];
      p.order[s.base[e] + __popcll(s.picked[e] & ((1ull << (i / k)) - 1))] = static_cast<int32_t>(r0 * k + i);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      s.base[e] += __popcll(s.picked[e]);
      s.picked[e] = 0ull;
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(const __grid_constant__ RouteParams p) {
  __shared__ RouteTables s;
  __shared__ int ids[kRouteThreads / 32 * 128];
  const int warp = threadIdx.x >> 5;
  const int E = p.rule.E, k = p.rule.k;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.per_cta;
  const int64_t t1 = min(p.T, t0 + p.per_cta);
  const bool sorting = p.counts != nullptr;
  if (sorting) {
    for (int e = threadIdx.x; e < E; e += kRouteThreads) s.base[e] = 0;
    __syncthreads();
  }
  pdl_wait();  // the logits may come from the kernel before
  pdl_trigger();
  for_spread<kRouteMaxE>(E, t1 - t0 <= kRouteThreads / 32, [&](auto spread) {
    using S = decltype(spread);
    for (int64_t t = t0 + warp * S::kTokens; t < t1; t += kRouteThreads / 32 * S::kTokens)
      choose_experts<S>(p.rule, t, t1, 1, ids + warp * 128, [&](int64_t token, int j, int e, float w) {
        p.ids[token * k + j] = e;
        p.weights[token * k + j] = w;
        if (sorting) atomicAdd(&s.base[e], 1);
      });
  });
  if (!sorting) return;
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < E; e += kRouteThreads) p.hist[static_cast<int64_t>(blockIdx.x) * E + e] = s.base[e];
    return;
  }
  for (int e = threadIdx.x; e < E; e += kRouteThreads) p.counts[e] = s.base[e];
  __syncthreads();
  exclusive_prefix(s, E);
  place_choices(p, s, t0, t1);
}

__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const __grid_constant__ RouteParams p) {
  __shared__ RouteTables s;
  __shared__ int before[kRouteMaxE];  // choices of expert e in earlier CTAs
  const int E = p.rule.E, nb = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
  for (int e = threadIdx.x; e < E; e += kRouteThreads) s.base[e] = before[e] = 0;
  __syncthreads();
  pdl_wait();  // the counts and the choices come from the kernel before
  pdl_trigger();
  // thread (part, e): the CTAs part, part + parts, ... of expert e; integer sums, any order
  const int cols = min(E, kRouteThreads), parts = kRouteThreads / cols;
  const int part = static_cast<int>(threadIdx.x) / cols;
  if (part < parts) {
    for (int e = static_cast<int>(threadIdx.x) % cols; e < E; e += cols) {
      int total = 0, earlier = 0;
#pragma unroll 8
      for (int c = part; c < nb; c += parts) {
        const int h = __ldcg(p.hist + static_cast<int64_t>(c) * E + e);
        total += h;
        if (c < b) earlier += h;
      }
      atomicAdd(&s.base[e], total);
      atomicAdd(&before[e], earlier);
    }
  }
  __syncthreads();
  if (b == 0)
    for (int e = threadIdx.x; e < E; e += kRouteThreads) p.counts[e] = s.base[e];
  __syncthreads();
  exclusive_prefix(s, E);
  for (int e = threadIdx.x; e < E; e += kRouteThreads) s.base[e] += before[e];
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(b) * p.per_cta;
  place_choices(p, s, t0, min(p.T, t0 + p.per_cta));
}

}  // namespace macaq
