// Routing of a mixture-of-experts layer: the k largest logits of each token (ties to
// the lowest index), their weights, and the (token, choice) pairs sorted by expert.
//
// A warp holds a token's logits as order-preserving 32-bit keys, key i of lane l
// belonging to expert 32 i + l, and takes the largest k times: one warp-wide integer
// maximum finds the value, one ballot (or, on a tie, one warp-wide minimum of the
// indices) the expert.  Selection compares the logits themselves, so it is exact:
// softmax and sigmoid are both increasing.  A NaN ranks as -infinity.
#pragma once
#include <type_traits>

#include "mx.cuh"
#include "ptx.cuh"

namespace macaq {

constexpr int kMaxChoices = 32;  // lane j of a warp ends up with choice j

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
// Logits are read past L1: in the layer's second kernel they may have been written
// since this SM's L1 last saw them.
__device__ __forceinline__ float load_logit(const RouteRule& r, int64_t at) {
  if (r.logits_f32) return __ldcg(static_cast<const float*>(r.logits) + at);
  return bf16lo(__ldcg(static_cast<const unsigned short*>(r.logits) + at));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One warp, one token: lane j < k receives choice j (the experts in falling order of
// their logits) and its weight.  L: keys per lane, 32 L >= E.
//   softmax: exp(l_j - max) / sum, over all E or (renorm) the chosen
//   sigmoid: 1 / (1 + exp(-l_j)), divided (renorm) by the sum of the chosen
// A logit of -infinity has weight zero, also where all are -infinity (a sigmoid
// below 2^-126 is zero too).  A NaN logit makes the weights of its token NaN where
// it is chosen or enters the sum.
template <int L>
__device__ __forceinline__ void choose_experts(const RouteRule& r, int64_t token, int& expert, float& weight) {
  const int lane = threadIdx.x & 31;
  const int64_t base = token * r.E;
  uint32_t key[L];
  bool nan = false;
  float v[L];
#pragma unroll
  for (int i = 0; i < L; ++i) v[i] = i * 32 + lane < r.E ? load_logit(r, base + i * 32 + lane) : 0.f;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    key[i] = i * 32 + lane < r.E ? logit_key(v[i]) : 0u;
    nan = nan || (i * 32 + lane < r.E && isnan(v[i]));
  }
  uint32_t mine = 0;  // key of this lane's choice
  float all = 0.f;    // softmax over all E: its sum
  uint32_t top = 0;   // the largest key
  expert = 0;
  for (int j = 0; j < r.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < L; ++i) best = max(best, key[i]);
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    int at = 0;
#pragma unroll
    for (int i = L - 1; i >= 0; --i)
      if (key[i] == m) at = i;  // the lowest of this lane's
    const uint32_t who = __ballot_sync(0xffffffffu, best == m);
    uint32_t e;
    if ((who & (who - 1)) == 0) e = static_cast<uint32_t>(__shfl_sync(0xffffffffu, at * 32 + lane, __ffs(who) - 1));
    else e = __reduce_min_sync(0xffffffffu, best == m ? static_cast<uint32_t>(at * 32 + lane) : 0xffffffffu);
    if (j == 0) {
      top = m;
      if (!r.sigmoid && !r.renorm) {
        const float mx = (m & 0x80000000u) ? __uint_as_float(m & 0x7FFFFFFFu) : __uint_as_float(~m);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i)
          if (i * 32 + lane < r.E && v[i] != -INFINITY) s += __expf(v[i] - mx);
        all = warp_sum(s);
      }
    }
    if (lane == j) {
      expert = static_cast<int>(e);
      mine = m;
    }
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (i * 32 + lane == static_cast<int>(e)) key[i] = 0u;
  }
  // the choice's own logit, NaN included (its key says -infinity)
  float l = (mine & 0x80000000u) ? __uint_as_float(mine & 0x7FFFFFFFu) : __uint_as_float(~mine);
  if (__any_sync(0xffffffffu, nan) && lane < r.k) l = load_logit(r, base + expert);
  const float mx = (top & 0x80000000u) ? __uint_as_float(top & 0x7FFFFFFFu) : __uint_as_float(~top);
  if (lane >= r.k || l == -INFINITY) weight = 0.f;  // also where the largest logit is -infinity itself
  else if (r.sigmoid) weight = __fdividef(1.0f, 1.0f + __expf(-l));
  else weight = __expf(l - mx);
  if (r.renorm || !r.sigmoid) {
    const float sum = r.renorm ? warp_sum(weight) : all;
    weight = sum == 0.f ? 0.f : __fdividef(weight, sum);
  }
  weight *= r.scale;
}

template <typename F>
__device__ __forceinline__ void for_keys_per_lane(int E, F&& f) {
  if (E <= 32) f(std::integral_constant<int, 1>());
  else if (E <= 64) f(std::integral_constant<int, 2>());
  else if (E <= 128) f(std::integral_constant<int, 4>());
  else if (E <= 256) f(std::integral_constant<int, 8>());
  else if (E <= 512) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 32>());
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  for_keys_per_lane(E, [&](auto keys) {
    for (int64_t t = t0 + warp; t < t1; t += kRouteThreads / 32) {
      int e;
      float w;
      choose_experts<decltype(keys)::value>(p.rule, t, e, w);
      if (lane < k) {
        p.ids[t * k + lane] = e;
        p.weights[t * k + lane] = w;
        if (sorting) atomicAdd(&s.base[e], 1);
      }
    }
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
