// Routing of a mixture-of-experts layer: the k largest logits of each token (ties to
// the lowest index), their weights, and the (token, choice) pairs sorted by expert.
//
// A warp holds a token's logits as order-preserving 32-bit keys and takes the largest k
// times.  Logits are read past L1: in the layer's second kernel they may
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
  const uint32_t u = __float_as_uint(fmaxf(v, -INFINITY) + 0.0f);  // the maximum of a NaN and a number is the number
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return (key & 0x80000000u) ? __uint_as_float(key & 0x7FFFFFFFu) : __uint_as_float(~key);
}
__device__ __forceinline__ float load_logit(const RouteRule& r, int64_t at) {
  if (r.logits_f32) return __ldcg(static_cast<const float*>(r.logits) + at);
  return bf16lo(__ldcg(static_cast<const unsigned short*>(r.logits) + at));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int kMaxE, typename F>
__device__ __forceinline__ void for_keys_per_lane(int E, F&& f) {
  if (E <= 64) f(std::integral_constant<int, 2>());
  else if (E <= 128) f(std::integral_constant<int, 4>());
  else if (E <= 256) f(std::integral_constant<int, 8>());
  else if (kMaxE <= 512 || E <= 512) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 32>());
}

// A token's logits, lane l the experts l L .. l L + L - 1 (32 L >= E).
template <int L, bool kBf16>
__device__ __forceinline__ void load_logits(const RouteRule& r, int64_t token, float (&v)[L]) {
  const int first = (threadIdx.x & 31) * L;
  const int64_t base = token * r.E + first;
  if (L % 4 == 0 && r.E % 4 == 0) {  // rows and lanes start on four logits
#pragma unroll
    for (int i = 0; i < L; i += 4) {
      float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (first + i < r.E) {
        if constexpr (kBf16) {
          const uint2 w = __ldcg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(r.logits) + base + i));
          x = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
        } else {
          x = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(r.logits) + base + i));
        }
      }
      v[i] = x.x;
      if constexpr (L % 4 == 0) {
        v[i + 1] = x.y;
        v[i + 2] = x.z;
        v[i + 3] = x.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      v[i] = -INFINITY;
      if (first + i < r.E)
        v[i] = kBf16 ? bf16lo(__ldcg(static_cast<const unsigned short*>(r.logits) + base + i))
                     : __ldcg(static_cast<const float*>(r.logits) + base + i);
    }
  }
}

// One warp, one token: returns this lane's choice (j = lane < k) and its weight, from the
// logits of load_logits.  `ids`: 32 words of shared memory of the warp's own.
//   softmax: exp(l_j - max) / sum, over all E or (renorm) the chosen
//   sigmoid: 1 / (1 + exp(-l_j)), divided (renorm) by the sum of the chosen
// in FP32 with the hardware's exponential and division: (2 + |x|) 2^-22 of exp(x), the rounding of
// its argument, and 2^-22 of a quotient are lost, where a chain of correctly rounded steps would
// lose some 2^-23 (one token of 128: 5.6e-8 against 4.0e-8 from 64 bits).
// A logit of -infinity has weight zero, also where all are -infinity (a sigmoid
// below 2^-126 is zero too).  A NaN logit makes the weights of its token NaN where
// it is chosen or enters the sum, one of +infinity those of a softmax.
// A round is a chain of steps that wait for one another (the lane's maximum, the warp's,
// the removal: 92 cycles at L = 4).  kPacked (bf16 logits): the key's upper half is the
// logit, the lower the expert, higher for a lower index, so keys differ and say which
// expert they are.  Else (fp32) a round takes every expert of the largest key; where that
// took more than k in the end, or left the last round nothing, some were equal and the
// rounds run once more, one expert a round, the lowest of the lowest lane.
// The code is kept short: a kernel of a few microseconds reads it once, from L2 (four
// tokens to a warp, eight lanes each, in four times the instructions, took as long).
template <int L, bool kPacked>
__device__ __forceinline__ void choose_experts(const RouteRule& r, int64_t token, const float (&v)[L], int* ids,
                                               int& expert, float& weight) {
  const int lane = threadIdx.x & 31, first = lane * L;
  uint32_t key[L];
  auto make_keys = [&] {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      uint32_t u = logit_key(v[i]);
      if constexpr (kPacked) u = (u & 0xFFFF0000u) | static_cast<uint32_t>(0xFFFF - (first + i));
      key[i] = first + i < r.E ? u : 0u;
    }
  };
  auto local_max = [&] {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < L; ++i) m = max(m, key[i]);
    return m;
  };
  make_keys();
  float any = v[0];
#pragma unroll
  for (int i = 1; i < L; ++i) any += v[i];
  const bool nan = __any_sync(0xffffffffu, isnan(any));  // a NaN (or infinities of both signs: no harm)
  uint32_t mine = 0u, m = 0u;  // the keys of this lane's choice and of the round's
#pragma unroll 1
  for (int j = 0; j < r.k; ++j) {
    m = __reduce_max_sync(0xffffffffu, local_max());
    mine = lane == j ? m : mine;
    if constexpr (kPacked) {
#pragma unroll
      for (int i = 0; i < L; ++i) key[i] = key[i] == m ? 0u : key[i];
    } else {
      int hit = -1;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const bool take = key[i] == m;
        hit = take ? first + i : hit;
        key[i] = take ? 0u : key[i];
      }
      if (hit >= 0) ids[j] = hit;
    }
  }
  if constexpr (kPacked) {
    expert = lane < r.k ? 0xFFFF - static_cast<int>(mine & 0xFFFFu) : 0;
    // the logit's key again: the bits below bf16 are those of a value whose low half is zero
    mine = (mine & 0x80000000u) ? mine & 0xFFFF0000u : mine | 0xFFFFu;
  } else {
    uint32_t taken = 0u;  // how many of this lane's experts are gone
#pragma unroll
    for (int i = 0; i < L; ++i) taken += key[i] == 0u && first + i < r.E ? 1u : 0u;
    if (__reduce_add_sync(0xffffffffu, taken) != static_cast<uint32_t>(r.k) || m == 0u) {
      make_keys();
#pragma unroll 1
      for (int j = 0; j < r.k; ++j) {
        const uint32_t best = local_max();
        m = __reduce_max_sync(0xffffffffu, best);
        mine = lane == j ? m : mine;
        bool own = lane == __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
#pragma unroll
        for (int i = 0; i < L; ++i) {
          if (own && key[i] == m) {
            ids[j] = first + i;
            key[i] = 0u;
            own = false;
          }
        }
      }
    }
    __syncwarp();
    expert = lane < r.k ? ids[lane] : 0;
  }
  float l = key_logit(mine);
  const float mx = __shfl_sync(0xffffffffu, l, 0);
  if (nan && lane < r.k) l = load_logit(r, token * r.E + expert);  // a NaN's key says -infinity
  const float e = __expf(r.sigmoid ? -l : l - mx);
  weight = r.sigmoid ? __fdividef(1.0f, 1.0f + e) : e;
  weight = lane >= r.k || l == -INFINITY ? 0.f : weight;  // also where the largest logit is -infinity itself
  if (r.renorm || !r.sigmoid) {
    float sum = weight;
    if (!r.renorm) {
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < L; ++i) sum += v[i] == -INFINITY ? 0.f : __expf(v[i] - mx);
    }
    sum = warp_sum(sum);
    weight = sum == 0.f ? 0.f : __fdividef(weight, sum);
  }
  weight *= r.scale;
  __syncwarp();  // `ids` may be written again
}

// A warp's tokens t0, t0 + step, ... below t1, the next one's logits loaded (700 cycles
// from L2) before the choice for this one: f(token, expert, weight), choice j in lane j < k.
template <int L, bool kPacked, typename F>
__device__ __forceinline__ void choose_all(const RouteRule& r, int64_t t0, int64_t t1, int step, int* ids, F&& f) {
  float v[L], next[L];
  if (t0 < t1) load_logits<L, kPacked>(r, t0, v);
#pragma unroll 1
  for (int64_t t = t0; t < t1; t += step) {
    load_logits<L, kPacked>(r, min(t + step, t1 - 1), next);
    int e;
    float w;
    choose_experts<L, kPacked>(r, t, v, ids, e, w);
    f(t, e, w);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < L; ++i) v[i] = next[i];
  }
}
template <int kMaxE, typename F>
__device__ __forceinline__ void choose_all(const RouteRule& r, int64_t t0, int64_t t1, int step, int* ids, F&& f) {
  for_keys_per_lane<kMaxE>(r.E, [&](auto keys) {
    constexpr int L = decltype(keys)::value;
    if (r.logits_f32) choose_all<L, false>(r, t0, t1, step, ids, f);
    else choose_all<L, true>(r, t0, t1, step, ids, f);
  });
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
// Measured on the GPU, experts x choices: one token of 128 x 8 2.9 us, 1001 of 60 x 4
// (fp32) 7.0, 8192 of 128 x 8 12.7 (0.23 TB/s; choosing alone 5.9), 8192 of 512 x 10
// (fp32) 29.5: chains of dependent steps and two launches bound it, not bytes.
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
  int32_t* hist;     // [gridDim.x, hist_stride(E)] (more than one CTA)
};
// Counts of a CTA: whole vectors of four experts.
__host__ __device__ constexpr int hist_stride(int E) { return (E + 3) / 4 * 4; }

struct RouteTables {
  int base[kRouteMaxE];                  // row that the next choice of expert e gets
  uint2 picked[kRouteMaxE];              // tokens of this run that picked e, a bit each
  int warp_total[kRouteThreads / 32];
};

// base[e] (0 <= e < E, counts on entry) becomes the sum of the counts before e, plus add[e].
__device__ __forceinline__ void exclusive_prefix(RouteTables& s, int E, const int* add) {
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
#pragma unroll
    for (int w = 0; w < kRouteThreads / 32; ++w) {
      before += w < warp ? s.warp_total[w] : 0;
      total += s.warp_total[w];
    }
    if (e < E) s.base[e] = before + inc - c + (add != nullptr ? add[e] : 0);
    carry += total;
    __syncthreads();
  }
}

// Places the choices of tokens [t0, t1), base[] holding the first free row of each expert
// and picked[] zeros; `mine` is the expert of this thread's choice of the first run.
__device__ __forceinline__ void place_choices(const RouteParams& p, RouteTables& s, int64_t t0, int64_t t1, int mine) {
  const int k = p.rule.k, E = p.rule.E;
  for (int64_t r0 = t0; r0 < t1; r0 += kRouteRun) {
    const int n = static_cast<int>(min(static_cast<int64_t>(kRouteRun), t1 - r0)) * k;
    const int32_t* run = p.ids + r0 * k;
    auto expert = [&](int i) { return r0 == t0 && i < kRouteThreads ? mine : run[i]; };
    for (int i = threadIdx.x; i < n; i += kRouteThreads) {
      const int t = i / k;
      atomicOr(t < 32 ? &s.picked[expert(i)].x : &s.picked[expert(i)].y, 1u << (t & 31));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kRouteThreads) {
      const int e = expert(i), t = i / k;
      const uint2 picked = s.picked[e];
      const uint32_t below = (1u << (t & 31)) - 1;
      p.order[s.base[e] + (t < 32 ? __popc(picked.x & below) : __popc(picked.x) + __popc(picked.y & below))] =
          static_cast<int32_t>(r0 * k + i);
    }
    if (r0 + kRouteRun >= t1) break;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      s.base[e] += __popc(s.picked[e].x) + __popc(s.picked[e].y);
      s.picked[e] = make_uint2(0u, 0u);
    }
    __syncthreads();
  }
}
// The expert of this thread's choice of the first run of tokens [t0, t1).
__device__ __forceinline__ int first_choice(const RouteParams& p, int64_t t0, int64_t t1) {
  const int i = static_cast<int>(threadIdx.x);
  return i < min(static_cast<int64_t>(kRouteRun), t1 - t0) * p.rule.k ? p.ids[t0 * p.rule.k + i] : 0;
}

__global__ void __launch_bounds__(kRouteThreads) route_choose_kernel(const __grid_constant__ RouteParams p) {
  __shared__ RouteTables s;
  __shared__ int ids[kRouteThreads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.rule.E, k = p.rule.k;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.per_cta;
  const int64_t t1 = min(p.T, t0 + p.per_cta);
  const bool sorting = p.counts != nullptr;
  if (sorting) {
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
      s.base[e] = 0;
      s.picked[e] = make_uint2(0u, 0u);
    }
    __syncthreads();
  }
  pdl_wait();  // the logits may come from the kernel before
  pdl_trigger();
  choose_all<kRouteMaxE>(p.rule, t0 + warp, t1, kRouteThreads / 32, ids + warp * 32, [&](int64_t t, int e, float w) {
    if (lane < k) {
      p.ids[t * k + lane] = e;
      p.weights[t * k + lane] = w;
      if (sorting) atomicAdd(&s.base[e], 1);
    }
  });
  if (!sorting) return;
  __syncthreads();
  if (gridDim.x > 1) {
    const int stride = hist_stride(E);
    for (int e = threadIdx.x; e < stride; e += kRouteThreads)
      p.hist[static_cast<int64_t>(blockIdx.x) * stride + e] = e < E ? s.base[e] : 0;
    return;
  }
  for (int e = threadIdx.x; e < E; e += kRouteThreads) p.counts[e] = s.base[e];
  __syncthreads();
  exclusive_prefix(s, E, nullptr);
  place_choices(p, s, t0, t1, first_choice(p, t0, t1));
}

__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const __grid_constant__ RouteParams p) {
  __shared__ RouteTables s;
  __shared__ int before[kRouteMaxE];  // choices of expert e in earlier CTAs
  const int E = p.rule.E, nb = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
  for (int e = threadIdx.x; e < E; e += kRouteThreads) {
    s.base[e] = before[e] = 0;
    s.picked[e] = make_uint2(0u, 0u);
  }
  __syncthreads();
  pdl_wait();  // the counts and the choices come from the kernel before
  pdl_trigger();
  const int64_t t0 = static_cast<int64_t>(b) * p.per_cta, t1 = min(p.T, t0 + p.per_cta);
  const int mine = first_choice(p, t0, t1);
  // thread (part, four experts): the CTAs part, part + parts, ..., eight loads in flight; integer sums, any order
  // (with a 4-byte load an expert, four times as many, 8192 tokens of 128 experts took 1.5 us more)
  const int vecs = hist_stride(E) / 4, parts = kRouteThreads / vecs;
  const int part = static_cast<int>(threadIdx.x) / vecs, v = static_cast<int>(threadIdx.x) % vecs;
  if (part < parts) {
    const int4* src = reinterpret_cast<const int4*>(p.hist) + v;
    int4 total = make_int4(0, 0, 0, 0), earlier = total;
    for (int c0 = part; c0 < nb; c0 += 8 * parts) {
      int4 h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + i * parts;
        h[i] = c < nb ? __ldcg(src + static_cast<int64_t>(c) * vecs) : make_int4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int m = c0 + i * parts < b ? -1 : 0;
        total.x += h[i].x; total.y += h[i].y; total.z += h[i].z; total.w += h[i].w;
        earlier.x += h[i].x & m; earlier.y += h[i].y & m; earlier.z += h[i].z & m; earlier.w += h[i].w & m;
      }
    }
    const int t[4] = {total.x, total.y, total.z, total.w}, e[4] = {earlier.x, earlier.y, earlier.z, earlier.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (v * 4 + i < E) {
        atomicAdd(&s.base[v * 4 + i], t[i]);
        atomicAdd(&before[v * 4 + i], e[i]);
      }
    }
  }
  __syncthreads();
  if (b == 0)
    for (int e = threadIdx.x; e < E; e += kRouteThreads) p.counts[e] = s.base[e];
  exclusive_prefix(s, E, before);
  place_choices(p, s, t0, t1, mine);
}

}  // namespace macaq
