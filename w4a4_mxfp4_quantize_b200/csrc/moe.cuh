// A whole mixture-of-experts layer for a few tokens (T <= 128), in two kernels:
//   up:   choose each token's experts from its logits; for every chosen expert e and
//         its tokens  (g, u) = 2^-5 Q(H(x / D1_e)) . W1_e^T,  a = RNE_bf16(act(g) u)
//   down: y[t] = RNE_bf16( sum_e w[t, e] 2^-5 Q(H(a / D2_e)) . W2_e^T )
// Reading the chosen experts' weights once is what the layer costs: 17/32 byte per
// weight, against at most 16 tokens' worth of arithmetic per byte, so everything
// else is arranged around an unbroken stream of weight tiles.
//
// Work: a group is an expert with up to 16 of its tokens (the N of the MMA); an item
// is a group times one 128-row weight tile.  The up kernel deals the items of all
// groups out evenly, in order, so a CTA quantises its tokens for an expert once and
// keeps them in shared memory for all of that expert's tiles it owns.  In the down
// kernel a cluster of S CTAs owns 128 output channels; its CTAs share the groups,
// each adds its own into an FP32 tile, and the S tiles are added in rank order
// through distributed shared memory: no atomics, no partial sums in memory.
//
// Both kernels choose the experts themselves (an integer selection, identical in
// every CTA), so the down kernel needs nothing from the up kernel but the
// activations a: launched as a programmatic dependent, it streams its first weight
// tiles while the up kernel still runs.
//
// Warps: 0 weight copies, 1 MMA, 2 scale copies, 4-7 epilogue, 8-11 activation
// quantiser; all of them choose experts first.
#pragma once
#include "route.cuh"

namespace macaq {

namespace moe {
constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;         // tokens of a group: the MMA's N
constexpr int kMaxTokens = 128;
constexpr int kMaxChoice = 16;
constexpr int kMaxExperts = 512;
constexpr int kMaxK = 8192;
constexpr int kMaxStages = 4;
constexpr int kMaxBufs = 4;
constexpr int kBCodeBytes = kRows * 128;  // codes of one K tile of a group
constexpr int kBSfBytes = 512;            // its scales: two blocks of 16 rows x 16 bytes
constexpr int kStageBytes = kTileCodeBytes + kTileSfBytes;
constexpr int kTmemCols = 128;            // two accumulators of 16 columns, then 16 scale columns a stage
constexpr int kSfCol = 32;
constexpr int kBarBytes = 512;
static_assert(kSfCol + 16 * kMaxStages <= kTmemCols, "tensor memory");

// Shared memory of one CTA, byte offsets from a 1024-byte boundary.
struct Layout {
  int stages, bufs;
  int sf, b, bsf, bar, ent, ent_tok, ent_w, grp, acc, bytes;
};
__host__ __device__ inline int max_groups(int T, int k, int E) {
  return (T * k < E ? T * k : E) + T * k / kRows;
}
__host__ __device__ inline int align16i(int v) { return (v + 15) & ~15; }
// Bytes of the tables that only choosing needs; they lie where the weight stages come later.
__host__ __device__ inline int scratch_bytes(int T, int k, int E) { return align16i(T * k * 6) + E * 20; }
__host__ inline Layout layout(int T, int k, int E, int K, bool down, int stages, int bufs) {
  const int KT = K / kKTile, tk = T * k, G = max_groups(T, k, E);
  Layout l;
  l.stages = stages;
  l.bufs = bufs;
  l.sf = stages * kTileCodeBytes;
  l.b = l.sf + stages * kTileSfBytes;
  l.b = (l.b + 1023) & ~1023;
  l.bsf = l.b + bufs * KT * kBCodeBytes;
  l.bar = l.bsf + bufs * KT * kBSfBytes + 256;  // the last scale copy reads 256 bytes past its rows
  l.ent = l.bar + kBarBytes;
  l.ent_tok = l.ent + align16i(tk * 2);
  l.ent_w = l.ent_tok + align16i(tk * 2);
  l.grp = l.ent_w + align16i(tk * 4);
  l.acc = l.grp + align16i(G * 8);
  l.bytes = l.acc + (down ? T * kRowsTile * 4 : 0) + 1024;
  return l;
}
}  // namespace moe

struct MoeParams {
  RouteRule rule;
  const uint8_t* Wq;     // weight images of this kernel's linear
  const uint8_t* Ws;
  const float* D;        // [E, K]
  const uint16_t* a;     // up: x bf16 [T, K]; down: a bf16 [T k, K]
  uint16_t* out;         // up: a bf16 [T k, N / 2]; down: y bf16 [T, N]
  int T, N, K, NT, KT;
  int gelu;              // up: act is GELU_TANH (else SILU)
  int S;                 // down: CTAs of a cluster
  int team;              // quantiser warps that share a group (1, 2 or 4)
  int32_t* status;
  moe::Layout l;
};

// act(g) u in FP32: SILU g / (1 + exp(-g)), GELU_TANH as g / (1 + exp(-2 z)), the same
// function, z = sqrt(2/pi) (g + 0.044715 g^3).  One exponential and one division each:
// the result is quantised to four bits next, and the half-precision tanh of the linear's
// own epilogue would move one code in some hundreds.
__device__ __forceinline__ float gated(float g, float u, int gelu) {
  const float z = gelu ? 1.5957691216057308f * fmaf(g * g * g, 0.044715f, g) : g;
  return __fdividef(g, 1.0f + __expf(-z)) * u;
}

// Half a 32-element activation block (16 bf16 values, their reciprocals of D) per lane,
// lanes 2 i and 2 i + 1 together: the arithmetic of act_block step by step, its last
// butterfly stage (h = 16) and the block maximum exchanged between the two lanes.
__device__ __forceinline__ void act_half_block(const uint4 (&xv)[2], const float2 (&r2)[8], bool upper, uint2& codes,
                                               uint32_t& scale) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(xv);
  float2 P[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t xs = f2_to_bf16x2(f2_mul(bf16x2_to_f2(w[j]), r2[j]));
    const float v0 = bf16lo(xs), v1 = bf16hi(xs);
    P[j] = f2(__fadd_rn(v0, v1), __fsub_rn(v0, v1));
  }
#pragma unroll
  for (int hp = 1; hp < 8; hp <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i & hp) continue;
      const float2 a = P[i], b = P[i + hp];
      P[i] = f2_add(a, b);
      P[i + hp] = f2_sub(a, b);
    }
  }
  const float sign = upper ? -1.0f : 1.0f;  // lower lane: mine + other, upper lane: other - mine
  const float2 s2 = f2(sign, sign);
  uint32_t u[8];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 o = f2(__shfl_xor_sync(0xffffffffu, P[j].x, 1), __shfl_xor_sync(0xffffffffu, P[j].y, 1));
    u[j] = f2_to_bf16x2(ffma2(P[j], s2, o));  // the product by +-1 is exact: one rounding
    m = max_u16x2(m, u[j] & 0x7FFF7FFFu);
  }
  m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t c = e8m0_from_amax_bits(max(m & 0xFFFFu, m >> 16) << 16);
  const float s = __uint_as_float((254u - min(c, 253u)) << 23);
  const float2 q2 = f2(s, s);
  codes.x = e2m1x8_f2(f2_mul(bf16x2_to_f2(u[0]), q2), f2_mul(bf16x2_to_f2(u[1]), q2),
                      f2_mul(bf16x2_to_f2(u[2]), q2), f2_mul(bf16x2_to_f2(u[3]), q2));
  codes.y = e2m1x8_f2(f2_mul(bf16x2_to_f2(u[4]), q2), f2_mul(bf16x2_to_f2(u[5]), q2),
                      f2_mul(bf16x2_to_f2(u[6]), q2), f2_mul(bf16x2_to_f2(u[7]), q2));
  scale = c;
}

// The groups of the call, from the logits (every CTA computes the same): ent[] lists the
// (token, choice) pairs t k + j by expert, then by token; a group is a run of at most
// 16 of them of one expert, grp = {first entry, expert | rows << 16}.  A pair of weight
// zero is left out: it adds nothing and its expert need not be read.  Returns the number
// of groups.  `scratch` overlaps the weight stages.
__device__ __forceinline__ int moe_groups(const MoeParams& p, uint8_t* smem, uint8_t* scratch, int* n_groups) {
  const int k = p.rule.k, E = p.rule.E, T = p.T, tk = T * k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* sel_w = reinterpret_cast<float*>(scratch);
  uint16_t* sel_e = reinterpret_cast<uint16_t*>(sel_w + tk);
  uint32_t* mask = reinterpret_cast<uint32_t*>(scratch + moe::align16i(tk * 6));  // [E][4]: tokens that chose e
  int* off = reinterpret_cast<int*>(mask + E * 4);                                // [E]: first entry
  uint16_t* ent = reinterpret_cast<uint16_t*>(smem + p.l.ent);
  uint16_t* ent_tok = reinterpret_cast<uint16_t*>(smem + p.l.ent_tok);
  float* ent_w = reinterpret_cast<float*>(smem + p.l.ent_w);
  int2* grp = reinterpret_cast<int2*>(smem + p.l.grp);
  for (int i = threadIdx.x; i < E * 4; i += moe::kThreads) mask[i] = 0u;
  __syncthreads();
  for_keys_per_lane(E, [&](auto keys) {
    if constexpr (decltype(keys)::value <= moe::kMaxExperts / 32) {
      for (int t = warp; t < T; t += moe::kWarps) {
        int e;
        float w;
        choose_experts<decltype(keys)::value>(p.rule, t, e, w);
        if (lane < k) {
          const bool used = w != 0.f;
          sel_w[t * k + lane] = w;
          sel_e[t * k + lane] = used ? static_cast<uint16_t>(e) : 0xFFFFu;
          if (used) atomicOr(&mask[e * 4 + (t >> 5)], 1u << (t & 31));
        }
      }
    }
  });
  __syncthreads();
  if (warp == 0) {  // entries and groups before each expert
    int ent_base = 0, grp_base = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      int c = 0;
      if (e < E) {
        const uint4 m = *reinterpret_cast<const uint4*>(mask + e * 4);
        c = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
      }
      const int g = (c + moe::kRows - 1) / moe::kRows;
      int both = c | (g << 16);  // at most 2048 entries and 128 + E groups: both sums stay below 2^15
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, both, o);
        if (lane >= o) both += u;
      }
      const int c0 = ent_base + (both & 0xFFFF) - c, g0 = grp_base + (both >> 16) - g;
      if (e < E) off[e] = c0;
      for (int i = 0; i < g; ++i)
        grp[g0 + i] = make_int2(c0 + i * moe::kRows, e | (min(moe::kRows, c - i * moe::kRows) << 16));
      const int total = __shfl_sync(0xffffffffu, both, 31);
      ent_base += total & 0xFFFF;
      grp_base += total >> 16;
    }
    if (lane == 0) *n_groups = grp_base;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tk; i += moe::kThreads) {
    const int e = sel_e[i];
    if (e != 0xFFFF) {
      const int t = i / k;
      int r = off[e] + __popc(mask[e * 4 + (t >> 5)] & ((1u << (t & 31)) - 1));
      for (int w = 0; w < (t >> 5); ++w) r += __popc(mask[e * 4 + w]);
      ent[r] = static_cast<uint16_t>(i);
      ent_tok[r] = static_cast<uint16_t>(t);
      ent_w[r] = sel_w[i];
    }
  }
  fence_proxy_async_smem();  // the stages' copies will overwrite the scratch
  __syncthreads();
  return *n_groups;
}

template <bool kDown>
__global__ void __launch_bounds__(moe::kThreads, 2) moe_kernel(const __grid_constant__ MoeParams p) {
  using namespace moe;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.l.bar);
  uint64_t* empty = full + kMaxStages;
  uint64_t* sfull = empty + kMaxStages;
  uint64_t* bfull = sfull + kMaxStages;   // a group's quantised tokens are in shared memory
  uint64_t* bempty = bfull + kMaxBufs;
  uint64_t* accf = bempty + kMaxBufs;     // [2]
  uint64_t* acce = accf + 2;              // [2]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acce + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* epi_ok = abort_flag + 1;  // [4], one per epilogue warp
  int* n_groups = reinterpret_cast<int*>(const_cast<int*>(epi_ok) + 4);
  const uint16_t* ent = reinterpret_cast<const uint16_t*>(smem + p.l.ent);
  const uint16_t* ent_tok = reinterpret_cast<const uint16_t*>(smem + p.l.ent_tok);
  const float* ent_w = reinterpret_cast<const float*>(smem + p.l.ent_w);
  const int2* grp = reinterpret_cast<const int2*>(smem + p.l.grp);
  float* acc = reinterpret_cast<float*>(smem + p.l.acc);  // down: [T][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.l.stages, bufs = p.l.bufs;

  if (warp == 1) {
    tmem_alloc(tmem_holder, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], 1);
    }
    for (int b = 0; b < kMaxBufs; ++b) {
      mbar_init(&bfull[b], p.team);
      mbar_init(&bempty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if constexpr (!kDown) {
    pdl_wait();     // x and the logits may come from the kernel before
    pdl_trigger();  // the down kernel may start: what it reads before its own wait is complete
  }
  tc_fence_before();
  const int G = moe_groups(p, smem, smem, n_groups);
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int KT = p.KT;
  // this CTA's items [i0, i1): up: item = group NT + tile; down: item = group, the tile is the cluster's
  const int rank = kDown ? static_cast<int>(cluster_ctarank()) : 0;
  const int total = kDown ? G : G * p.NT;
  const int share = kDown ? rank : static_cast<int>(blockIdx.x), shares = kDown ? p.S : static_cast<int>(gridDim.x);
  const int i0 = static_cast<int>(static_cast<int64_t>(total) * share / shares);
  const int i1 = static_cast<int>(static_cast<int64_t>(total) * (share + 1) / shares);
  const int tile0 = kDown ? static_cast<int>(blockIdx.x) / p.S : 0;
  auto group_of = [&](int i) { return kDown ? i : i / p.NT; };
  auto tile_of = [&](int i) { return kDown ? tile0 : i % p.NT; };
  const int g0 = group_of(i0), g1 = i1 > i0 ? group_of(i1 - 1) + 1 : g0;  // this CTA's groups

  if (warp == 0) {
    // ---- producer: lane 0 copies a stage's weight codes, lane 1 its scales ----
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = i0; i < i1 && ok; ++i) {
      const int e = grp[group_of(i)].y & 0xFFFF;
      const size_t img = weight_image(e, tile_of(i), 0, p.NT / 2, KT);
      const uint8_t* src = (lane & 1) ? p.Ws + img * kTileSfBytes : p.Wq + img * kTileCodeBytes;
      const uint32_t bytes = (lane & 1) ? kTileSfBytes : kTileCodeBytes;
      uint8_t* dst0 = (lane & 1) ? smem + p.l.sf : smem;
      for (int kt = 0; kt < KT; ++kt) {
        int got = 1;
        if (lane == 0) {
          got = mbar_wait(&empty[stage], phase ^ 1, abort_flag, kWaitTimeoutNs) ? 1 : 0;
          if (got) mbar_arrive_expect_tx(&full[stage], kStageBytes);
        }
        __syncwarp();  // the stage is free for both lanes
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          ok = false;
          break;
        }
        bulk_g2s_if(lane < 2, dst0 + stage * bytes, src, bytes, &full[stage]);
        src += 2 * bytes;  // the next K tile's image pair
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    if (lane == 0) {
      const uint32_t idesc_lo = idesc_mxf4(128, kRows, 0, 0), idesc_hi = idesc_mxf4(128, kRows, 2, 2);
      const uint64_t a0 = sdesc_kmajor_sw128(smem_u32(smem)), b0 = sdesc_kmajor_sw128(smem_u32(smem + p.l.b));
      int stage = 0, g = -1, buf = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = i0; i < i1 && ok; ++i) {
        const int ab = (i - i0) & 1;
        if (group_of(i) != g) {
          g = group_of(i);
          buf = (g - g0) % bufs;
          if (!mbar_wait(&bfull[buf], ((g - g0) / bufs) & 1, abort_flag, kWaitTimeoutNs)) break;
        }
        if (!mbar_wait(&acce[ab], (((i - i0) >> 1) & 1) ^ 1, abort_flag, kWaitTimeoutNs)) break;
        tc_fence_after();
        for (int kt = 0; kt < KT; ++kt) {
          if (!mbar_wait(&full[stage], phase, abort_flag, kWaitTimeoutNs) ||
              !mbar_wait(&sfull[stage], phase, abort_flag, kWaitTimeoutNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sf = tmem + kSfCol + 16 * stage;
          mma_stage(a0 + (static_cast<uint32_t>(stage * kTileCodeBytes) >> 4),
                    b0 + (static_cast<uint32_t>((buf * KT + kt) * kBCodeBytes) >> 4), sf, sf + 8, tmem + ab * kRows,
                    idesc_lo, idesc_hi, kt == 0);
          tc_commit(&empty[stage]);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        tc_commit(&accf[ab]);
        if (i + 1 == i1 || group_of(i + 1) != g) tc_commit(&bempty[buf]);
      }
    }
  } else if (warp == 2) {
    // ---- scale copies of a stage into its TMEM slot: weights 8 columns, tokens 8 columns ----
    if (lane == 0) {
      const uint64_t sfa0 = sdesc_sf_block(smem_u32(smem + p.l.sf)), sfb0 = sdesc_sf_block(smem_u32(smem + p.l.bsf));
      int stage = 0, g = -1, buf = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = i0; i < i1 && ok; ++i) {
        if (group_of(i) != g) {
          g = group_of(i);
          buf = (g - g0) % bufs;
          if (!mbar_wait(&bfull[buf], ((g - g0) / bufs) & 1, abort_flag, kWaitTimeoutNs)) break;
        }
        for (int kt = 0; kt < KT; ++kt) {
          if (!mbar_wait(&full[stage], phase, abort_flag, kWaitTimeoutNs)) {
            ok = false;
            break;
          }
          const uint32_t sf = tmem + kSfCol + 16 * stage;
          const uint64_t sa = sfa0 + (static_cast<uint32_t>(stage * kTileSfBytes) >> 4);
          const uint64_t sb = sfb0 + (static_cast<uint32_t>((buf * KT + kt) * kBSfBytes) >> 4);
          tc_cp_32x128b_warpx4(sf, sa);
          tc_cp_32x128b_warpx4(sf + 4, sa + (512 >> 4));
          tc_cp_32x128b_warpx4(sf + 8, sb);
          tc_cp_32x128b_warpx4(sf + 12, sb + (256 >> 4));
          tc_commit(&sfull[stage]);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ---- epilogue: 16 accumulator columns (tokens) of this thread's weight row ----
    const int q = warp & 3, row = q * 32 + lane;
    if constexpr (kDown) {
      for (int t = 0; t < p.T; ++t) acc[t * kRowsTile + row] = 0.f;
    }
    for (int i = i0; i < i1; ++i) {
      const int ab = (i - i0) & 1;
      if (lane == 0) epi_ok[q] = mbar_wait(&accf[ab], ((i - i0) >> 1) & 1, abort_flag, kWaitTimeoutNs) ? 1 : 0;
      __syncwarp();
      if (!epi_ok[q]) break;
      tc_fence_after();
      uint32_t r[kRows];
      tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + ab * kRows, r);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce[ab]);
      const int2 gr = grp[group_of(i)];
      const int first = gr.x, rows = gr.y >> 16;
      if constexpr (kDown) {
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          if (j < rows) {
            float* o = acc + ent_tok[first + j] * kRowsTile + row;
            *o = fmaf(ent_w[first + j] * 0.03125f, __uint_as_float(r[j]), *o);
          }
        }
      } else {
        // weight rows 2 c and 2 c + 1 are the gate and the up row of channel c: of two tokens
        // the even lane finishes the first, the odd lane the second
        const bool odd = lane & 1;
        const int64_t half = p.N / 2;
        uint16_t* o = p.out + (tile_of(i) * kRowsTile + row) / 2;
#pragma unroll
        for (int j = 0; j < kRows; j += 2) {
          if (j < rows) {
            const float a = __uint_as_float(r[j]) * 0.03125f, b = __uint_as_float(r[j + 1]) * 0.03125f;
            const float other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
            const float h = gated(odd ? other : a, odd ? b : other, p.gelu);
            const int jj = j + (odd ? 1 : 0);
            if (jj < rows) o[ent[first + jj] * half] = bf16_bits(h);
          }
        }
      }
    }
  } else if (warp >= 8) {
    // ---- activation quantiser: team m of `team` warps takes this CTA's groups m, m + teams, ... ----
    if constexpr (kDown) {
      pdl_wait();  // the activations come from the up kernel
      pdl_trigger();
    }
    const int team = (warp - 8) / p.team, teams = 4 / p.team;
    const int tt = (warp - 8) % p.team * 32 + lane, TT = p.team * 32;
    const int HB = p.K / 16;  // half blocks of a row, two lanes to a block
    const int split = HB < TT ? TT / HB : 1;  // threads left over take other rows
    const int rs = HB < TT ? tt / HB : 0, hb0 = HB < TT ? tt % HB : tt;
    const bool upper = lane & 1;
    for (int g = g0 + team; g < g1; g += teams) {
      const int buf = (g - g0) % bufs;
      int ok = 1;
      if (lane == 0) ok = mbar_wait(&bempty[buf], (((g - g0) / bufs) & 1) ^ 1, abort_flag, kWaitTimeoutNs) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      const int2 gr = grp[g];
      const int first = gr.x, e = gr.y & 0xFFFF, rows = gr.y >> 16;
      uint8_t* bq = smem + p.l.b + buf * KT * kBCodeBytes;
      uint8_t* bs = smem + p.l.bsf + buf * KT * kBSfBytes;
      for (int hb = hb0; hb - hb0 < HB; hb += TT) {  // the same number of turns for every lane
        const bool in = hb < HB && rs < split;
        float2 r2[8] = {};
        if (in) {
          const float4* d = reinterpret_cast<const float4*>(p.D + static_cast<int64_t>(e) * p.K + hb * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 v = __ldg(d + j);
            r2[2 * j] = f2(__frcp_rn(v.x), __frcp_rn(v.y));
            r2[2 * j + 1] = f2(__frcp_rn(v.z), __frcp_rn(v.w));
          }
        }
        const int kt = hb >> 4, c = (hb >> 1) & 7;
        for (int j0 = 0; j0 < rows; j0 += 2 * split) {  // two rows in flight
          uint4 xv[2][2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int j = j0 + n * split + rs;
            xv[n][0] = xv[n][1] = make_uint4(0, 0, 0, 0);
            if (in && j < rows) {
              const int64_t src = kDown ? ent[first + j] : ent_tok[first + j];
              const uint4* s = reinterpret_cast<const uint4*>(p.a + src * p.K + hb * 16);
              xv[n][0] = s[0];
              xv[n][1] = s[1];
            }
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int j = j0 + n * split + rs;
            uint2 codes;
            uint32_t scale;
            act_half_block(xv[n], r2, upper, codes, scale);
            if (in && j < rows) {
              *reinterpret_cast<uint2*>(bq + kt * kBCodeBytes + code_chunk_offset(j, c) + (upper ? 8 : 0)) = codes;
              if (!upper) bs[kt * kBSfBytes + (c >> 2) * 256 + j * 16 + (c & 3)] = static_cast<uint8_t>(scale);
            }
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bfull[buf]);
    }
  }
  __syncwarp();

  if constexpr (kDown) {
    // ---- sum of the cluster's tiles in rank order: task (token, 8 channels), dealt out to the ranks ----
    pdl_wait();  // y may still be read by an earlier kernel
    __syncthreads();
    cluster_sync_all();  // every CTA's tile is complete
    const uint32_t local = smem_u32(acc);
    for (int task = static_cast<int>(threadIdx.x) * p.S + rank; task < p.T * 16; task += kThreads * p.S) {
      const int t = task >> 4, c = (task & 15) * 8;
      float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int o = 0; o < p.S; ++o) {
        const uint32_t at = mapa_shared(local + static_cast<uint32_t>((t * kRowsTile + c) * 4), static_cast<uint32_t>(o));
        const float4 a = ld_dsmem_f32x4(at), b = ld_dsmem_f32x4(at + 16);
        s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
        s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
      }
      *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(t) * p.N + tile0 * kRowsTile + c) =
          make_uint4(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7]));
    }
    cluster_sync_all();  // no CTA leaves while another may still read its tile
  }
  if (*abort_flag && threadIdx.x == 0 && p.status) *p.status = MACAQ_ERR_DEVICE_TIMEOUT;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace macaq
