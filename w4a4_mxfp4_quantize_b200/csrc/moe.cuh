// A whole mixture-of-experts layer for a few tokens (T <= 128), in two kernels:
//   up:   choose each token's experts from its logits; for every chosen expert e and
//         its tokens  (g, u) = 2^-5 Q(H(x / D1_e)) . W1_e^T,  a = RNE_bf16(act(g) u),
//         stored as the MXFP4 operand Q(H(a / D2_e)) of the second linear
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
// each adds its own into an FP32 tile, and the S tiles are added in a fixed order
// through distributed shared memory: no atomics, no partial sums in memory.
//
// The experts are chosen from the logits, an integer selection that is identical in
// every CTA.  With few choices (T k <= 32) both kernels choose for themselves: a CTA of
// each fits on an SM, and the down kernel, a programmatic dependent, streams its first
// weight tiles while the up kernel still runs.  With more, clusters of the up kernel
// share the choosing and its first CTA writes the groups' tables to the workspace.  In
// both cases the up kernel copies weights to L2 while it chooses, and behind its own the
// down kernel's first.  The activations are quantised where they are made: in the down
// kernel every one of its N / 128 tiles would do it again.
//
// Measured with 128 experts, 8 a token, H = 2048, I = 768, in a captured graph: 1 token
// 16.4 us, 16 tokens 46.2, 128 tokens 77.1 (calls in a row: 17, 47, 78 to 79).  At 128
// tokens all the experts' weights are read, 321 MB at 4.2 TB/s over the whole.  The up
// kernel's stream keeps the rate of a copy (6.6 TB/s, with what the early copies left in
// L2), the down kernel's 5.6 TB/s on 96 SMs.  Around the streams, in part beside the
// copies to L2, stand choosing (8.7 us), the first group's activations (6), the change of
// kernels with the last items of one and the first of the other (10), the cluster's sum
// (6) and uneven shares.  One token is a chain of latencies: 8 experts' weights are 20 MB,
// 3 us.
//
// Warps: 0 weight copies, 1 MMA, 2 scale copies, 4-7 epilogue; up: 8-15 quantise x;
// down: 3 gathers the activations.  All of them choose experts first.
#pragma once
#include "route.cuh"

namespace macaq {

namespace moe {
constexpr int kUpThreads = 512;
constexpr int kDownThreads = 256;
constexpr int kQuantThreads = 256;  // of the up kernel, from warp 8 on
constexpr int kRows = 16;           // tokens of a group: the MMA's N
constexpr int kMaxTokens = 128;
constexpr int kFewTokens = 32;    // down: up to here the cluster's tiles are added by single loads
constexpr int kMaxChoice = 16;
constexpr int kMaxExperts = 512;
constexpr int kMaxK = 8192;
constexpr int kMaxStages = 8;
constexpr int kMaxBufs = 2;
constexpr int kPrefetch = 8;
constexpr int kBCodeBytes = kRows * 128;  // codes of one K tile of a group
constexpr int kBSfBytes = 512;            // its scales: two blocks of 16 rows x 16 bytes
constexpr int kStageBytes = kTileCodeBytes + kTileSfBytes;
constexpr int kSfCol = 32;                // tensor memory: two accumulators of 16 columns, then 16 scale columns a stage
constexpr int kBarBytes = 512;
constexpr int kChunk = kQuantThreads * 8;  // up: channels that the quantiser takes at a time
// up: an item's activations, 16 tokens x 64 channels of bf16, rows 144 bytes apart
constexpr int kActStride = 72;
constexpr int kActBytes = kRows * kActStride * 2;
// Columns to allocate.  An allocation waits until the SM has them free, and the CTAs of a cluster wait
// for one another, so whatever may be resident together (three CTAs of the down kernel from three
// streams, one of each kernel) has to fit in the 512: 3 x 128, 128 + 256.  More than 6 stages are never
// on an SM with a second CTA of as many: they take more than half of its shared memory.
__device__ __forceinline__ int tmem_cols(int stages) { return kSfCol + 16 * stages <= 128 ? 128 : 256; }
static_assert(kSfCol + 16 * kMaxStages <= 256, "tensor memory");

// Shared memory of one CTA, byte offsets from a 1024-byte boundary.
struct Layout {
  int stages, bufs;
  int sf, b, bsf, bar, ent, ent_tok, ent_w, grp, extra, bytes;
};
__host__ __device__ inline int max_groups(int T, int k, int E) {
  return (T * k < E ? T * k : E) + T * k / kRows;
}
__host__ __device__ inline int align16i(int v) { return (v + 15) & ~15; }
// Bytes of the tables that only choosing needs; they lie where the weight stages come later.
__host__ __device__ inline int scratch_bytes(int T, int k, int E) { return align16i(T * k * 8) + E * 20 + kUpThreads * 4; }
__host__ inline Layout layout(int T, int k, int E, int K, bool down, int stages, int bufs) {
  const int KT = K / kKTile, tk = T * k, G = max_groups(T, k, E);
  Layout l;
  l.stages = stages;
  l.bufs = bufs;
  l.sf = stages * kTileCodeBytes;
  l.b = (l.sf + stages * kTileSfBytes + 1023) & ~1023;
  l.bsf = l.b + bufs * KT * kBCodeBytes;
  l.bar = l.bsf + bufs * KT * kBSfBytes + 256;  // the last scale copy reads 256 bytes past its rows
  l.ent = l.bar + kBarBytes;
  l.ent_tok = l.ent + align16i(tk * 2);
  l.ent_w = l.ent_tok + align16i(tk * 2);
  l.grp = l.ent_w + align16i(tk * 4);
  l.extra = l.grp + align16i(G * 8);  // down: the FP32 tile; up: activations
  l.bytes = l.extra + (down ? T * kRowsTile * 4 : 2 * kActBytes) + 1024;
  return l;
}
}  // namespace moe

struct MoeParams {
  RouteRule rule;
  const uint8_t* Wq;     // weight images of this kernel's linear
  const uint8_t* Ws;
  const float* D;        // up: [E, K]
  const float* D_next;   // up: the second linear's [E, N / 2]
  const uint16_t* x;     // up: bf16 [T, K]
  uint8_t* codes;        // the activations' MXFP4 codes [T k, I / 2]: up writes them, down reads them
  uint8_t* scales;       // and scales [T k, I / 32]
  uint16_t* y;           // down: bf16 [T, N]
  int T, N, K, NT, KT;
  int gelu;              // up: act is GELU_TANH (else SILU)
  uint8_t* tables;       // the groups' tables, copied from the up kernel's first CTA (nullptr: the down
                         // kernel chooses for itself, while the up kernel runs)
  int S;                 // CTAs of a cluster (up: those that share the choosing)
  // up: K tiles' weight images that a CTA has copied to L2, of its own linear while the experts are chosen
  // and of the down kernel's, whose shape follows, behind its own: the memory works where it would wait
  int early, ahead;
  const uint8_t* Wq_next;
  const uint8_t* Ws_next;
  int NT_next, KT_next, S_next;
  int32_t* status;
  moe::Layout l;
};

// act(g) u in FP32: SILU g / (1 + exp(-g)), GELU_TANH as g / (1 + exp(-2 z)), the same
// function, z = sqrt(2/pi) (g + 0.044715 g^3).  One exponential and one division each, the
// hardware's: within (4 + 2 |z|) 2^-22 of the value, and zero where z < -87.  The result is
// quantised to four bits next; the half-precision tanh of the linear's own epilogue would
// move one code in some hundreds.
__device__ __forceinline__ float gated(float g, float u, int gelu) {
  const float z = gelu ? 1.5957691216057308f * fmaf(g * g * g, 0.044715f, g) : g;
  return __fdividef(g, 1.0f + __expf(-z)) * u;
}

// bar.sync over `n` threads that also tells them whether all of them passed true.
__device__ __forceinline__ bool named_bar_all(uint32_t id, uint32_t n, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float block_scale(uint32_t c) { return __uint_as_float((254u - min(c, 253u)) << 23); }

// A quarter of a 32-element activation block (8 bf16 values, their reciprocals of D) per
// lane, four lanes to a block: the arithmetic of act_block step by step, its last two
// butterfly stages (h = 8, 16) and the block maximum exchanged between the lanes.
__device__ __forceinline__ void act_quarter_block(const uint4& xv, const float2 (&r2)[4], uint32_t& codes,
                                                  uint32_t& scale) {
  const int lane = threadIdx.x & 31;
  const uint32_t w[4] = {xv.x, xv.y, xv.z, xv.w};
  float2 P[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t xs = f2_to_bf16x2(f2_mul(bf16x2_to_f2(w[j]), r2[j]));
    const float v0 = bf16lo(xs), v1 = bf16hi(xs);
    P[j] = f2(__fadd_rn(v0, v1), __fsub_rn(v0, v1));
  }
#pragma unroll
  for (int hp = 1; hp < 4; hp <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & hp) continue;
      const float2 a = P[i], b = P[i + hp];
      P[i] = f2_add(a, b);
      P[i + hp] = f2_sub(a, b);
    }
  }
#pragma unroll
  for (int h = 1; h < 4; h <<= 1) {
    // lower lane: mine + other, upper lane: other - mine; the product by +-1 is exact: one rounding
    const float sign = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      P[j] = ffma2(P[j], f2(sign, sign),
                   f2(__shfl_xor_sync(0xffffffffu, P[j].x, h), __shfl_xor_sync(0xffffffffu, P[j].y, h)));
  }
  uint32_t u[4], m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    u[j] = f2_to_bf16x2(P[j]);
    m = max_u16x2(m, u[j] & 0x7FFF7FFFu);
  }
  m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  scale = e8m0_from_amax_bits(max(m & 0xFFFFu, m >> 16) << 16);
  const float2 q2 = f2(block_scale(scale), block_scale(scale));
  codes = e2m1x8_f2(f2_mul(bf16x2_to_f2(u[0]), q2), f2_mul(bf16x2_to_f2(u[1]), q2), f2_mul(bf16x2_to_f2(u[2]), q2),
                    f2_mul(bf16x2_to_f2(u[3]), q2));
}

// One 32-element block per warp, element `lane` of R rows: the same steps with every
// butterfly stage an exchange between lanes.  The even lanes receive the byte of codes of
// elements lane and lane + 1.
template <int R>
__device__ __forceinline__ void act_lane_blocks(const float (&x)[R], float r, uint32_t (&byte)[R], uint32_t (&scale)[R]) {
  const int lane = threadIdx.x & 31;
  float v[R];
#pragma unroll
  for (int n = 0; n < R; ++n) v[n] = __bfloat162float(__float2bfloat16_rn(__fmul_rn(x[n], r)));
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const float sign = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
    for (int n = 0; n < R; ++n) v[n] = __fmaf_rn(v[n], sign, __shfl_xor_sync(0xffffffffu, v[n], h));
  }
#pragma unroll
  for (int n = 0; n < R; ++n) {
    const float u = __bfloat162float(__float2bfloat16_rn(v[n]));
    const uint32_t c = e8m0_from_amax_bits(__reduce_max_sync(0xffffffffu, __float_as_uint(u) & 0x7FFFFFFFu));
    const float q = __fmul_rn(u, block_scale(c));
    byte[n] = e2m1x2(q, __shfl_xor_sync(0xffffffffu, q, 1));
    scale[n] = c;
  }
}

// A load that is issued where it stands, before the barrier that lets the weights follow.
__device__ __forceinline__ float4 ld_now(const float* p) {
  float4 v;
  asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The groups of the call, from the logits (every CTA computes the same): ent[] lists the
// (token, choice) pairs t k + j by expert, then by token; a group is a run of at most
// 16 of them of one expert, grp = {first entry, expert | rows << 16}.  A pair of weight
// zero is left out: it adds nothing and its expert need not be read.  Returns the number
// of groups.  `scratch` overlaps the weight stages.
template <int kThreads>
__device__ __forceinline__ int moe_groups(const MoeParams& p, uint8_t* smem, uint8_t* scratch, int* warp_total,
                                          int share, int shares) {
  constexpr int kWarps = kThreads / 32;
  const int k = p.rule.k, E = p.rule.E, T = p.T, tk = T * k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* sel_w = reinterpret_cast<float*>(scratch);
  uint32_t* sel_e = reinterpret_cast<uint32_t*>(sel_w + tk);
  uint32_t* mask = reinterpret_cast<uint32_t*>(scratch + moe::align16i(tk * 8));  // [E][4]: tokens that chose e
  int* off = reinterpret_cast<int*>(mask + E * 4);                                // [E]: first entry
  int* ids = off + E;                                                             // [kWarps][32]
  uint16_t* ent = reinterpret_cast<uint16_t*>(smem + p.l.ent);
  uint16_t* ent_tok = reinterpret_cast<uint16_t*>(smem + p.l.ent_tok);
  float* ent_w = reinterpret_cast<float*>(smem + p.l.ent_w);
  int2* grp = reinterpret_cast<int2*>(smem + p.l.grp);
  for (int i = threadIdx.x; i < E * 4; i += kThreads) mask[i] = 0u;
  __syncthreads();
  // the CTAs of a cluster share the tokens, and each writes its choices to all of them
  if (shares > 1) cluster_wait_acquire();  // the others run
  choose_all<moe::kMaxExperts>(p.rule, warp + share * kWarps, T, shares * kWarps, ids + warp * 32, [&](int64_t token, int e, float w) {
    if (lane < k) {
      const int i = static_cast<int>(token) * k + lane;
      const uint32_t ee = w != 0.f ? static_cast<uint32_t>(e) : 0xFFFFu;
      sel_w[i] = w;
      sel_e[i] = ee;
      if (shares > 1) {
        for (int o = 1; o < shares; ++o) {
          const uint32_t other = static_cast<uint32_t>(share + o < shares ? share + o : share + o - shares);
          st_dsmem_b32(mapa_shared(smem_u32(sel_w + i), other), __float_as_uint(w));
          st_dsmem_b32(mapa_shared(smem_u32(sel_e + i), other), ee);
        }
      } else if (ee != 0xFFFFu) {
        atomicOr(&mask[ee * 4 + (token >> 5)], 1u << (token & 31));
      }
    }
  });
  if (shares > 1) {
    cluster_sync_all();
    for (int i = threadIdx.x; i < tk; i += kThreads) {
      const uint32_t e = sel_e[i];
      const int t = i / k;
      if (e != 0xFFFFu) atomicOr(&mask[e * 4 + (t >> 5)], 1u << (t & 31));
    }
  }
  __syncthreads();
  // entries and groups before each expert, one expert per thread
  int ent_base = 0, grp_base = 0;
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    int c = 0;
    if (e < E) {
      const uint4 m = *reinterpret_cast<const uint4*>(mask + e * 4);
      c = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
    }
    const int g = (c + moe::kRows - 1) / moe::kRows;
    int both = c | (g << 16);  // at most 2048 entries and 640 groups: the sums stay apart
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, both, o);
      if (lane >= o) both += u;
    }
    if (lane == 31) warp_total[warp] = both;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int n = warp_total[w];
      before += w < warp ? n : 0;
      total += n;
    }
    both += before;
    const int c0 = ent_base + (both & 0xFFFF) - c, g0 = grp_base + (both >> 16) - g;
    if (e < E) off[e] = c0;
    for (int i = 0; i < g; ++i)
      grp[g0 + i] = make_int2(c0 + i * moe::kRows, e | (min(moe::kRows, c - i * moe::kRows) << 16));
    ent_base += total & 0xFFFF;
    grp_base += total >> 16;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < tk; i += kThreads) {
    const int e = static_cast<int>(sel_e[i]);
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
  return grp_base;
}

// Lanes' part of copying a K tile's weight image to L2: an even one the codes, an odd one the scales.
__device__ __forceinline__ void prefetch_image(const uint8_t* Wq, const uint8_t* Ws, size_t img, int lane) {
  if (lane & 1) l2_prefetch(Ws + img * kTileSfBytes, kTileSfBytes);
  else l2_prefetch(Wq + img * kTileCodeBytes, kTileCodeBytes);
}

// 80 registers: a CTA of each kernel on one SM is (512 + 256) x 80 of its 65536.
template <bool kDown>
__global__ void __maxnreg__(80) moe_kernel(const __grid_constant__ MoeParams p) {
  using namespace moe;
  constexpr int kThreads = kDown ? kDownThreads : kUpThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.l.bar);
  uint64_t* empty = full + kMaxStages;
  uint64_t* sfull = empty + kMaxStages;
  uint64_t* bfull = sfull + kMaxStages;   // a group's quantised tokens are in shared memory
  uint64_t* bempty = bfull + kMaxBufs;
  uint64_t* accf = bempty + kMaxBufs;     // [2]
  uint64_t* acce = accf + 2;              // [2]
  uint64_t* recv = acce + 2;              // down: the other CTAs' rows have landed
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(recv + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* warp_total = const_cast<int*>(abort_flag) + 1;  // [kWarps], while the groups are formed
  const uint16_t* ent = reinterpret_cast<const uint16_t*>(smem + p.l.ent);
  const uint16_t* ent_tok = reinterpret_cast<const uint16_t*>(smem + p.l.ent_tok);
  const float* ent_w = reinterpret_cast<const float*>(smem + p.l.ent_w);
  const int2* grp = reinterpret_cast<const int2*>(smem + p.l.grp);
  float* acc = reinterpret_cast<float*>(smem + p.l.extra);  // down: [T][128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = p.l.stages, bufs = p.l.bufs;

  if (warp == 1) {
    tmem_alloc(tmem_holder, tmem_cols(p.l.stages));
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], 1);
    }
    for (int b = 0; b < kMaxBufs; ++b) {
      mbar_init(&bfull[b], kDown ? 1 : kQuantThreads / 32);
      mbar_init(&bempty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 4);
    }
    mbar_init(recv, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if constexpr (!kDown) {
    __syncwarp();  // lane 0 of warp 0 was away
    if (p.S > 1) cluster_arrive_release();
    if (warp == 0) {
      // the weights that this CTA begins with if every expert is chosen by up to 16 tokens
      const int first = static_cast<int>(static_cast<uint32_t>(p.rule.E * p.NT * blockIdx.x) / gridDim.x) * p.KT;
      for (int i = lane; i < 2 * p.early; i += 32) {
        const int kt = first + i / 2, item = kt / p.KT, e = item / p.NT;
        if (e < p.rule.E)
          prefetch_image(p.Wq, p.Ws, weight_image(e, item - e * p.NT, 0, p.NT / 2, p.KT) + 2 * (kt - item * p.KT), lane);
      }
    }
    pdl_wait();  // x and the logits may come from the kernel before
    // The down kernel may start: what it reads before its own wait is complete.  Warp 1 says so, after
    // its tensor memory is allocated: a CTA of the down kernel may take the rest of it and wait for us.
    if (warp == 1) pdl_trigger();
  }
  tc_fence_before();
  // ent, ent_tok, ent_w and grp are one run of shared memory from l.ent to l.extra, the same in both
  // kernels; the count follows it in the copy
  const int table_words = (p.l.extra - p.l.ent) / 16;
  int G;
  if (kDown && p.tables != nullptr) {
    pdl_wait();
    const uint4* src = reinterpret_cast<const uint4*>(p.tables);
    for (int i = threadIdx.x; i < table_words; i += kThreads) reinterpret_cast<uint4*>(smem + p.l.ent)[i] = src[i];
    G = *reinterpret_cast<const int*>(src + table_words);
    __syncthreads();
  } else {
    G = moe_groups<kThreads>(p, smem, smem, warp_total, kDown ? 0 : static_cast<int>(cluster_ctarank()), kDown ? 1 : p.S);
    if (!kDown && p.tables != nullptr && blockIdx.x == 0) {
      uint4* dst = reinterpret_cast<uint4*>(p.tables);
      for (int i = threadIdx.x; i < table_words; i += kThreads) dst[i] = reinterpret_cast<const uint4*>(smem + p.l.ent)[i];
      if (threadIdx.x == 0) *reinterpret_cast<int*>(dst + table_words) = G;
    }
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int KT = p.KT;
  // this CTA's items [i0, i1): up: item = group NT + tile; down: item = group, the tile is the cluster's
  const int rank = kDown ? static_cast<int>(cluster_ctarank()) : 0;
  const int total = kDown ? G : G * p.NT;
  const int share = kDown ? rank : static_cast<int>(blockIdx.x), shares = kDown ? p.S : static_cast<int>(gridDim.x);
  // (at most 640 groups of 128 tiles times 148 shares: below 2^24)
  const int i0 = static_cast<int>(static_cast<uint32_t>(total * share) / static_cast<uint32_t>(shares));
  const int i1 = static_cast<int>(static_cast<uint32_t>(total * (share + 1)) / static_cast<uint32_t>(shares));
  const int n_items = i1 - i0;
  const int g0 = kDown ? i0 : i0 / p.NT, g1 = n_items <= 0 ? g0 : kDown ? i1 : (i1 - 1) / p.NT + 1;  // this CTA's groups
  const int tile0 = kDown ? static_cast<int>(blockIdx.x) / p.S : i0 - g0 * p.NT;
  // a role's walk over the items, no division in it: group (its buffer, the parity of the buffer's
  // turn), tile, and whether this is the group's last item here
  struct Walk {
    int i = 0, g, tile, buf = 0;
    uint32_t turn = 0;
    bool fresh = true;  // first item of its group
  };
  auto walk = [&] {
    Walk w;
    w.g = g0;
    w.tile = tile0;
    return w;
  };
  auto last_of_group = [&](const Walk& w) { return kDown || w.tile + 1 == p.NT || w.i + 1 == n_items; };
  auto next_item = [&](Walk& w) {
    ++w.i;
    w.fresh = kDown || w.tile + 1 == p.NT;
    if (!kDown) w.tile = w.fresh ? 0 : w.tile + 1;
    if (w.fresh) {
      ++w.g;
      if (++w.buf == bufs) {
        w.buf = 0;
        w.turn ^= 1;
      }
    }
  };

  if (warp == 0) {
    // ---- producer: lane 0 copies a stage's weight codes, lane 1 its scales ----
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    // the first group's channel factors go ahead of the weights: behind them they would wait for as
    // many bytes as the stages hold
    if constexpr (!kDown) named_bar_sync(3, kQuantThreads + 32);
    const uint64_t policy = l2_evict_first();  // read once: the rest of L2 keeps its lines
    for (Walk w = walk(); w.i < n_items && ok; next_item(w)) {
      const int e = grp[w.g].y & 0xFFFF;
      const size_t img = weight_image(e, w.tile, 0, p.NT / 2, KT);
      const uint8_t* src = (lane & 1) ? p.Ws + img * kTileSfBytes : p.Wq + img * kTileCodeBytes;
      const uint32_t bytes = (lane & 1) ? kTileSfBytes : kTileCodeBytes;
      uint8_t* dst0 = (lane & 1) ? smem + p.l.sf : smem;
      for (int kt = 0; kt < KT; ++kt) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, kWaitTimeoutNs)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], kStageBytes);
        __syncwarp();
        bulk_g2s_hint_if(lane < 2, dst0 + stage * bytes, src, bytes, &full[stage], policy);
        src += 2 * bytes;  // the next K tile's image pair
        if (++stage == stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if constexpr (!kDown) {
      // the down kernel's first items: of every share its first group, tile by tile, and so on
      for (int i = lane; i < 2 * p.ahead; i += 32) {
        int at = (i / 2) * shares + share;
        const int kt = at % p.KT_next;
        at /= p.KT_next;
        const int tile = at % p.NT_next;
        at /= p.NT_next;
        const int r = at % p.S_next, g = G * r / p.S_next + at / p.S_next;
        if (g < G * (r + 1) / p.S_next)
          prefetch_image(p.Wq_next, p.Ws_next, weight_image(grp[g].y & 0xFFFF, tile, 0, p.NT_next / 2, p.KT_next) + 2 * kt, lane);
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer: the whole warp takes every step and one elected lane issues, so addresses and
    // descriptors stay in uniform registers (a stage's four MMAs issue in 260 cycles, from a lone lane
    // in 300, and its scale copies in 350, from a lone lane in 440) ----
    {
      const uint32_t idesc_lo = idesc_mxf4(128, kRows, 0, 0), idesc_hi = idesc_mxf4(128, kRows, 2, 2);
      const uint64_t a0 = sdesc_kmajor_sw128(smem_u32(smem)), b0 = sdesc_kmajor_sw128(smem_u32(smem + p.l.b));
      int stage = 0;
      uint32_t phase = 0;
      uint64_t ad = a0;  // the stage's weights and scales, stepped along with it
      uint32_t sf = tmem + kSfCol;
      bool ok = true;
      for (Walk w = walk(); w.i < n_items && ok; next_item(w)) {
        const int ab = w.i & 1;
        uint64_t bd = b0 + (static_cast<uint32_t>(w.buf * KT * kBCodeBytes) >> 4);
        const uint32_t acc = tmem + ab * kRows;
        if (w.fresh && !mbar_wait_warp(&bfull[w.buf], w.turn, abort_flag, kWaitTimeoutNs)) break;
        if (!mbar_wait_warp(&acce[ab], ((w.i >> 1) & 1) ^ 1, abort_flag, kWaitTimeoutNs)) break;
        tc_fence_after();
        for (int kt = 0; kt < KT; ++kt) {
          // the scales are copied once the stage is complete: their arrival stands for both
          if (!mbar_wait_warp(&sfull[stage], phase, abort_flag, kWaitTimeoutNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            mma_stage(ad, bd, sf, sf + 8, acc, idesc_lo, idesc_hi, kt == 0);
            tc_commit(&empty[stage]);
          }
          __syncwarp();
          ad += kTileCodeBytes >> 4;
          bd += kBCodeBytes >> 4;
          sf += 16;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
            ad = a0;
            sf = tmem + kSfCol;
          }
        }
        if (!ok) break;
        if (elect_one()) {
          tc_commit(&accf[ab]);
          if (last_of_group(w)) tc_commit(&bempty[w.buf]);
        }
        __syncwarp();
      }
    }
  } else if (warp == 2) {
    // ---- scale copies of a stage into its TMEM slot: weights 8 columns, tokens 8 columns ----
    {
      const uint64_t sfa0 = sdesc_sf_block(smem_u32(smem + p.l.sf)), sfb0 = sdesc_sf_block(smem_u32(smem + p.l.bsf));
      int stage = 0;
      uint32_t phase = 0;
      uint64_t sa = sfa0;
      uint32_t sf = tmem + kSfCol;
      bool ok = true;
      for (Walk w = walk(); w.i < n_items && ok; next_item(w)) {
        uint64_t sb = sfb0 + (static_cast<uint32_t>(w.buf * KT * kBSfBytes) >> 4);
        if (w.fresh && !mbar_wait_warp(&bfull[w.buf], w.turn, abort_flag, kWaitTimeoutNs)) break;
        for (int kt = 0; kt < KT; ++kt) {
          if (!mbar_wait_warp(&full[stage], phase, abort_flag, kWaitTimeoutNs)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            tc_cp_32x128b_warpx4(sf, sa);
            tc_cp_32x128b_warpx4(sf + 4, sa + (512 >> 4));
            tc_cp_32x128b_warpx4(sf + 8, sb);
            tc_cp_32x128b_warpx4(sf + 12, sb + (256 >> 4));
            tc_commit(&sfull[stage]);
          }
          __syncwarp();
          sa += kTileSfBytes >> 4;
          sb += kBSfBytes >> 4;
          sf += 16;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
            sa = sfa0;
            sf = tmem + kSfCol;
          }
        }
      }
    }
  } else if (warp == 3) {
    if constexpr (kDown) {
      // ---- the groups' activations into the tensor core's layout: codes in 16-byte pieces, scales in
      // words of four blocks ----
      pdl_wait();  // they come from the up kernel
      pdl_trigger();
      const int code_row = p.K / 2, sf_row = p.K / 32;
      int buf = 0;
      uint32_t turn = 1;
      for (int g = g0; g < g1; ++g) {
        if (!mbar_wait_warp(&bempty[buf], turn, abort_flag, kWaitTimeoutNs)) break;
        const int2 gr = grp[g];
        const int first = gr.x, rows = gr.y >> 16;
        uint8_t* bq = smem + p.l.b + buf * KT * kBCodeBytes;
        uint8_t* bs = smem + p.l.bsf + buf * KT * kBSfBytes;
        // lane: piece c of row j, four rows at a time (lanes past the last row repeat it)
        const int c = lane & 7;
        for (int j0 = 0; j0 < rows; j0 += 4) {
          const int j = min(j0 + (lane >> 3), rows - 1);
          const int e = ent[first + j];
          const uint8_t* src = p.codes + static_cast<int64_t>(e) * code_row + c * 16;
          uint8_t* dst = bq + code_chunk_offset(j, c);
#pragma unroll 4
          for (int kt = 0; kt < KT; ++kt) cp_async16(dst + kt * kBCodeBytes, src + kt * 128);
          const uint8_t* sf = p.scales + static_cast<int64_t>(e) * sf_row;
          for (int w0 = 0; w0 < 2 * KT; w0 += 8) {
            const int w = min(w0 + c, 2 * KT - 1);
            cp_async4(bs + (w >> 1) * kBSfBytes + (w & 1) * 256 + j * 16, sf + w * 4);
          }
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bfull[buf]);
        if (++buf == bufs) {
          buf = 0;
          turn ^= 1;
        }
      }
    }
  } else if (warp < 8) {
    // ---- epilogue: 16 accumulator columns (tokens) of this thread's weight row ----
    const int q = warp & 3, row = q * 32 + lane;
    if constexpr (kDown) {
      for (int t = 0; t < p.T; ++t) acc[t * kRowsTile + row] = 0.f;
    }
    for (Walk w = walk(); w.i < n_items; next_item(w)) {
      const int ab = w.i & 1;
      const int2 gr = grp[w.g];
      const int first = gr.x, e = gr.y & 0xFFFF, rows = gr.y >> 16;
      // up: of the item's 64 channels warps 0 and 1 quantise the first block of 32, warps 2 and 3 the second
      const int channel = w.tile * (kRowsTile / 2) + (q >> 1) * 32 + lane;
      float rcp = 1.f;
      if constexpr (!kDown) rcp = __frcp_rn(__ldg(p.D_next + static_cast<int64_t>(e) * (p.N / 2) + channel));
      __syncwarp();
      const bool ok = mbar_wait_warp(&accf[ab], (w.i >> 1) & 1, abort_flag, kWaitTimeoutNs);
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + ab * kRows;
      if constexpr (kDown) {
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int j0 = 0; j0 < rows; j0 += 4) {
          uint32_t r[4];
          tmem_ld_32x32b_x4(taddr + j0, r);
          // the tokens of a group differ, so their sums are read together, then written
          float* o[4];
          float wt[4], v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int jj = first + min(j0 + j, rows - 1);
            o[j] = acc + ent_tok[jj] * kRowsTile + row;
            wt[j] = ent_w[jj] * 0.03125f;
            v[j] = *o[j];
          }
          tmem_wait_ld(r);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j0 + j < rows) *o[j] = fmaf(wt[j], __uint_as_float(r[j]), v[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acce[ab]);
      } else {
        // weight rows 2 c and 2 c + 1 are the gate and the up row of channel c: of two tokens
        // the even lane finishes the first, the odd lane the second
        uint16_t* act = reinterpret_cast<uint16_t*>(smem + p.l.extra + ab * kActBytes);
        if (ok) {
          tc_fence_after();
          const bool odd = lane & 1;
#pragma unroll 1
          for (int j0 = 0; j0 < rows; j0 += 4) {
            uint32_t r[4];
            tmem_ld_32x32b_x4(taddr + j0, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const float a = __uint_as_float(r[j]) * 0.03125f, b = __uint_as_float(r[j + 1]) * 0.03125f;
              const float other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
              act[(j0 + j + (odd ? 1 : 0)) * kActStride + (row >> 1)] =
                  bf16_bits(gated(odd ? other : a, odd ? b : other, p.gelu));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acce[ab]);
        }
        // (the two copies of `act` alternate: this barrier also separates an item's reads from
        // the writes of the item after the next)
        if (!named_bar_all(1, 128, ok)) break;
        const uint16_t* mine = act + (q >> 1) * 32 + lane;
#pragma unroll 1
        for (int j = q & 1; j < rows; j += 4) {  // tokens j and j + 2
          const int j2 = min(j + 2, rows - 1);
          const float h[2] = {bf16lo(mine[j * kActStride]), bf16lo(mine[j2 * kActStride])};
          uint32_t byte[2], scale[2];
          act_lane_blocks<2>(h, rcp, byte, scale);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (n == 0 || j + 2 < rows) {
              const int64_t at = ent[first + (n == 0 ? j : j2)];
              if (!(lane & 1)) p.codes[at * (p.N / 4) + channel / 2] = static_cast<uint8_t>(byte[n]);
              if (lane == 0) p.scales[at * (p.N / 64) + channel / 32] = static_cast<uint8_t>(scale[n]);
            }
          }
          __syncwarp();
        }
      }
    }
  } else {
    if constexpr (!kDown) {
      // ---- x quantiser: all of its warps on one group after the other.  A thread owns eight channels of a
      // chunk of 2048, so their reciprocals stay in its registers; threads left over take other rows ----
      const int tt = static_cast<int>(threadIdx.x) - 8 * 32;
      // the channel factors of the next chunk (of this group or the next) are loaded ahead
      float4 d[2];
      auto load_d = [&](int g, int k0) {
        const int ch = min(k0 + tt % (min(kChunk, p.K - k0) / 8) * 8, p.K - 8);
        const float* src = p.D + static_cast<int64_t>(grp[g].y & 0xFFFF) * p.K + ch;
        d[0] = ld_now(src);
        d[1] = ld_now(src + 4);
      };
      if (g0 < g1) load_d(g0, 0);
      asm volatile("bar.arrive 3, %0;" ::"n"(kQuantThreads + 32) : "memory");
      bool ok = true;
      int buf = 0;
      uint32_t buf_turn = 1;
      for (int g = g0; g < g1 && ok; ++g) {
        const int2 gr = grp[g];
        const int first = gr.x, rows = gr.y >> 16;
        uint8_t* bq = smem + p.l.b + buf * KT * kBCodeBytes;
        uint8_t* bs = smem + p.l.bsf + buf * KT * kBSfBytes;
        ok = mbar_wait_warp(&bempty[buf], buf_turn, abort_flag, kWaitTimeoutNs);
        if (!ok) break;
#pragma unroll 1
        for (int k0 = 0; k0 < p.K; k0 += kChunk) {
          const int pieces = min(kChunk, p.K - k0) / 8, split = kQuantThreads / pieces;
          const int rs = tt / pieces, ch = k0 + tt % pieces * 8;
          const int kt = ch >> 8, c = (ch >> 5) & 7;
          const float2 r2[4] = {f2(__frcp_rn(d[0].x), __frcp_rn(d[0].y)), f2(__frcp_rn(d[0].z), __frcp_rn(d[0].w)),
                                f2(__frcp_rn(d[1].x), __frcp_rn(d[1].y)), f2(__frcp_rn(d[1].z), __frcp_rn(d[1].w))};
          if (k0 + kChunk < p.K) load_d(g, k0 + kChunk);
          else if (g + 1 < g1) load_d(g + 1, 0);
          const uint16_t* x = p.x + ch;
          // lanes without a row repeat the last one and store nothing
          auto load_x = [&](int j) {
            return *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(ent_tok[first + min(j, rows - 1)]) * p.K);
          };
          uint4 next = load_x(rs);
#pragma unroll 1
          for (int j0 = 0; j0 < rows; j0 += split) {
            const uint4 xv = next;
            const int j = j0 + rs;
            next = load_x(j + split);
            __syncwarp();
            uint32_t codes, scale;
            act_quarter_block(xv, r2, codes, scale);
            if (rs < split && j < rows) {
              *reinterpret_cast<uint32_t*>(bq + kt * kBCodeBytes + code_chunk_offset(j, c) + (lane & 3) * 4) = codes;
              if ((lane & 3) == 0) bs[kt * kBSfBytes + (c >> 2) * 256 + j * 16 + (c & 3)] = static_cast<uint8_t>(scale);
            }
            __syncwarp();
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bfull[buf]);
        if (++buf == bufs) {
          buf = 0;
          buf_turn ^= 1;
        }
      }
    }
  }
  __syncwarp();

  if constexpr (kDown) {
    // ---- sum of the cluster's tiles ----
    pdl_wait();  // y may still be read by an earlier kernel
    fence_proxy_async_smem();  // the tile may leave by bulk copy
    if (p.T <= kFewTokens) {
      // task (token, 4 channels), dealt out to the ranks; each rank adds from its own tile on, round the
      // cluster: an order that the sizes fix
      __syncthreads();
      cluster_sync_all();  // every CTA's tile is complete
      const uint32_t local = smem_u32(acc);
      for (int task = static_cast<int>(threadIdx.x) * p.S + rank; task < p.T * 32; task += kThreads * p.S) {
        const int t = task >> 5, c = (task & 31) * 4;
        // all loads first, one round trip
        float4 part[8];
#pragma unroll
        for (int o = 0; o < 8; ++o) {
          if (o < p.S) {
            const int from = rank + o < p.S ? rank + o : rank + o - p.S;
            part[o] = ld_dsmem_f32x4(
                mapa_shared(local + static_cast<uint32_t>((t * kRowsTile + c) * 4), static_cast<uint32_t>(from)));
          }
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int o = 0; o < 8; ++o) {
          if (o < p.S) {
            s[0] += part[o].x; s[1] += part[o].y; s[2] += part[o].z; s[3] += part[o].w;
          }
        }
        *reinterpret_cast<uint2*>(p.y + static_cast<int64_t>(t) * p.N + tile0 * kRowsTile + c) =
            make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
      }
    } else {
      // rank o sums tokens [o n, (o + 1) n): every CTA copies it those rows of its tile, into the place of the
      // weight stages (128 tokens: 3.4 us, by single loads from the other CTAs 4.8)
      const int n = (p.T + p.S - 1) / p.S;
      auto rows_of = [&](int o) { return max(0, min(n, p.T - o * n)); };
      const int mine = rows_of(rank);
      if (threadIdx.x == 0) mbar_arrive_expect_tx(recv, static_cast<uint32_t>(p.S * mine * kRowsTile * 4));
      __syncthreads();
      cluster_sync_all();  // every CTA's tile is complete, its stages done with, its barrier armed
      const int o = static_cast<int>(threadIdx.x);
      if (o < p.S && rows_of(o) > 0)
        bulk_s2s_cluster(mapa_shared(smem_u32(smem) + static_cast<uint32_t>(rank * n * kRowsTile * 4), static_cast<uint32_t>(o)),
                         acc + o * n * kRowsTile, static_cast<uint32_t>(rows_of(o) * kRowsTile * 4),
                         mapa_shared(smem_u32(recv), static_cast<uint32_t>(o)));
      __syncwarp();
      if (mine == 0 || mbar_wait_warp(recv, 0, abort_flag, kWaitTimeoutNs)) {
        const float* from = reinterpret_cast<const float*>(smem);
        for (int task = static_cast<int>(threadIdx.x); task < mine * 32; task += kThreads) {
          const int t = task >> 5, c = (task & 31) * 4;
          float s[4] = {0.f, 0.f, 0.f, 0.f};
          for (int q = 0; q < p.S; ++q) {  // rank order
            const float4 v = *reinterpret_cast<const float4*>(from + (q * n + t) * kRowsTile + c);
            s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
          }
          *reinterpret_cast<uint2*>(p.y + static_cast<int64_t>(rank * n + t) * p.N + tile0 * kRowsTile + c) =
              make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
        }
      }
      __syncthreads();
    }
    cluster_sync_all();  // no CTA leaves while another, or a copy, may still read its tile
  }
  if (*abort_flag && threadIdx.x == 0 && p.status) *p.status = MACAQ_ERR_DEVICE_TIMEOUT;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, tmem_cols(stages));
}

}  // namespace macaq
