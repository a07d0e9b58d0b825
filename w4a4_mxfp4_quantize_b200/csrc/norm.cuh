// The norms between two blocks, fused with the gate and the scale of the residual
// branch:
//   p  = y                       or  y rsqrt(mean y^2 + eps) (offset + w_post)
//   h' = round_T(h + scale gate p)                 (T: bf16 or fp32, the stream's type)
//   n  = RNE_bf16(h' rsqrt(mean h'^2 + eps) (offset + w_pre))
// Sums, means and products in FP32; h' is rounded once to the stream's type and the
// second norm reads that rounded value, so n is what a norm run on the stored h'
// would give.
#pragma once
#include "mx.cuh"
#include "ptx.cuh"

namespace macaq {

struct NormParams {
  const void* h;         // bf16 or fp32 [M, C]
  const uint16_t* y;     // bf16 [M, C] or nullptr: h' = h, nothing is added or written
  const float* w_post;   // fp32 [C] or nullptr: y is used as it is
  const void* gate;      // bf16 or fp32 [ceil(M / rows_per_gate), C] or nullptr
  const float* w_pre;    // fp32 [C] or nullptr: no n
  void* h_out;           // [M, C] in h's type (may be h itself)
  uint16_t* n_out;       // bf16 [M, C]
  int rows_per_gate;
  int M, C;
  int h_f32, gate_f32;
  float scale, eps, offset;
};

namespace norm {

__device__ __forceinline__ void bf16x8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(w[i]);
    f[2 * i + 1] = bf16hi(w[i]);
  }
}
__device__ __forceinline__ uint4 to_bf16x8(const float (&f)[8]) {
  return make_uint4(f2_to_bf16x2(f2(f[0], f[1])), f2_to_bf16x2(f2(f[2], f[3])), f2_to_bf16x2(f2(f[4], f[5])),
                    f2_to_bf16x2(f2(f[6], f[7])));
}
// Eight elements of a row in their stored form: 16 bytes of bf16 or 32 of fp32.
template <bool kF32>
struct Raw {
  uint4 v[kF32 ? 2 : 1];
};
template <bool kF32>
__device__ __forceinline__ Raw<kF32> load8(const void* p, int64_t i) {
  Raw<kF32> r;
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (kF32 ? 4 : 2));
  r.v[0] = s[0];
  if constexpr (kF32) r.v[1] = s[1];
  return r;
}
template <bool kF32>
__device__ __forceinline__ void widen(const Raw<kF32>& r, float (&f)[8]) {
  if constexpr (kF32) {
    f[0] = __uint_as_float(r.v[0].x); f[1] = __uint_as_float(r.v[0].y);
    f[2] = __uint_as_float(r.v[0].z); f[3] = __uint_as_float(r.v[0].w);
    f[4] = __uint_as_float(r.v[1].x); f[5] = __uint_as_float(r.v[1].y);
    f[6] = __uint_as_float(r.v[1].z); f[7] = __uint_as_float(r.v[1].w);
  } else {
    bf16x8(r.v[0], f);
  }
}
__device__ __forceinline__ void weights8(const float* w, int c, float offset, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + c)), b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
  f[0] = offset + a.x; f[1] = offset + a.y; f[2] = offset + a.z; f[3] = offset + a.w;
  f[4] = offset + b.x; f[5] = offset + b.y; f[6] = offset + b.z; f[7] = offset + b.w;
}
__device__ __forceinline__ void gate8(const NormParams& p, int64_t at, float (&f)[8]) {
  if (p.gate_f32) widen<true>(load8<true>(p.gate, at), f);
  else widen<false>(load8<false>(p.gate, at), f);
}

// Sum over the threads that share a row: a warp, or the whole CTA.  The CTA form
// alternates between two sets of partial sums, so one barrier per sum is enough.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float (&part)[2][32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (!kWarpRow) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) part[turn][warp] = v;
    __syncthreads();
    v = lane < nw ? part[turn][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    turn ^= 1;
  }
  return v;
}

}  // namespace norm

// One row per warp (kWarpRow) or per CTA, V vectors of eight elements per thread,
// the row held in registers between the two sums: every byte is read and written
// once.  The next row of this warp or CTA is loaded while this one's sums run: 16385
// fp32 rows of 2048 take 70.5 us so in a captured graph (5.7 TB/s; 71 to 78 us a call),
// 82.5 with one row in flight; the two sums, each a wait of the whole CTA, are what is
// left.  Above 8192 columns (V = 4, one CTA of 512 threads on an SM) they are hidden
// less: 2048 rows of 16384 take 73.6 us in bf16 (3.7 TB/s), 99.4 in fp32 (4.1).
template <bool kWarpRow, int V, bool kF32>
__global__ void __launch_bounds__(kWarpRow ? 256 : V == 1 ? 1024 : 512) block_norm_kernel(
    const __grid_constant__ NormParams p) {
  __shared__ float part[2][32];
  int turn = 0;
  const int group = kWarpRow ? 32 : static_cast<int>(blockDim.x);
  const int t = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int rows_per_cta = static_cast<int>(blockDim.x) / group;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows_per_cta;
  const float inv_c = 1.0f / static_cast<float>(p.C);
  norm::Raw<kF32> hr[V];
  uint4 yr[V];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * group + t) * 8;
      if (row < p.M && c < p.C) {
        hr[v] = norm::load8<kF32>(p.h, row * p.C + c);
        if (p.y != nullptr) yr[v] = *reinterpret_cast<const uint4*>(p.y + row * p.C + c);
      }
    }
  };
  pdl_wait();  // h, y and the gate may come from the kernel before
  pdl_trigger();
  int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_cta + (kWarpRow ? threadIdx.x >> 5 : 0);
  load(row);
  for (; row < p.M; row += step) {
    const int64_t base = row * p.C;
    float hn[V][8], f[V][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if ((v * group + t) * 8 < p.C) {
        norm::widen<kF32>(hr[v], hn[v]);
        if (p.y != nullptr) {
          norm::bf16x8(yr[v], f[v]);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(f[v][i], f[v][i], ss);
        }
      }
    }
    load(row + step);
    float rs_post = 1.f;
    if (p.w_post != nullptr) rs_post = rsqrtf(norm::row_sum<kWarpRow>(ss, part, turn) * inv_c + p.eps);
    const int64_t gate_base =
        p.gate != nullptr ? static_cast<int64_t>(static_cast<int>(row) / p.rows_per_gate) * p.C : 0;
    ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * group + t) * 8;
      if (c < p.C) {
        if (p.y != nullptr) {
          float w[8];
          if (p.w_post != nullptr) {
            norm::weights8(p.w_post, c, p.offset, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[v][i] = f[v][i] * rs_post * w[i];
          }
          if (p.gate != nullptr) {
            norm::gate8(p, gate_base + c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[v][i] *= w[i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) hn[v][i] = hn[v][i] + p.scale * f[v][i];
          if constexpr (kF32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.h_out) + base + c);
            o[0] = make_float4(hn[v][0], hn[v][1], hn[v][2], hn[v][3]);
            o[1] = make_float4(hn[v][4], hn[v][5], hn[v][6], hn[v][7]);
          } else {
            const uint4 o = norm::to_bf16x8(hn[v]);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h_out) + base + c) = o;
            norm::bf16x8(o, hn[v]);  // the second norm reads the stored value
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(hn[v][i], hn[v][i], ss);
      }
    }
    if (p.w_pre != nullptr) {
      const float rs = rsqrtf(norm::row_sum<kWarpRow>(ss, part, turn) * inv_c + p.eps);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * group + t) * 8;
        if (c < p.C) {
          float w[8];
          norm::weights8(p.w_pre, c, p.offset, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) hn[v][i] = hn[v][i] * rs * w[i];
          *reinterpret_cast<uint4*>(p.n_out + base + c) = norm::to_bf16x8(hn[v]);
        }
      }
    }
  }
}

// Rows too wide for the registers of one CTA: the same sums over passes that read
// the row again, mostly from L2 (each thread only what it read or wrote itself).  1024
// rows of 32768 take 76.6 us in bf16, 92.9 in fp32 (3.5 and 4.3 TB/s of what has to move).
template <bool kF32>
__global__ void __launch_bounds__(1024) block_norm_wide_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[2][32];
  int turn = 0;
  const float inv_c = 1.0f / static_cast<float>(p.C);
  pdl_wait();
  pdl_trigger();
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const int64_t base = row * p.C;
    float rs_post = 1.f;
    if (p.w_post != nullptr) {
      float ss = 0.f;
      for (int c = threadIdx.x * 8; c < p.C; c += blockDim.x * 8) {
        float f[8];
        norm::bf16x8(*reinterpret_cast<const uint4*>(p.y + base + c), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
      }
      rs_post = rsqrtf(norm::row_sum<false>(ss, part, turn) * inv_c + p.eps);
    }
    const int64_t gate_base =
        p.gate != nullptr ? static_cast<int64_t>(static_cast<int>(row) / p.rows_per_gate) * p.C : 0;
    float ss = 0.f;
    for (int c = threadIdx.x * 8; c < p.C; c += blockDim.x * 8) {
      float hn[8];
      norm::widen<kF32>(norm::load8<kF32>(p.h, base + c), hn);
      if (p.y != nullptr) {
        float f[8], w[8];
        norm::bf16x8(*reinterpret_cast<const uint4*>(p.y + base + c), f);
        if (p.w_post != nullptr) {
          norm::weights8(p.w_post, c, p.offset, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = f[i] * rs_post * w[i];
        }
        if (p.gate != nullptr) {
          norm::gate8(p, gate_base + c, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) hn[i] = hn[i] + p.scale * f[i];
        if constexpr (kF32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.h_out) + base + c);
          o[0] = make_float4(hn[0], hn[1], hn[2], hn[3]);
          o[1] = make_float4(hn[4], hn[5], hn[6], hn[7]);
        } else {
          const uint4 o = norm::to_bf16x8(hn);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h_out) + base + c) = o;
          norm::bf16x8(o, hn);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(hn[i], hn[i], ss);
    }
    if (p.w_pre != nullptr) {
      const float rs = rsqrtf(norm::row_sum<false>(ss, part, turn) * inv_c + p.eps);
      const void* src = p.y != nullptr ? p.h_out : p.h;
      for (int c = threadIdx.x * 8; c < p.C; c += blockDim.x * 8) {
        float hn[8], w[8];
        norm::widen<kF32>(norm::load8<kF32>(src, base + c), hn);
        norm::weights8(p.w_pre, c, p.offset, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) hn[i] = hn[i] * rs * w[i];
        *reinterpret_cast<uint4*>(p.n_out + base + c) = norm::to_bf16x8(hn);
      }
    }
  }
}

}  // namespace macaq
