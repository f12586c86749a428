// Norms of queries and keys for each head and the position rotation, one pass.
//
// Per token and head x [d]:
//   y = x * w / sqrt(mean(x^2) + eps)          (w given; else y = x)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq[i]
// for the pairs (y[i], y[i + rot/2]), or (y[2i], y[2i + 1]) interleaved, of the
// first rot values; the others pass. fp32 throughout, one rounding to bf16.
//
// The angle is formed in float64 (a position of 2^20 times a frequency of 1
// keeps 2^-32 there; in fp32 it would be off by up to 2^-4) and reduced by
// whole turns before the fp32 sine and cosine.
//
// Memory bound: every element is read and written once (4 bytes an element).
// A vector of d values is held by d/8 neighbouring lanes, 16 bytes each, so
// the sum of squares and the partner values of a pair are register shuffles.
// A block takes kRopeTokens tokens, computes their sines and cosines once
// for all heads, and keeps kRopeUnroll vectors a lane in flight.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace respin {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 2;

struct RopeArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  const int32_t* positions;
  const float* inv_freq;
  long long ldq, ldk, ldqo, ldko;   // elements between tokens
  int N, Hq, Hkv, rot;
  int tokens;                       // tokens of a block
  float eps;
};

// Sine and cosine of position * freq, reduced by whole turns in float64.
__device__ __forceinline__ float2 rope_cos_sin(int position, float freq) {
  const double kTurn = 6.283185307179586476925;           // 2 pi, rounded to float64
  const double kTurnRest = 2.4492935982947064e-16;        // 2 pi - kTurn
  const double a = static_cast<double>(position) * static_cast<double>(freq);
  const double n = rint(a * 0.15915494309189533577);      // 1 / (2 pi)
  const double r = fma(-n, kTurnRest, fma(-n, kTurn, a));
  float s, c;
  sincosf(static_cast<float>(r), &s, &c);
  return make_float2(c, s);
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 6) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int L = D / 8;                         // lanes of one vector
  constexpr int V = kRopeThreads / L;              // vectors of one pass of the block
  extern __shared__ float2 rope_cs[];              // [tokens][rot / 2]
  const int tid = threadIdx.x, li = tid % L;
  const int half = a.rot / 2;
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, a.N - t0);
  const int heads = a.Hq + a.Hkv;
  const int total = nt * heads;

  grid_dep_wait();
  grid_dep_launch();
  // A lane reads the angles of its 8 values (4 pairs interleaved): angle E l + i lies at i * (half / E) + l,
  // so that neighbouring lanes read neighbouring ones.
  constexpr int E = INTERLEAVED ? 4 : 8;
  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int t = i / half, f = i - t * half;
    rope_cs[t * half + (f % E) * (half / E) + f / E] = rope_cos_sin(a.positions[t0 + t], a.inv_freq[f]);
  }
  uint4 wq = make_uint4(0u, 0u, 0u, 0u), wk = wq;
  if (a.q_weight != nullptr) wq = reinterpret_cast<const uint4*>(a.q_weight)[li];
  if (a.k_weight != nullptr) wk = reinterpret_cast<const uint4*>(a.k_weight)[li];
  __syncthreads();

  // Blocks of one row of the grid share its tokens: each takes every
  // gridDim.y-th pass of V vectors.
  for (int base = blockIdx.y * V; base < total; base += gridDim.y * V * kRopeUnroll) {
    uint4 raw[kRopeUnroll];
    int vec[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      vec[u] = base + u * static_cast<int>(gridDim.y) * V + tid / L;
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (vec[u] < total) {
        const int t = vec[u] / heads, h = vec[u] - t * heads;
        const __nv_bfloat16* p = h < a.Hq ? a.q + (t0 + t) * a.ldq + static_cast<long long>(h) * D
                                          : a.k + (t0 + t) * a.ldk + static_cast<long long>(h - a.Hq) * D;
        raw[u] = reinterpret_cast<const uint4*>(p)[li];
      }
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const bool live = vec[u] < total;   // lanes of dead vectors still take part in the shuffles
      const int t = live ? vec[u] / heads : 0, h = live ? vec[u] - t * heads : 0;
      const bool is_q = h < a.Hq;
      float x[8], y[8];
      bf16x8_to_f32(raw[u], x);
      if (a.q_weight != nullptr || a.k_weight != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        float inv = rsqrtf(ss * (1.0f / D) + a.eps);
        // Values above 2^60 or so: their squares leave binary32. Scaled by
        // 2^-96 the sum is finite for any bf16 values; x takes the same scale.
        if (__any_sync(0xFFFFFFFFu, !(ss < __int_as_float(0x7F800000)))) {
          const float down = __int_as_float((127 - 96) << 23);
          float s2 = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) s2 = fmaf(x[i] * down, x[i] * down, s2);
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, o);
          if (!(ss < __int_as_float(0x7F800000))) {
            inv = rsqrtf(s2 * (1.0f / D));   // eps * 2^-192 is nothing beside it
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= down;
          }
        }
        const bool on = is_q ? a.q_weight != nullptr : a.k_weight != nullptr;
        if (on) {
          float w[8];
          bf16x8_to_f32(is_q ? wq : wk, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
        } else {
          bf16x8_to_f32(raw[u], x);
        }
      }
      const float2* cs = rope_cs + t * half;
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 r = make_float2(1.0f, 0.0f);
          if (8 * li + 2 * i < a.rot) r = cs[i * (half / 4) + li];
          y[2 * i] = x[2 * i] * r.x - x[2 * i + 1] * r.y;
          y[2 * i + 1] = x[2 * i + 1] * r.x + x[2 * i] * r.y;
        }
        if (8 * li >= a.rot) {   // a rotation by nothing, without its 0 * inf
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i];
        }
      } else {
        const int hl = half / 8;   // lanes of half the rotated values
        const bool first = li < hl, in = li < 2 * hl;
        const int lane = tid & 31;
        const int src = (lane & ~(L - 1)) + (in ? (first ? li + hl : li - hl) : li);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xFFFFFFFFu, x[i], src);
        if (in) {
          const float2* c = cs + (first ? li : li - hl);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 r = c[i * hl];
            y[i] = first ? x[i] * r.x - y[i] * r.y : x[i] * r.x + y[i] * r.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i];
        }
      }
      if (live) {
        __nv_bfloat16* p = is_q ? a.q_out + (t0 + t) * a.ldqo + static_cast<long long>(h) * D
                                : a.k_out + (t0 + t) * a.ldko + static_cast<long long>(h - a.Hq) * D;
        reinterpret_cast<uint4*>(p)[li] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                     pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
      }
    }
  }
}

}  // namespace respin
