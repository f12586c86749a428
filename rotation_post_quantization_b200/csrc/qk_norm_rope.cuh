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
// Every element is read and written once (4 bytes an element), which would take
// 13 us for 4096 tokens of 40 heads. What it takes beyond that: a block loads no
// vector before its angles are formed, with all blocks in one wave, and the
// warps then issue in 66 % of the cycles.
// A vector of d values is held by d/8 neighbouring lanes, both values of a
// pair in the same one (two runs of 8 bytes a lane, half the rotated width
// apart), so only the sum of squares needs shuffles. A block takes several
// tokens and computes their sines and cosines once for all heads; the next
// vectors are loaded while the last ones are turned. (With 16 consecutive
// bytes a lane and the partner fetched by shuffles: 27 us for 4096 tokens of
// 40 heads; this way 21 us, 3.9 TB/s.)
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
__global__ void __launch_bounds__(kRopeThreads, 5) qk_norm_rope_kernel(const RopeArgs a) {
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
  // Lane l turns the angles 4 l .. 4 l + 3; angle 4 l + i lies at i * (half / 4) + l, so that
  // neighbouring lanes read neighbouring ones.
  const int turning = half / 4;   // lanes
  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int t = i / half, f = i - t * half;
    rope_cs[t * half + (f & 3) * turning + (f >> 2)] = rope_cos_sin(a.positions[t0 + t], a.inv_freq[f]);
  }
  // This lane's values: 4 from o0 on and 4 from o1 on (in units of 4).
  const bool in = li < turning;
  const int o0 = INTERLEAVED || !in ? 2 * li : li;
  const int o1 = INTERLEAVED || !in ? 2 * li + 1 : li + turning;
  auto read8 = [&](const __nv_bfloat16* p) {
    const uint2 x = reinterpret_cast<const uint2*>(p)[o0], y = reinterpret_cast<const uint2*>(p)[o1];
    return make_uint4(x.x, x.y, y.x, y.y);
  };
  uint4 wq = make_uint4(0u, 0u, 0u, 0u), wk = wq;
  if (a.q_weight != nullptr) wq = read8(a.q_weight);
  if (a.k_weight != nullptr) wk = read8(a.k_weight);
  __syncthreads();

  // Blocks of one row of the grid share its tokens: each takes every
  // gridDim.y-th pass of V vectors.
  const int step = static_cast<int>(gridDim.y) * V;
  const int dt = step / heads, dh = step - dt * heads;   // a step on
  uint4 next[kRopeUnroll];
  int next_t[kRopeUnroll], next_h[kRopeUnroll];   // token (of the block) and head; token nt or more: none
  int at_t = (static_cast<int>(blockIdx.y) * V + tid / L) / heads;
  int at_h = static_cast<int>(blockIdx.y) * V + tid / L - at_t * heads;
  auto load = [&]() {   // the next vectors are on their way while the last ones are turned
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      next_t[u] = at_t;
      next_h[u] = at_h;
      next[u] = make_uint4(0u, 0u, 0u, 0u);
      if (at_t < nt)
        next[u] = read8(at_h < a.Hq ? a.q + (t0 + at_t) * a.ldq + at_h * D : a.k + (t0 + at_t) * a.ldk + (at_h - a.Hq) * D);
      at_t += dt;
      at_h += dh;
      if (at_h >= heads) {
        at_h -= heads;
        ++at_t;
      }
    }
  };
  load();
  for (int base = blockIdx.y * V; base < total; base += step * kRopeUnroll) {
    uint4 raw[kRopeUnroll];
    int vt[kRopeUnroll], vh[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      raw[u] = next[u];
      vt[u] = next_t[u];
      vh[u] = next_h[u];
    }
    load();
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const bool live = vt[u] < nt;   // lanes of absent vectors still take part in the shuffles
      const int t = live ? vt[u] : 0, h = vh[u];
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
      const float2* cs = rope_cs + t * half + li;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i];
      if (in) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 r = cs[i * turning];
          const int p = INTERLEAVED ? 2 * i : i, q = INTERLEAVED ? 2 * i + 1 : i + 4;
          y[p] = x[p] * r.x - x[q] * r.y;
          y[q] = x[q] * r.x + x[p] * r.y;
        }
      }
      if (live) {
        __nv_bfloat16* p = is_q ? a.q_out + (t0 + t) * a.ldqo + h * D : a.k_out + (t0 + t) * a.ldko + (h - a.Hq) * D;
        reinterpret_cast<uint2*>(p)[o0] = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
        reinterpret_cast<uint2*>(p)[o1] = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
      }
    }
  }
}

}  // namespace respin
