// Attention over the 8-bit cache for many rows a key head (prefill, chunks):
// the 5th-generation tensor cores. Mathematics and numbers as in
// kv_attention.cuh: fp16 products of exact codes, weights 2^(s log2 e +
// log2 vs - M) rounded to fp16, sums in fp32.
//
// A block takes 256 rows of one key head (rows are (token, query head of the
// group), so grouped heads share every tile of the cache) as two 128-row
// tiles, and walks the cache in 128-token steps:
//   warps 0-3, 4-7   one row a thread of tile 0 / 1: S from tensor memory,
//                    maximum, weights back to tensor memory as fp16;
//   warps 8-11       codes from global memory to registers, widened to fp16
//                    into shared memory (128-byte swizzle, two stages of K
//                    and two of V);
//   warp 12          one thread issues S = Q K^T (both from shared memory) and
//                    O += P V (P from tensor memory, V with its dims
//                    contiguous, i.e. N-major).
// While one tile's rows are in the exponentials, the tensor core works for
// the other. P takes the place of the S it comes from, so S of the next step
// waits for the product that reads P. The running maximum may lag by 2^8
// before the accumulators are rescaled, so rescaling is rare after the first
// steps and is done by the row's own thread.
//
// Tensor memory: S0, S1 (128 columns each, P in their first 64), O0, O1 (D
// columns each). Shared memory at D = 128: Q 64 KB, K and V 128 KB.
//
// Work: as in kv_attention.cuh one line of steps cut into equal pieces, here
// with each row group's own number of steps (causal rows see fewer).
#pragma once

#include "kv_attention.cuh"

namespace respin {

constexpr int kTcaRows = 128;       // rows of a tile
constexpr int kTcaGroup = 256;      // rows of a block
constexpr int kTcaTile = 128;       // tokens of a step
constexpr int kTcaThreads = 13 * 32;
constexpr int kTcaMinTiles = 4;     // least piece of a block
constexpr int kTcaMaxBlocks = 160;  // one per SM
constexpr int kTcaMeta = 4;         // steps whose scales are kept

// D[tmem] (+)= A[tmem] * B[smem]: A holds two 16-bit values a column.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor: fp16 A and B, fp32 accumulator; n_major: B with its
// N index contiguous.
__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N, bool n_major) {
  return (1u << 4) | (n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Descriptor of an N-major operand in the 128-byte swizzle: rows (k) of 64
// contiguous values, 8-row atoms of 1024 bytes one after the other, the next
// 64 values of N `n_stride` bytes on.
__device__ __forceinline__ uint64_t umma_desc_sw128_n(uint32_t smem_addr, uint32_t n_stride) {
  return (umma_desc_sw128(smem_addr) & ~(0x3FFFull << 16)) | (static_cast<uint64_t>(n_stride >> 4) << 16);
}

// Packed pairs of fp32.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 f32x2_split(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A sequence's row groups.
struct TcaSeq {
  int begin, n, len, rows, groups;
};

__device__ __forceinline__ TcaSeq tca_seq(const KvAttnArgs& a, int b) {
  TcaSeq s;
  int end;
  kv_rows(a.c, b, s.begin, end, s.len);
  s.n = end - s.begin;
  s.rows = s.n * a.G;
  s.groups = s.rows > a.few_rows ? (s.rows + kTcaGroup - 1) / kTcaGroup : 0;
  return s;
}

// First step and number of steps (at least 1) of row group g.
__device__ __forceinline__ int2 tca_steps(const KvAttnArgs& a, int n, int len, int rows, int g) {
  const int first = len - n + g * kTcaGroup / a.G;
  const int last = len - n + (min(rows, (g + 1) * kTcaGroup) - 1) / a.G;
  const int hi = a.causal ? min(last, len - 1) : len - 1;
  if (hi < 0) return make_int2(0, 1);
  const int lo = a.window > 0 ? min(hi, max(0, first - a.window + 1)) : 0;
  const int t0 = lo / kTcaTile;
  return make_int2(t0, hi / kTcaTile - t0 + 1);
}

// Where a role stands in the block's piece of the line.
struct TcaCursor {
  TcaSeq s;
  int b, g, h, z;   // sequence, row group, head, steps of the unit already behind
  int t0, tiles;    // of the unit
  int left;

  __device__ __forceinline__ void unit(const KvAttnArgs& a) {
    const int2 t = tca_steps(a, s.n, s.len, s.rows, g);
    t0 = t.x;
    tiles = t.y;
  }
  __device__ __forceinline__ int steps() const { return min(left, tiles - z); }
  __device__ __forceinline__ void next(const KvAttnArgs& a) {
    left -= steps();
    z = 0;
    if (left <= 0 || ++h < a.c.H) return;
    h = 0;
    if (++g >= s.groups) {
      g = 0;
      do {
        if (++b >= a.c.B) {
          left = 0;
          return;
        }
        s = tca_seq(a, b);
      } while (s.groups == 0);
    }
    unit(a);
  }
};

// The block's piece: every lane of one warp.
__device__ __forceinline__ void tca_locate(const KvAttnArgs& a, volatile int* sh) {
  const int lane = threadIdx.x & 31;
  long long total = 0, p0 = 0, before = 0, chunk = 0;
  int at_b = -1, at_g = 0, at_h = 0, at_z = 0, at_tiles = 0;
  for (int pass = 0; pass < 2 && at_b < 0; ++pass) {
    for (int b0 = 0; b0 < a.c.B && at_b < 0; b0 += 32) {
      TcaSeq mine{0, 0, 0, 0, 0};
      if (b0 + lane < a.c.B) mine = tca_seq(a, b0 + lane);
      unsigned some = __ballot_sync(0xFFFFFFFFu, mine.groups > 0);
      while (some && at_b < 0) {
        const int f = __ffs(some) - 1;
        some &= some - 1;
        const int n = __shfl_sync(0xFFFFFFFFu, mine.n, f), len = __shfl_sync(0xFFFFFFFFu, mine.len, f);
        const int rows = __shfl_sync(0xFFFFFFFFu, mine.rows, f), groups = __shfl_sync(0xFFFFFFFFu, mine.groups, f);
        for (int g0 = 0; g0 < groups; g0 += 32) {
          const int tiles = g0 + lane < groups ? tca_steps(a, n, len, rows, g0 + lane).y : 0;
          long long incl = static_cast<long long>(tiles) * a.c.H;
          if (pass == 0) {
            total += incl;
            continue;
          }
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += t;
          }
          const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + incl > p0);
          if (hit) {
            const int l = __ffs(hit) - 1;
            at_tiles = __shfl_sync(0xFFFFFFFFu, tiles, l);
            const long long off =
                p0 - before - __shfl_sync(0xFFFFFFFFu, incl - static_cast<long long>(tiles) * a.c.H, l);
            at_b = b0 + f;
            at_g = g0 + l;
            at_h = static_cast<int>(off / at_tiles);
            at_z = static_cast<int>(off % at_tiles);
            break;
          }
          before += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
      }
    }
    if (pass == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
      chunk = max(static_cast<long long>(kTcaMinTiles), (total + gridDim.x - 1) / gridDim.x);
      p0 = chunk * blockIdx.x;
      if (p0 >= total) break;
    }
  }
  if (lane == 0) {
    sh[0] = at_b;
    sh[1] = at_g;
    sh[2] = at_h;
    sh[3] = at_z;
    sh[4] = at_b < 0 ? 0 : static_cast<int>(min(chunk, total - p0));
    a.plan[2 * blockIdx.x] = make_int4(at_b, at_g * kTcaGroup, at_h, at_z);
    a.plan[2 * blockIdx.x + 1] = make_int4(at_tiles, static_cast<int>(chunk), 0, 0);
  }
}

template <int D>
struct TcaCfg {
  static constexpr int Op = kTcaTile * D * 2;            // bytes of one fp16 operand tile
  static constexpr int OQ = 0, OK = 2 * Op, OV = 4 * Op, OMeta = 6 * Op;
  static constexpr int OBar = OMeta + kTcaMeta * 8 * 16;
  static constexpr int Bars = 17;
  static constexpr int Smem = 1024 + OBar + 8 * Bars + 64;
  static constexpr int Columns = 512;
  static constexpr int SlotFloats = kTcaGroup * (D + 2);
};

template <int D>
__global__ void __launch_bounds__(kTcaThreads, 1) kv_attn_tc_kernel(const KvAttnArgs a) {
  using C = TcaCfg<D>;
  constexpr int KB = D / 64;         // 64-value blocks of a row
  constexpr int Block = kTcaTile * 128;   // bytes of one block of an operand tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t bars = base + C::OBar;
  const uint32_t kfull = bars, kempty = bars + 16, vfull = bars + 32, vempty = bars + 48;   // [2] stages
  const uint32_t qfull = bars + 64, sfull = bars + 80, pfull = bars + 96, odone = bars + 112;   // [2] tiles
  const uint32_t drained = bars + 128;
  volatile int* sh = reinterpret_cast<volatile int*>(smem + C::OBar + 8 * C::Bars);
  const uint32_t tslot = base + C::OBar + 8 * C::Bars + 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + 8 * i, 4);
      mbar_init(kempty + 8 * i, 1);
      mbar_init(vfull + 8 * i, 4);
      mbar_init(vempty + 8 * i, 1);
      mbar_init(qfull + 8 * i, 4);
      mbar_init(sfull + 8 * i, 2);   // the product, and the issuing thread (it saw the step's scales)
      mbar_init(pfull + 8 * i, 4);
      mbar_init(odone + 8 * i, 1);
    }
    mbar_init(drained, 1);
    fence_mbarrier_init();
  }
  if (warp == 12) {
    tmem_alloc(tslot, C::Columns);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_launch();
  if (warp == 0) tca_locate(a, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (tslot - base));
  TcaCursor cur;
  cur.b = sh[0];
  cur.g = sh[1];
  cur.h = sh[2];
  cur.z = sh[3];
  cur.left = sh[4];
  if (cur.left > 0) {
    cur.s = tca_seq(a, cur.b);
    cur.unit(a);
  }

  if (warp < 8) {
    // ------------------------------------------------ rows: weights
    const int tile = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // 32 lanes of tensor memory a warp
    const uint32_t ts = tmem + lanes + tile * 128, to = tmem + lanes + 256 + tile * D;
    bool ok = true;
    int ph_s = 0, ph_o = 0, step = 0, seg = 0;
    while (cur.left > 0) {
      const int n = cur.steps();
      const int row0 = cur.g * kTcaGroup;
      if (row0 + tile * kTcaRows < cur.s.rows) {
        const int row = row0 + tile * kTcaRows + r;
        const bool live = row < cur.s.rows;
        const int rr = min(row, cur.s.rows - 1);
        const int tok = rr / a.G, hq = cur.h * a.G + rr % a.G;
        const int pos = cur.s.len - cur.s.n + tok;
        const int hi = a.causal ? min(pos, cur.s.len - 1) : cur.s.len - 1;
        const int lo = a.window > 0 ? pos - a.window + 1 : 0;
        // ---- Q: scaled by a power of two to fp16
        float coef;
        {
          const uint4* qp = reinterpret_cast<const uint4*>(a.q + (cur.s.begin + tok) * a.ldq + static_cast<long long>(hq) * D);
          uint8_t* qs = smem + C::OQ + tile * C::Op + (r >> 3) * 1024 + (r & 7) * 128;
          uint4 w[D / 8];
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) w[i] = live ? qp[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) m = max(m, bf16x8_finite_amax(w[i]));
          const int e = max(-110, static_cast<int>(m >> 7) - 127);
          const float up = __int_as_float((14 - e + 127) << 23);
          coef = __int_as_float((e - 14 + 127) << 23) * a.scale;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            float f[8];
            bf16x8_to_f32(w[i], f);
            const uint4 v = make_uint4(pack_f16x2(f[0] * up, f[1] * up), pack_f16x2(f[2] * up, f[3] * up),
                                       pack_f16x2(f[4] * up, f[5] * up), pack_f16x2(f[6] * up, f[7] * up));
            *reinterpret_cast<uint4*>(qs + (i >> 3) * Block + (((i & 7) ^ (r & 7)) << 4)) = v;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(qfull + 8 * tile);
        }
        float M = -INFINITY, l = 0.0f;
        for (int j = 0; j < n; ++j) {
          if (ok) ok = mbar_wait(sfull + 8 * tile, ph_s, kSiteKvAccum);
          ph_s ^= 1;
          tc_fence_after();
          const int t = (cur.t0 + cur.z + j) * kTcaTile;
          const KvScale* meta = reinterpret_cast<const KvScale*>(smem + C::OMeta) + ((step + j) % kTcaMeta) * 8;
          const bool whole = __all_sync(0xFFFFFFFFu, t >= lo && t + kTcaTile - 1 <= hi);
          // ---- maximum of the exponents
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(ts + 32 * c, v);
            tmem_wait_ld();
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
              const KvScale sc = meta[2 * c + hb];
              const float ck = coef * sc.k;
              const uint64_t ck2 = f32x2(ck, ck), lv2 = f32x2(sc.lv, sc.lv);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                float2 e = f32x2_split(fma_f32x2(f32x2(__uint_as_float(v[16 * hb + i]), __uint_as_float(v[16 * hb + i + 1])), ck2, lv2));
                if (!whole) {
                  const int at = t + 32 * c + 16 * hb + i;
                  if (at > hi || at < lo) e.x = -INFINITY;
                  if (at + 1 > hi || at + 1 < lo) e.y = -INFINITY;
                }
                mx = fmaxf(mx, fmaxf(e.x, e.y));
              }
            }
          }
          if (__any_sync(0xFFFFFFFFu, mx > M + (kKvBias + kKvLazy))) {
            const float Mn = mx > M + (kKvBias + kKvLazy) ? mx - kKvBias : M;
            const float f = Mn == M ? 1.0f : ex2(M - Mn);   // 0 from nothing
            M = Mn;
            l *= f;
            if (j > 0) {   // the products before this S are complete
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32], u[16];
                tmem_ld_32x32b_x32(to + 32 * c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                tmem_st_32x32b_x16(to + 32 * c, u);
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(v[16 + i]) * f);
                tmem_st_32x32b_x16(to + 32 * c + 16, u);
              }
            }
          }
          // ---- weights, their sum, and P
          const float Ms = M == -INFINITY ? 0.0f : M;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32], p[16];
            tmem_ld_32x32b_x32(ts + 32 * c, v);
            tmem_wait_ld();
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
              const KvScale sc = meta[2 * c + hb];
              const float ck = coef * sc.k, of = sc.lv - Ms;
              const uint64_t ck2 = f32x2(ck, ck), of2 = f32x2(of, of);
              uint64_t sum = 0;
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                float2 e = f32x2_split(fma_f32x2(f32x2(__uint_as_float(v[16 * hb + i]), __uint_as_float(v[16 * hb + i + 1])), ck2, of2));
                if (!whole) {
                  const int at = t + 32 * c + 16 * hb + i;
                  if (at > hi || at < lo) e.x = -INFINITY;
                  if (at + 1 > hi || at + 1 < lo) e.y = -INFINITY;
                }
                const float x = ex2(e.x), y = ex2(e.y);
                sum = add_f32x2(sum, f32x2(x, y));
                p[8 * hb + i / 2] = pack_f16x2(x, y);
              }
              const float2 s2 = f32x2_split(sum);
              l = fmaf(s2.x + s2.y, sc.iv, l);
            }
            tmem_st_32x32b_x16(ts + 16 * c, p);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull + 8 * tile);
          // the phase of odone for this step passes whether or not it is waited for
          if (j + 1 < n) ph_o ^= 1;
        }
        if (ok) ok = mbar_wait(odone + 8 * tile, ph_o, kSiteKvAccum);
        ph_o ^= 1;
        tc_fence_after();
        const bool split = n < cur.tiles;
        float* slot = a.part + (static_cast<long long>(blockIdx.x) * 2 + (seg > 0 ? 1 : 0)) * C::SlotFloats;
        const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;
        __nv_bfloat16* op = a.out + (cur.s.begin + tok) * a.ldo + static_cast<long long>(hq) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(to + 32 * c, v);
          tmem_wait_ld();
          if (!live || !ok) continue;
          if (split) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              kv_put_partial(slot, kTcaGroup, row - row0, 32 * c + i,
                             make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]),
                                         __uint_as_float(v[i + 3])));
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16x2(__uint_as_float(v[i + 2 * k]) * inv, __uint_as_float(v[i + 2 * k + 1]) * inv);
              *reinterpret_cast<uint4*>(op + 32 * c + i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        tc_fence_before();
        if (live && ok) {
          if (split)
            reinterpret_cast<float2*>(slot + kTcaGroup * D)[row - row0] = make_float2(M, l);
          else if (a.lse != nullptr)
            a.lse[(cur.s.begin + tok) * static_cast<long long>(a.Hq) + hq] =
                l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.693147180559945f;
        }
      }
      step += n;
      ++seg;
      cur.next(a);
    }
  } else if (warp < 12) {
    // ------------------------------------------------ codes to fp16
    const int pt = tid - 256;
    constexpr int Pieces = D / 16;                 // 16-byte pieces of a token's codes
    constexpr int Per = kTcaTile * Pieces / 128;   // pieces of a thread
    constexpr int Step = 128 / Pieces;             // tokens between them
    const int c = pt % Pieces, tk = pt / Pieces;
    bool ok = true;
    int step = 0;
    while (cur.left > 0) {
      const int n = cur.steps();
      // lane l < 8: the 16 tokens from 16 l on of a step
      auto look = [&](int j, int& row, KvScale& sc) {
        row = -1;
        sc = kv_scale_of(0.0f, 0.0f);
        sc.lv = -INFINITY;
        const int t = (cur.t0 + cur.z + j) * kTcaTile + 16 * lane;
        if (j < n && lane < 8 && t < cur.s.len) {
          const int page = kv_page(a.c, cur.b, t);
          if (page >= 0) {
            const int phd = page * a.c.H + cur.h;
            row = phd * a.c.P + t % a.c.P;
            if (warp == 8) sc = kv_scale_of(a.c.k_scale[phd], a.c.v_scale[phd]);
          }
        }
      };
      auto fetch = [&](const int8_t* codes, int row, uint4 (&w)[Per]) {
#pragma unroll
        for (int i = 0; i < Per; ++i) {
          const int t = tk + Step * i;
          const int rw = __shfl_sync(0xFFFFFFFFu, row, t / 16);
          w[i] = make_uint4(0u, 0u, 0u, 0u);   // tokens of no page: zeros, whatever weight is 0 times them
          if (rw >= 0) w[i] = reinterpret_cast<const uint4*>(codes + static_cast<long long>(rw + t % 16) * D)[c];
        }
      };
      auto widen = [&](uint8_t* to, const uint4 (&w)[Per]) {
#pragma unroll
        for (int i = 0; i < Per; ++i) {
          const int t = tk + Step * i;
          uint8_t* p = to + (c >> 2) * Block + (t >> 3) * 1024 + (t & 7) * 128;
          const uint32_t x[4] = {w[i].x ^ 0x80808080u, w[i].y ^ 0x80808080u, w[i].z ^ 0x80808080u, w[i].w ^ 0x80808080u};
          const uint4 lo = make_uint4(codes_f16x2<0>(x[0]), codes_f16x2<1>(x[0]), codes_f16x2<0>(x[1]), codes_f16x2<1>(x[1]));
          const uint4 hi = make_uint4(codes_f16x2<0>(x[2]), codes_f16x2<1>(x[2]), codes_f16x2<0>(x[3]), codes_f16x2<1>(x[3]));
          const int p0 = 2 * (c & 3);
          // the two blocks of a row lie on the same banks: their lanes store the other half first
          const bool flip = c >= 4;
          *reinterpret_cast<uint4*>(p + (((flip ? p0 + 1 : p0) ^ (t & 7)) << 4)) = flip ? hi : lo;
          *reinterpret_cast<uint4*>(p + (((flip ? p0 : p0 + 1) ^ (t & 7)) << 4)) = flip ? lo : hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      int row, row_n;
      KvScale sc, sc_n;
      uint4 wk[Per], wv[Per];
      look(0, row, sc);
      fetch(a.c.k, row, wk);
      for (int j = 0; j < n; ++j, ++step) {
        const int st = step & 1, par = ((step >> 1) & 1) ^ 1;
        fetch(a.c.v, row, wv);
        look(j + 1, row_n, sc_n);
        if (ok) ok = mbar_wait(kempty + 8 * st, par, kSiteKvFree);
        if (warp == 8 && lane < 8)
          reinterpret_cast<KvScale*>(smem + C::OMeta)[(step % kTcaMeta) * 8 + lane] = sc;
        widen(smem + C::OK + st * C::Op, wk);
        if (lane == 0) mbar_arrive(kfull + 8 * st);
        if (j + 1 < n) fetch(a.c.k, row_n, wk);
        if (ok) ok = mbar_wait(vempty + 8 * st, par, kSiteKvFree);
        widen(smem + C::OV + st * C::Op, wv);
        if (lane == 0) mbar_arrive(vfull + 8 * st);
        row = row_n;
        sc = sc_n;
      }
      cur.next(a);
    }
  } else if (lane == 0) {
    // ------------------------------------------------ tensor core
    constexpr uint32_t is = umma_idesc_f16(kTcaRows, kTcaTile, false), io = umma_idesc_f16(kTcaRows, D, true);
    bool ok = true;
    int step = 0, ph_q[2] = {0, 0}, ph_p[2] = {0, 0}, ph_o[2] = {0, 0};
    auto scores = [&](int tile, int st) {
      tc_fence_after();
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_bf16(tmem + tile * 128, umma_desc_sw128(base + C::OQ + tile * C::Op + kb * Block + 32 * k),
                      umma_desc_sw128(base + C::OK + st * C::Op + kb * Block + 32 * k), is, kb + k > 0);
      mbar_arrive(sfull + 8 * tile);
      tc_commit(sfull + 8 * tile);
    };
    while (cur.left > 0 && ok) {
      const int n = cur.steps();
      const int nt = cur.g * kTcaGroup + kTcaRows < cur.s.rows ? 2 : 1;
      ok = mbar_wait(kfull + 8 * (step & 1), (step >> 1) & 1, kSiteKvLoad);
      for (int t = 0; t < nt && ok; ++t) {
        ok = mbar_wait(qfull + 8 * t, ph_q[t], kSiteKvLoad);
        ph_q[t] ^= 1;
        if (ok) scores(t, step & 1);
      }
      if (ok) tc_commit(kempty + 8 * (step & 1));
      for (int j = 0; j < n && ok; ++j, ++step) {
        const int st = step & 1, nx = (step + 1) & 1;
        ok = mbar_wait(vfull + 8 * st, (step >> 1) & 1, kSiteKvLoad);
        for (int t = 0; t < nt && ok; ++t) {
          ok = mbar_wait(pfull + 8 * t, ph_p[t], kSiteKvAccum);
          ph_p[t] ^= 1;
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kTcaTile / 16; ++k)
            tc_mma_f16_ta(tmem + 256 + t * D, tmem + t * 128 + 8 * k,
                          umma_desc_sw128_n(base + C::OV + st * C::Op + 2048 * k, Block), io, j + k > 0);
          tc_commit(odone + 8 * t);
          if (j + 1 < n) {
            if (t == 0) ok = mbar_wait(kfull + 8 * nx, ((step + 1) >> 1) & 1, kSiteKvLoad);
            if (ok) ok = mbar_wait(odone + 8 * t, ph_o[t], kSiteKvAccum);   // S takes the place of P
            if (ok) scores(t, nx);
          }
          ph_o[t] ^= 1;
        }
        if (ok) {
          tc_commit(vempty + 8 * st);
          if (j + 1 < n) tc_commit(kempty + 8 * nx);
        }
      }
      cur.next(a);
    }
    // nothing issued here may still run when the tensor memory is given back
    tc_commit(drained);
    mbar_wait(drained, 0, kSiteKvAccum);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, C::Columns);
}

}  // namespace respin
