// Attention of a ragged batch of queries over the 8-bit paged cache, for few
// rows a key head (single tokens, short drafts): the cache is streamed once.
//
//   s_j = (q . k_j) * scale,  out = sum_j softmax(s)_j v_j,  lse = log sum_j e^(s_j)
//
// Numbers. Codes are whole numbers up to 127 and exact in fp16; so are a row
// of q scaled by a power of two (amax to [2^14, 2^15)) down to 2^-31 of its
// amax; smaller values of q are off by 2^-39 of it at most. The products of the tensor cores are then exact and summed in fp32,
// and the page's scale is applied to the sum. The weights of a page carry
// its v scale: p_j = 2^(s_j log2 e + log2 vs - M), M a running maximum of
// that exponent, so p <= 2^15 fits fp16 and the accumulators need no scale of
// their own; the sum l = sum p_j ref / vs takes them in fp32 before the rounding.
// ref is a value scale near those of the unit, so that neither the sum nor 1 / vs
// leaves binary32 however small or large the values are: out = O / l * ref,
// lse = M + log2 l - log2 ref (times ln 2).
// Rounding p to fp16 is the one loss: half a step is 2^-11 of each weight
// down to 2^-20 of the largest, and 2^-31 of the largest below (bf16 would
// lose 2^-8), beside the 2^-8 of the bf16 output. (The largest is 2^6 at least.
// With 2^2 and a lag of 2^13 weights below 2^-27 of it were lost; wide logits
// rescale more often now, see kv_attention_tc.cuh, decode takes the same time.)
//
// Layout. A warp takes 16 tokens of a 64-token tile and 8 rows at a time with
// the transposed products S^T = K Q^T and O^T = V^T P^T: with at most 8 rows
// (one n = 8 instruction) nothing is multiplied for absent rows, and the
// codes are the A operand, whose fragments come straight from 16-byte reads
// of the tile, because the order of the summed index and of the output rows
// is free: a thread's 32 consecutive dims of K are four-byte steps of k, and
// its 16 consecutive dims of V are the rows of eight tiles. P^T needs one
// transposition in registers (movmatrix).
//
// Work. The tiles of all (sequence, head, row group)s form one line that is
// cut into equal pieces, one per block, so long and short sequences balance
// without the host knowing a length. A piece that ends inside a line's unit
// leaves its out and log2 of its sum in the workspace; kv_combine_kernel joins those.
//
// Bound: the cache's bytes. Four consumer warps and a producer warp (tensor
// copies through a ring of kKvStages tiles of 2 * 64 * D bytes), three blocks
// an SM (two with four stages: 75 us where three take 66). 64 sequences of 32
// query heads over 8 at 4096 tokens: 97 us, 5.5 TB/s with the join; two of 64
// over 8 at 131071: 92 us, 5.8 TB/s, and 11 us for the join of 28 pieces a unit.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "kv_cache.cuh"
#include "ptx.cuh"

namespace respin {

constexpr int kKvTile = 64;          // tokens of a tile
constexpr int kKvStages = 3;         // three blocks fit an SM (66 KB each at D = 128)
constexpr int kKvWarps = 4;          // consumer warps, 16 tokens each
constexpr int kKvThreads = (kKvWarps + 1) * 32;
constexpr int kKvMaxBlocks = 592;    // 4 per SM
constexpr int kKvMinTiles = 4;       // least piece of a block
// Rows a key head up to which a sequence is this kernel's: what it is built for. kv_attention_tc.cuh takes
// longer at 16 rows and below: 64 sequences at 4096 tokens, 8 key heads of 128, 16 rows 240 us (here 170),
// 12 rows 154 (107), 8 rows 236 (86); heads of 64 215 (78); one sequence of 200 tokens 24.6 (18.0).
constexpr int kKvFewRows = 16;
constexpr int kKvPlan = 3;           // int4s a block leaves about its piece (KvJoin)
constexpr float kKvBias = 6.0f;      // p <= 2^(kKvBias + kKvLazy) = 2^15 in fp16
constexpr float kKvLazy = 9.0f;      // the running maximum may lag by 2^9

struct KvAttnArgs {
  KvView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;            // or null
  long long ldq, ldo;    // elements between tokens
  int Hq, G;             // query heads; per key head
  int causal, window;
  float scale;           // times log2 e
  unsigned long long div_g;   // ceil(2^64 / G), 0 for G = 1
  int few_rows;          // sequences of more rows (tokens * G) are another kernel's
  int others;            // whether that kernel runs; else such a sequence is refused
  int4* plan;            // workspace: [blocks][kKvPlan] where a block's piece begins
  float* part;           // workspace: [blocks][2] partial results
};

// n / G, n >= 0: the multiplier is off by less than G / 2^64 of itself, so the
// product's integer part is exact for any 32-bit n.
__device__ __forceinline__ int kv_div_g(const KvAttnArgs& a, int n) {
  return a.div_g == 0 ? n : static_cast<int>(__umul64hi(static_cast<unsigned long long>(n), a.div_g));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 1024 + u -> u - 128 in both halves (u = code + 128): exact.
__device__ __forceinline__ uint32_t unbias_f16x2(uint32_t x) {
  const uint32_t k = 0x64806480u;   // 1152
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&k));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Codes of bytes 2i, 2i + 1 of w (biased by an XOR with 0x80 before) as fp16.
template <int I>
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t w) {
  return unbias_f16x2(__byte_perm(w, 0x64646464u, I == 0 ? 0x4140 : 0x4342));
}

// Codes of byte I of a (low half) and of b (high half) as fp16.
template <int I>
__device__ __forceinline__ uint32_t codes_pair_f16x2(uint32_t a, uint32_t b) {
  const uint32_t y = __byte_perm(a, b, I | (4 + I) << 8);   // bytes 1 and 3: anything
  return unbias_f16x2((y & 0x00FF00FFu) ^ 0x64806480u);
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// What a page's 16 tokens need of its scales.
struct KvScale {
  float k;        // k scale
  float lv;       // log2 of the v scale; -inf: tokens of a bad page, left out
  float iv;       // ref / v scale
  float ref;      // the largest v scale of the unit's first looked-up pages; 1 where those are all 0
};

// A v scale counts as at least 2^-64 of ref: one of 0 goes with codes of 0, so
// any positive number stands for it, and this one keeps the page's weights in
// range beside pages whose scales are up to 2^64 smaller than ref. (Values of a
// smaller scale are off by less than 2^-57 ref.)
__device__ __forceinline__ KvScale kv_scale_of(float ks, float vs, float ref) {
  KvScale s;
  const float v = fmaxf(vs, fmaxf(ref * 5.421010862427522e-20f, 1.17549435e-38f));
  s.k = ks;
  s.lv = __log2f(v);
  s.iv = __fdiv_rn(ref, v);
  s.ref = ref;
  return s;
}

// Partial results: [D / 4][rows] float4 (the piece's out), then [rows] log2 of
// its sum of exponentials.
__device__ __forceinline__ void kv_put_partial(float* slot, int rows, int row, int d, float4 v) {
  reinterpret_cast<float4*>(slot)[(d / 4) * rows + row] = v;
}

// The line of work: sequence b has units (row group, head) of `tiles` tiles
// each, in this order.
struct KvSeq {
  int begin, rows, len;   // first row of the batch, rows * G, length
  int groups;             // row groups of RB rows
  int t0, tiles;          // first tile and tiles of each unit (at least 1 where there are rows)
  int low;                // first token that any row sees
};

template <int RB>
__device__ __forceinline__ KvSeq kv_seq(const KvAttnArgs& a, int b) {
  KvSeq s;
  int end;
  kv_rows(a.c, b, s.begin, end, s.len);
  const int n = end - s.begin;
  s.rows = n * a.G;
  if (s.rows > a.few_rows) {
    if (!a.others) record_status(kSiteKvLength);
    s.rows = 0;
  }
  s.groups = (s.rows + RB - 1) / RB;
  const int first = s.len - n;   // position of the first row
  s.low = a.window > 0 ? max(0, first - a.window + 1) : 0;
  s.t0 = min(s.low, s.len) / kKvTile;
  s.tiles = max(1, (s.len + kKvTile - 1) / kKvTile - s.t0);
  return s;
}

template <int RB>
__device__ __forceinline__ long long kv_weight(const KvAttnArgs& a, int b) {
  const KvSeq s = kv_seq<RB>(a, b);
  return static_cast<long long>(s.groups) * a.c.H * s.tiles;
}

template <int D, int NT>
struct KvAttnCfg {
  static constexpr int RB = 8 * NT;                       // rows of a group
  static constexpr int Half = kKvTile * D;                // bytes of K (or V) of a tile
  static constexpr int Stage = 2 * Half;
  static constexpr int Pitch = D + 4;                     // floats of a row of the joined output
  static constexpr int Join = kKvWarps * 8 * Pitch * 4 + kKvWarps * 8 * 8;
  static constexpr int Meta = kKvStages * 4 * 16;         // KvScale of each 16 tokens
  static constexpr int Smem = 1024 + kKvStages * Stage + Join + Meta + 2 * 8 * kKvStages + 64;
  static constexpr int SlotFloats = RB * (D + 1);         // a partial result
};

// tmK, tmV: uint8 [pages * H * P, D], box {D, min(P, 64)}, swizzle of D bytes.
template <int D, int NT>
__global__ void __launch_bounds__(kKvThreads)
kv_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const KvAttnArgs a) {
  using C = KvAttnCfg<D, NT>;
  constexpr int KS = D / 16;       // k steps of S^T, m tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t o_join = kKvStages * C::Stage, o_meta = o_join + C::Join, o_bar = o_meta + C::Meta;
  const uint32_t full0 = base + o_bar, empty0 = full0 + 8 * kKvStages;
  volatile int* sh = reinterpret_cast<volatile int*>(smem + o_bar + 16 * kKvStages);   // [16]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, kKvWarps);
    }
    fence_mbarrier_init();
  }
  grid_dep_wait();
  grid_dep_launch();

  // ---- this block's piece of the line
  if (warp == 0) {
    constexpr int kKept = 4;   // weights of the first 128 sequences stay in registers for the second look
    long long total = 0, kept[kKept];
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      kept[i] = 32 * i + lane < a.c.B ? kv_weight<C::RB>(a, 32 * i + lane) : 0;
      total += kept[i];
    }
    for (int b = 32 * kKept + lane; b < a.c.B; b += 32) total += kv_weight<C::RB>(a, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    const long long g = gridDim.x;
    const long long chunk = max(static_cast<long long>(kKvMinTiles), (total + g - 1) / g);
    const long long p0 = chunk * blockIdx.x;
    const long long left = min(chunk, total - p0);
    int b_at = a.c.B;
    long long off = 0;
    if (left > 0) {
      long long before = 0;
      for (int b0 = 0; b0 < a.c.B; b0 += 32) {
        long long w = 0;
#pragma unroll
        for (int i = 0; i < kKept; ++i)
          if (b0 == 32 * i) w = kept[i];
        if (b0 >= 32 * kKept && b0 + lane < a.c.B) w = kv_weight<C::RB>(a, b0 + lane);
        long long incl = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += t;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + incl > p0);
        if (hit) {
          const int f = __ffs(hit) - 1;
          b_at = b0 + f;
          off = p0 - (before + __shfl_sync(0xFFFFFFFFu, incl - w, f));
          break;
        }
        before += __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
    }
    if (lane == 0) {
      const long long cap = left > 0 ? left : 0;   // < 2^31: the host bounds the line
      sh[0] = b_at;
      *reinterpret_cast<volatile long long*>(sh + 4) = off;
      sh[2] = static_cast<int>(cap);
      const long long from = min(p0, total);
      int4 pl = make_int4(-1, 0, 0, 0), pm = make_int4(1, static_cast<int>(from & 0xFFFFFFFF), static_cast<int>(from >> 32), 0);
      if (cap > 0) {   // where the piece begins: sequence, row, head, tiles of the unit before it; its tiles
        const KvSeq s = kv_seq<C::RB>(a, b_at);
        const int unit = static_cast<int>(off / s.tiles);
        pl = make_int4(b_at, unit / a.c.H * C::RB, unit % a.c.H, static_cast<int>(off % s.tiles));
        pm.x = s.tiles;
        pm.w = 1 + static_cast<int>((s.tiles - pl.w + chunk - 1) / chunk);
        a.plan[kKvPlan * blockIdx.x + 2] = make_int4(s.begin, s.rows, 0, 0);
      }
      a.plan[kKvPlan * blockIdx.x] = pl;
      a.plan[kKvPlan * blockIdx.x + 1] = pm;
    }
  }
  __syncthreads();
  int b = sh[0], left = sh[2];
  long long off = *reinterpret_cast<volatile long long*>(sh + 4);   // tiles of sequence b before the piece
  if (left <= 0) return;

  if (warp == kKvWarps) {
    // ------------------------------------------------ producer
    const int SP = min(a.c.P, kKvTile), nsub = kKvTile / SP;
    int stage = 0, phase = 0, issued = 0;
    bool ok = true;
    while (left > 0 && b < a.c.B && ok) {
      const KvSeq s = kv_seq<C::RB>(a, b);
      const int unit = static_cast<int>(off / s.tiles), t = static_cast<int>(off % s.tiles);
      const int n = min(left, s.tiles - t);
      const int h = unit % a.c.H;
      const int batch = 32 / nsub;   // tiles whose pages a lane each looks up at once
      float ref = 1.0f;
      for (int i0 = 0; i0 < n && ok; i0 += batch) {
        // lane: sub-box `lane` of the batch
        const int tok = (s.t0 + t + i0) * kKvTile + lane * SP;
        int row = -1;
        float ks = 0.0f, vs = 0.0f;
        if (tok < s.len && tok + SP > s.low && lane / nsub < n - i0) {   // (pages behind the window may be gone)
          const int page = kv_page(a.c, b, tok);
          if (page >= 0) {
            const int ph = page * a.c.H + h;
            row = ph * a.c.P + tok % a.c.P;
            ks = a.c.k_scale[ph];
            vs = a.c.v_scale[ph];
          }
        }
        if (i0 == 0) {
          const float most = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, vs > 0.0f ? __float_as_uint(vs) : 0u));
          if (most > 0.0f) ref = most;
        }
        KvScale sc = kv_scale_of(ks, vs, ref);
        if (row < 0) sc.lv = -INFINITY;
        for (int i = i0; i < min(n, i0 + batch) && ok; ++i) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty0 + 8 * stage, phase ^ 1, kSiteKvFree));
          if (!ok) break;
          const int l0 = (i - i0) * nsub;
          const bool mine = lane >= l0 && lane < l0 + nsub;
          KvScale* meta = reinterpret_cast<KvScale*>(smem + o_meta) + stage * 4;
          if (mine)
            for (int j = 0; j < SP / 16; ++j) meta[(lane - l0) * (SP / 16) + j] = sc;
          const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, mine && row >= 0));
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(full0 + 8 * stage, static_cast<uint32_t>(2 * boxes * SP * D));
          __syncwarp();
          if (mine && row >= 0) {
            const uint32_t dst = base + stage * C::Stage + (lane - l0) * SP * D;
            tma_load_2d(dst, &tmK, 0, row, full0 + 8 * stage);
            tma_load_2d(dst + C::Half, &tmV, 0, row, full0 + 8 * stage);
          }
          if (++stage == kKvStages) { stage = 0; phase ^= 1; }
          ++issued;
        }
      }
      left -= n;
      off += n;
      if (off >= static_cast<long long>(s.groups) * a.c.H * s.tiles) {
        off = 0;
        do { ++b; } while (b < a.c.B && left > 0 && kv_seq<C::RB>(a, b).groups == 0);
      }
    }
    // leave only once the last copies have landed, whatever became of the consumers
    for (int i = max(0, issued - kKvStages); i < issued; ++i)
      mbar_wait(full0 + 8 * (i % kKvStages), (i / kKvStages) & 1, kSiteKvLoad);
    return;
  }

  // -------------------------------------------------- consumers
  const int r = lane >> 2, qd = lane & 3;   // fragment row / column group
  const int Gq = a.G;
  int stage = 0, phase = 0, seg = 0;
  bool ok = true;
  while (left > 0 && b < a.c.B) {
    const KvSeq s = kv_seq<C::RB>(a, b);
    const int unit = static_cast<int>(off / s.tiles), t = static_cast<int>(off % s.tiles);
    const int n = min(left, s.tiles - t);
    const int h = unit % a.c.H, row0 = (unit / a.c.H) * C::RB;
    const int first_pos = s.len - s.rows / Gq;   // of the sequence's first row

    // Q^T fragments: row n = lane / 4 of each group of 8, scaled by a power of two
    uint32_t qf[NT][KS][2];
    float coef[NT][2];     // for the rows (columns of S^T) 2 qd, 2 qd + 1
    int hi[NT][2], lo[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      const int row = row0 + 8 * x + r;
      float down = 0.0f;   // an absent row: zeros, weights of no use
      if (row < s.rows) {
        const __nv_bfloat16* qp = a.q + (s.begin + row / Gq) * a.ldq + static_cast<long long>(h * Gq + row % Gq) * D + qd * (D / 4);
        uint4 w[D / 32];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          w[i] = reinterpret_cast<const uint4*>(qp)[i];
          m = max(m, bf16x8_finite_amax(w[i]));
        }
        m = max(m, __shfl_xor_sync(0xFu << (lane & ~3), m, 1));
        m = max(m, __shfl_xor_sync(0xFu << (lane & ~3), m, 2));
        // exponent e of the amax: q * 2^(14 - e); e held to where both powers are normal
        const int e = max(-110, static_cast<int>(m >> 7) - 127);
        const float up = __int_as_float((14 - e + 127) << 23);
        down = __int_as_float((e - 14 + 127) << 23);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float f[8];
          bf16x8_to_f32(w[i], f);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            qf[x][2 * i + j / 2][j & 1] = pack_f16x2(f[2 * j] * up, f[2 * j + 1] * up);
        }
      } else {
#pragma unroll
        for (int i = 0; i < KS; ++i) qf[x][i][0] = qf[x][i][1] = 0u;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        coef[x][j] = __shfl_sync(0xFFFFFFFFu, down, (2 * qd + j) * 4) * a.scale;
        const int rr = min(row0 + 8 * x + 2 * qd + j, s.rows - 1);
        const int pos = first_pos + rr / Gq;
        hi[x][j] = a.causal ? min(pos, s.len - 1) : s.len - 1;
        lo[x][j] = a.window > 0 ? pos - a.window + 1 : 0;
      }
    }
    // limits that hold for every row of the group: no mask inside them
    const int last = min(row0 + C::RB, s.rows) - 1;
    const int all_hi = a.causal ? min(first_pos + row0 / Gq, s.len - 1) : s.len - 1;
    const int all_lo = a.window > 0 ? first_pos + last / Gq - a.window + 1 : 0;
    // tokens that some row sees
    const int any_hi = a.causal ? min(first_pos + last / Gq, s.len - 1) : s.len - 1;
    const int any_lo = a.window > 0 ? first_pos + row0 / Gq - a.window + 1 : 0;

    float acc[NT][KS][4];
    float M[NT][2], l[NT][2], ref = 1.0f;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[x][i][j] = 0.0f;
      M[x][0] = M[x][1] = -INFINITY;
      l[x][0] = l[x][1] = 0.0f;
    }

    for (int i = 0; i < n; ++i) {
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(full0 + 8 * stage, phase, kSiteKvLoad));
      if (i == 0 && ok) ref = reinterpret_cast<const KvScale*>(smem + o_meta)[stage * 4].ref;
      const int tok = (s.t0 + t + i) * kKvTile + warp * 16;
      if (ok && tok <= any_hi && tok + 15 >= any_lo) {
        const KvScale sc = reinterpret_cast<const KvScale*>(smem + o_meta)[stage * 4 + warp];
        const uint32_t kb = base + stage * C::Stage + warp * 16 * D, vb = kb + C::Half;
        // S^T = K Q^T
        float S[NT][4];
#pragma unroll
        for (int x = 0; x < NT; ++x) S[x][0] = S[x][1] = S[x][2] = S[x][3] = 0.0f;
#pragma unroll
        for (int i2 = 0; i2 < D / 64; ++i2) {
          uint32_t w[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int row = r + 8 * u;
            uint32_t at;
            if constexpr (D == 128)
              at = kb + row * 128 + (((2 * qd + i2) ^ (row & 7)) << 4);
            else
              at = kb + row * 64 + ((qd ^ ((row >> 1) & 3)) << 4);
            const uint4 v = lds128(at);
            w[u][0] = v.x ^ 0x80808080u;
            w[u][1] = v.y ^ 0x80808080u;
            w[u][2] = v.z ^ 0x80808080u;
            w[u][3] = v.w ^ 0x80808080u;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t af[4] = {codes_f16x2<0>(w[0][k]), codes_f16x2<0>(w[1][k]), codes_f16x2<1>(w[0][k]),
                                    codes_f16x2<1>(w[1][k])};
#pragma unroll
            for (int x = 0; x < NT; ++x) mma_f16_16816(S[x], af, qf[x][4 * i2 + k][0], qf[x][4 * i2 + k][1]);
          }
        }
        // weights
        const bool whole = tok + 15 <= all_hi && tok >= all_lo;
        uint32_t pf[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = fmaf(S[x][j], coef[x][j & 1] * sc.k, sc.lv);
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int at = tok + r + 8 * (j >> 1);
              if (at > hi[x][j & 1] || at < lo[x][j & 1]) e[j] = -INFINITY;
            }
          }
          const float m0 = fmaxf(e[0], e[2]), m1 = fmaxf(e[1], e[3]);
          // M is the maximum less kKvBias; it moves when a weight would pass 2^(kKvBias + kKvLazy)
          const float over = kKvBias + kKvLazy;
          if (__any_sync(0xFFFFFFFFu, m0 > M[x][0] + over || m1 > M[x][1] + over)) {
            float mm[2] = {m0, m1};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mm[j] = fmaxf(mm[j], __shfl_xor_sync(0xFFFFFFFFu, mm[j], o));
              const float Mn = fmaxf(M[x][j], mm[j] - kKvBias);
              const float f = Mn == -INFINITY ? 0.0f : ex2(M[x][j] - Mn);
              M[x][j] = Mn;
              l[x][j] *= f;
#pragma unroll
              for (int i2 = 0; i2 < KS; ++i2) {
                acc[x][i2][j] *= f;
                acc[x][i2][j + 2] *= f;
              }
            }
          }
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = e[j] == -INFINITY ? 0.0f : ex2(e[j] - M[x][j & 1]);
            l[x][j & 1] = fmaf(p[j], sc.iv, l[x][j & 1]);
          }
          pf[x][0] = transpose_8x8(pack_f16x2(p[0], p[1]));
          pf[x][1] = transpose_8x8(pack_f16x2(p[2], p[3]));
        }
        // O^T += V^T P^T
        uint32_t v[4][D / 32];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = 2 * qd + (u & 1) + 8 * (u >> 1);
          if constexpr (D == 128) {
            const uint4 x = lds128(vb + row * 128 + ((r ^ (row & 7)) << 4));
            v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
          } else {
            const uint2 x = lds64(vb + row * 64 + (((r >> 1) ^ ((row >> 1) & 3)) << 4) + (r & 1) * 8);
            v[u][0] = x.x; v[u][1] = x.y;
          }
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int w = k / 2;
          uint32_t af[4];
          if (k & 1) {
            af[0] = codes_pair_f16x2<2>(v[0][w], v[1][w]);
            af[1] = codes_pair_f16x2<3>(v[0][w], v[1][w]);
            af[2] = codes_pair_f16x2<2>(v[2][w], v[3][w]);
            af[3] = codes_pair_f16x2<3>(v[2][w], v[3][w]);
          } else {
            af[0] = codes_pair_f16x2<0>(v[0][w], v[1][w]);
            af[1] = codes_pair_f16x2<1>(v[0][w], v[1][w]);
            af[2] = codes_pair_f16x2<0>(v[2][w], v[3][w]);
            af[3] = codes_pair_f16x2<1>(v[2][w], v[3][w]);
          }
#pragma unroll
          for (int x = 0; x < NT; ++x) mma_f16_16816(acc[x][k], af, pf[x][0], pf[x][1]);
        }
      }
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(empty0 + 8 * stage);   // (after a wait that gave up: no more signals)
      if (++stage == kKvStages) { stage = 0; phase ^= 1; }
    }

    // ---- join the four warps, 8 rows at a time; write the rows, or a partial result
    const bool split = n < s.tiles;
    float* slot = a.part + (static_cast<long long>(blockIdx.x) * 2 + (seg > 0 ? 1 : 0)) * C::SlotFloats;
    float* jo = reinterpret_cast<float*>(smem + o_join);                 // [warp][8][Pitch]
    float* jm = jo + kKvWarps * 8 * C::Pitch;                            // [warp][8][2]
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      if (row0 + 8 * x >= s.rows) break;
      named_bar_sync(1, kKvWarps * 32);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[x][j] += __shfl_xor_sync(0xFFFFFFFFu, l[x][j], o);
        if (r == 0) {
          jm[(warp * 8 + 2 * qd + j) * 2] = M[x][j];
          jm[(warp * 8 + 2 * qd + j) * 2 + 1] = l[x][j];
        }
        float* at = jo + (warp * 8 + 2 * qd + j) * C::Pitch + r * (D / 8);
#pragma unroll
        for (int k = 0; k < KS; ++k)
          *reinterpret_cast<float2*>(at + 2 * k) = make_float2(acc[x][k][j], acc[x][k][j + 2]);
      }
      named_bar_sync(1, kKvWarps * 32);
      if (!ok) continue;   // a wait gave up: nothing is stored
      // thread: row tid / 16 of 8, dims (tid % 16) * D / 16 ..
      const int row = tid >> 4, d0 = (tid & 15) * (D / 16);
      const int gr = row0 + 8 * x + row;
      if (gr >= s.rows) continue;
      float Mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kKvWarps; ++w) Mx = fmaxf(Mx, jm[(w * 8 + row) * 2]);
      float o[D / 16], ls = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kKvWarps; ++w) {
        const float mw = jm[(w * 8 + row) * 2];
        const float f = mw == -INFINITY ? 0.0f : ex2(mw - Mx);
        ls = fmaf(jm[(w * 8 + row) * 2 + 1], f, ls);
        const float* at = jo + (w * 8 + row) * C::Pitch + d0;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i] = fmaf(at[i], f, o[i]);
      }
      const float inv = ls > 0.0f ? __fdiv_rn(1.0f, ls) : 0.0f;   // a row that sees nothing is 0
      const float L = ls == 0.0f ? -INFINITY : Mx + log2f(ls) - log2f(ref);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i] = o[i] * inv * ref;
      if (split) {
#pragma unroll
        for (int i = 0; i < D / 16; i += 4)
          kv_put_partial(slot, C::RB, 8 * x + row, d0 + i, make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
        if (d0 == 0) slot[C::RB * D + 8 * x + row] = L;
      } else {
        const long long tokr = s.begin + gr / Gq;
        const int hq = h * Gq + gr % Gq;
        uint32_t w[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
        __nv_bfloat16* to = a.out + tokr * a.ldo + static_cast<long long>(hq) * D + d0;
        if constexpr (D == 128) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        if (a.lse != nullptr && d0 == 0) a.lse[tokr * a.Hq + hq] = L * 0.693147180559945f;
      }
    }
    ++seg;
    left -= n;
    off += n;
    if (off >= static_cast<long long>(s.groups) * a.c.H * s.tiles) {
      off = 0;
      do { ++b; } while (b < a.c.B && left > 0 && kv_seq<C::RB>(a, b).groups == 0);
    }
  }
}

// Joins the partial results of units that several blocks of a kernel share.
// Of `blocks` pieces: the unit that piece c begins inside of, if that is the
// second of the unit's pieces; `parts` blocks share its rows and dims.
struct KvJoin {
  // [blocks]: (sequence or -1, first row, head, tiles of the unit before the piece); (the unit's tiles,
  // the line's tiles before the piece in two halves, pieces from the unit's start on or 0: to be
  // counted); (the sequence's first row of the batch, its rows)
  const int4* plan;
  const float* part;
  int blocks, rows;   // pieces; rows of a partial result
  int parts;
};

constexpr int kKvJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kKvJoinThreads) kv_combine_kernel(const KvAttnArgs a, const KvJoin few, const KvJoin many) {
  grid_dep_wait();
  grid_dep_launch();
  const int n_few = max(0, few.blocks - 1) * few.parts, i0 = blockIdx.x;
  const KvJoin j = i0 < n_few ? few : many;
  const int at0 = i0 < n_few ? i0 : i0 - n_few, part = at0 % j.parts, c = at0 / j.parts + 1;
  // (asked for together; the last two are unused where the first says so)
  const int4 pl = j.plan[kKvPlan * c], pm = j.plan[kKvPlan * c + 1], pr = j.plan[kKvPlan * c + 2],
             pb = j.plan[kKvPlan * (c - 1) + 1];
  const int z = pl.w, tiles = pm.x;
  if (pl.x < 0 || z == 0) return;   // no piece, or one that begins with a unit
  // the unit's tiles [u0, u1) of the line; pieces c - 1, c, ... begin at from(c - 1), ...
  auto from = [](const int4& m) { return (static_cast<long long>(m.z) << 32) | static_cast<unsigned>(m.y); };
  const long long u0 = from(pm) - z, u1 = u0 + tiles, f0 = from(pb);
  if (f0 > u0) return;              // a later piece of the unit
  const int begin = pr.x, rows = pr.y - pl.y, RB = j.rows;
  int pieces = pm.w;
  if (pieces == 0) {
    pieces = 1;
    for (int i = c; i < j.blocks; i += 32) {   // 32 looked at in a step
      const int l = i + static_cast<int>(threadIdx.x & 31);
      const int n = __popc(__ballot_sync(0xFFFFFFFFu, l < j.blocks && from(j.plan[kKvPlan * l + 1]) < u1));
      pieces += n;
      if (n < 32) break;
    }
  }
  // their results: of piece c - 1 its last segment (the second slot unless it begins with the unit), of the others the first
  const long long slot = static_cast<long long>(RB) * (D + 1);
  const float* first = j.part + (2LL * (c - 1) + (f0 == u0 ? 0 : 1)) * slot;
  const float* rest = j.part + 2LL * c * slot;
  // Few pieces: a thread for each (row, 4 dims). Many (a long context over many blocks): a warp takes 32
  // of those and every eighth piece, and the warps' sums meet in shared memory.
  constexpr int W = kKvJoinThreads / 32;
  __shared__ float join[W][32][6];
  const bool wide = pieces > 4;
  const int lanes = wide ? 32 : kKvJoinThreads, warp = threadIdx.x >> 5;
  const int i0p = wide ? warp : 0, di = wide ? W : 1;
  for (int base = part * lanes; base < RB * (D / 4); base += j.parts * lanes) {
    const int at = base + (wide ? threadIdx.x & 31 : threadIdx.x);
    const int row = at % RB, d0 = at / RB * 4;
    const bool live = at < RB * (D / 4) && row < rows;
    float M = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](float m2, float l2, const float4& x) {   // l2 times 2^m2 of weight, x the weighted sum
      const float Mn = fmaxf(M, m2);
      const float f = M == -INFINITY ? 0.0f : ex2(M - Mn), g = m2 == -INFINITY ? 0.0f : ex2(m2 - Mn);
      M = Mn;
      l = l * f + l2 * g;
      o[0] = o[0] * f + x.x * g;
      o[1] = o[1] * f + x.y * g;
      o[2] = o[2] * f + x.z * g;
      o[3] = o[3] * f + x.w * g;
    };
    if (live) {
#pragma unroll 4
      for (int i = i0p; i < pieces; i += di) {
        const float* p = i == 0 ? first : rest + 2LL * (i - 1) * slot;
        add(p[RB * D + row], 1.0f, reinterpret_cast<const float4*>(p)[at]);
      }
    }
    if (wide) {   // the same for the whole block
      float* mine = join[warp][threadIdx.x & 31];
      mine[0] = M;
      mine[1] = l;
#pragma unroll
      for (int k = 0; k < 4; ++k) mine[2 + k] = o[k];
      __syncthreads();
      if (warp == 0)
        for (int w = 1; w < W; ++w) {
          const float* p = join[w][threadIdx.x];
          add(p[0], p[1], make_float4(p[2], p[3], p[4], p[5]));
        }
      __syncthreads();
      if (warp != 0) continue;
    }
    if (!live) continue;
    const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;
    const int gr = pl.y + row;
    const long long tok = begin + gr / a.G;
    const int hq = pl.z * a.G + gr % a.G;
    *reinterpret_cast<uint2*>(a.out + tok * a.ldo + static_cast<long long>(hq) * D + d0) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    if (a.lse != nullptr && d0 == 0)
      a.lse[tok * a.Hq + hq] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.693147180559945f;
  }
}

}  // namespace respin
