// Attention over the 8-bit cache for many rows a key head (prefill, chunks):
// the 5th-generation tensor cores. Mathematics and numbers as in
// kv_attention.cuh: fp16 products of exact codes, weights 2^(s log2 e +
// log2 vs - M) rounded to fp16, sums in fp32.
//
// A block takes 256 rows of one key head (rows are (token, query head of the
// group), so grouped heads share every tile of the cache) as two 128-row
// tiles, and walks the cache in 64-token steps:
//   warps 0-3, 4-7   one row a thread of tile 0 / 1: S from tensor memory,
//                    maximum, weights back to tensor memory as fp16;
//   warps 8-11, 12-15 queries of tile 0 and K / of tile 1 and V, each half from
//                    a ring of its own of 8 KB slots, to fp16 operand tiles
//                    (128-byte swizzle; two of K, three of V);
//   warps 16, 18     one thread each issues a tile's S = Q K^T (both from
//                    shared memory) and O += P V (P from tensor memory, V with
//                    its dims contiguous, i.e. N-major);
//   warp 17          fills the rings: looks up page ids and scales of eight
//                    steps at a time, copies pages and queries with tensor
//                    copies (queries with asynchronous ones where a slot's rows
//                    are no whole tokens), as far ahead as the rings are deep,
//                    across units. (A parity wait knows only the phase before,
//                    so whoever waits on a slot has to take all that it holds:
//                    a ring that both halves share, each leaving out the other's
//                    entries, lets one pass a slot whose copy is on its way.)
// S of the next step is issued as soon as a tile's rows have read theirs, and
// P has two places of its own, so the rows never wait for the tensor core:
// their exponentials follow one another. (With 128-token steps S and P do not
// both fit beside O at D = 128; P in the place of S makes each step a chain of
// weights, product, scores: measured 5700 cycles for 128 tokens.) The running
// maximum may lag by 2^9 before the accumulators are rescaled, so rescaling is
// rare after the first steps and is done by the row's own thread.
//
// A row's 64 scores stay in registers: one read of tensor memory, one
// multiply-add and one exponential a score against the maximum of the steps
// before; the weights' own maximum (of the packed fp16) says whether they must
// be formed again.
//
// Bound. A step of 64 tokens takes 2450 cycles for both tiles at D = 128, 1900
// for one alone. The tensor core's share is 1024 of them, the exponentials'
// 1024, shared memory's 1536 (Q 64 KB, read anew for every 64 tokens, K and V
// 64 KB, codes in, out and widened 64 KB, at 128 bytes a cycle). With half of
// Q's reads or the widening left out a step is 5 % shorter, without the
// exponentials 15 %: the rest is a row warp's own chain of waits and tensor
// memory reads and writes, about 1000 cycles beside the weights. Sixteen warps
// for the rows (half a row a thread, the maxima exchanged) took 3000 cycles.
// Two 4096-token prompts, 32 query heads over 8: 380 us, 723 TFLOP/s; one of
// 8192: 675 us, 814 TFLOP/s. Logits of a standard deviation of 8 (natural units)
// move the maximum often enough to take 31 % longer (498 us; 454 with a lag of
// 2^13 in place of 2^9, which loses the weights below 2^-27 of the largest).
//
// Tensor memory: S0, S1 (64 columns each), P0, P1 (2 x 32 each), O0, O1 (D
// each). Shared memory at D = 128: Q 64 KB, K 32 KB, V 48 KB, rings 64 KB.
//
// Work: as in kv_attention.cuh one line of steps cut into equal pieces, here
// with each row group's own number of steps (causal rows see fewer).
#pragma once

#include "kv_attention.cuh"

namespace respin {

constexpr int kTcaRows = 128;       // rows of a tile
constexpr int kTcaGroup = 256;      // rows of a block
constexpr int kTcaTile = 64;        // tokens of a step
constexpr int kTcaThreads = 20 * 32;
// registers of a thread of the rows', the operands' and the last warps:
// 2 * 144 + 2 * 56 + 80 = 5 * 96, what 640 threads are launched with
constexpr int kTcaRegsRows = 144, kTcaRegsCodes = 56, kTcaRegsLast = 80;
constexpr int kTcaVStages = 3;
constexpr int kTcaMinTiles = 8;     // least piece of a block
// A unit's queries, first step and output cost about as much as six steps;
// the line of work counts them, so that blocks of many short units (a causal
// prompt's first rows) get fewer of their steps. Two 4096-token prompts of
// heads of 128, at a cost of 3, 4, 6, 8, 10: 453, 414, 379, 385, 391 us; 64 of
// 512 tokens: 295, 277, 272, 279, 283. Heads of 64 would have 4: 324, 326, 332,
// 340, 346 us and 209, 209, 217, 223, 225; chunks of 511 rows behind 8000 tokens
// with a window of 1000 are within 3 % of one another.
constexpr int kTcaUnitCost = 6;
static_assert(kTcaMinTiles > kTcaUnitCost, "a piece has a step");
constexpr int kTcaMaxBlocks = 160;  // one per SM
constexpr int kTcaMeta = 16;        // steps whose scales are kept (the rings are at most eight ahead of the rows)
constexpr int kTcaSlots = 4;        // of a ring
constexpr int kTcaSlot = 8192;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

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

// A bounded wait of a whole warp: the same answer in every lane, and the warp
// together again (lanes may leave a wait apart). A role that gives up signals
// and issues nothing more, so the others run into their own limits and leave.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, int site) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, site));
}

// One lane of the (converged) warp, known to the compiler as one: operands of
// the tensor-core instructions then stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Whether the phase has completed, without suspending the thread.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// One arrival of a converged warp, without a branch.
__device__ __forceinline__ void mbar_arrive_warp(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar)
      : "memory");
}

template <int R>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// A point before which values read from tensor memory are not used.
__device__ __forceinline__ void tmem_values(uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]),
                      "+r"(v[i + 6]), "+r"(v[i + 7]));
}

// 32 bytes at once (32-byte aligned).
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 16 bytes global -> shared by this thread (zeros where `in` is false), and an
// arrival on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
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

// First step and number of steps (at least 1) of row group g, and the first token that one of its rows sees.
__device__ __forceinline__ int3 tca_steps(const KvAttnArgs& a, int n, int len, int rows, int g) {
  const int first = len - n + kv_div_g(a, g * kTcaGroup);
  const int last = len - n + kv_div_g(a, min(rows, (g + 1) * kTcaGroup) - 1);
  const int hi = a.causal ? min(last, len - 1) : len - 1;
  if (hi < 0) return make_int3(0, 1, 0);
  const int lo = a.window > 0 ? min(hi, max(0, first - a.window + 1)) : 0;
  const int t0 = lo / kTcaTile;
  return make_int3(t0, hi / kTcaTile - t0 + 1, lo);
}

// Where a role stands in the block's piece of the line.
struct TcaCursor {
  TcaSeq s;
  int b, g, h, z;   // sequence, row group, head, steps of the unit already behind
  int t0, tiles, low;   // of the unit
  int left;

  __device__ __forceinline__ void unit(const KvAttnArgs& a) {
    const int3 t = tca_steps(a, s.n, s.len, s.rows, g);
    t0 = t.x;
    tiles = t.y;
    low = t.z;
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

// Position p of the line (each unit: kTcaUnitCost, then its steps): the unit
// it falls in, the steps of that unit before it, and of the whole line.
struct TcaPlace {
  int b, g, h, z, tiles;
  long long before;
};

// The block's piece: every lane of one warp.
__device__ __forceinline__ void tca_locate(const KvAttnArgs& a, volatile int* sh) {
  const int lane = threadIdx.x & 31;
  long long total = 0, steps = 0, chunk = 0, p[2] = {0, 0};
  TcaPlace at[2] = {{-1, 0, 0, 0, 0, 0}, {-1, 0, 0, 0, 0, 0}};   // where this piece and the next one begin
  for (int pass = 0; pass < 2; ++pass) {
    long long before = 0, sbefore = 0;
    for (int b0 = 0; b0 < a.c.B && at[1].b < 0; b0 += 32) {
      TcaSeq mine{0, 0, 0, 0, 0};
      if (b0 + lane < a.c.B) mine = tca_seq(a, b0 + lane);
      unsigned some = __ballot_sync(0xFFFFFFFFu, mine.groups > 0);
      while (some && at[1].b < 0) {
        const int f = __ffs(some) - 1;
        some &= some - 1;
        const int n = __shfl_sync(0xFFFFFFFFu, mine.n, f), len = __shfl_sync(0xFFFFFFFFu, mine.len, f);
        const int rows = __shfl_sync(0xFFFFFFFFu, mine.rows, f), groups = __shfl_sync(0xFFFFFFFFu, mine.groups, f);
        for (int g0 = 0; g0 < groups && at[1].b < 0; g0 += 32) {
          const int tiles = g0 + lane < groups ? tca_steps(a, n, len, rows, g0 + lane).y : 0;
          const int cost = tiles > 0 ? tiles + kTcaUnitCost : 0;
          long long incl = static_cast<long long>(cost) * a.c.H, sincl = static_cast<long long>(tiles) * a.c.H;
          if (pass == 0) {
            total += incl;
            steps += sincl;
            continue;
          }
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xFFFFFFFFu, incl, o), u = __shfl_up_sync(0xFFFFFFFFu, sincl, o);
            if (lane >= o) {
              incl += t;
              sincl += u;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + incl > p[e]);
            if (at[e].b >= 0 || !hit) continue;
            const int l = __ffs(hit) - 1;
            const int lt = __shfl_sync(0xFFFFFFFFu, tiles, l);
            const long long off = p[e] - before - __shfl_sync(0xFFFFFFFFu, incl - static_cast<long long>(cost) * a.c.H, l);
            const int h = static_cast<int>(off / (lt + kTcaUnitCost));
            const int z = max(0, static_cast<int>(off - static_cast<long long>(h) * (lt + kTcaUnitCost)) - kTcaUnitCost);
            at[e] = {b0 + f, g0 + l, h, z, lt,
                     sbefore + __shfl_sync(0xFFFFFFFFu, sincl - static_cast<long long>(tiles) * a.c.H, l) +
                         static_cast<long long>(h) * lt + z};
          }
          before += __shfl_sync(0xFFFFFFFFu, incl, 31);
          sbefore += __shfl_sync(0xFFFFFFFFu, sincl, 31);
        }
      }
    }
    if (pass == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        steps += __shfl_xor_sync(0xFFFFFFFFu, steps, o);
      }
      chunk = max(static_cast<long long>(kTcaMinTiles), (total + gridDim.x - 1) / gridDim.x);
      p[0] = chunk * blockIdx.x;
      p[1] = p[0] + chunk;
      if (p[0] >= total) break;
    }
  }
  if (lane == 0) {
    const long long first = at[0].b < 0 ? steps : at[0].before, end = at[1].b < 0 ? steps : at[1].before;
    sh[0] = at[0].b;
    sh[1] = at[0].g;
    sh[2] = at[0].h;
    sh[3] = at[0].z;
    sh[4] = static_cast<int>(end - first);
    a.plan[kKvPlan * blockIdx.x] = make_int4(at[0].b, at[0].g * kTcaGroup, at[0].h, at[0].z);
    a.plan[kKvPlan * blockIdx.x + 1] = make_int4(at[0].tiles, static_cast<int>(first & 0xFFFFFFFF), static_cast<int>(first >> 32), 0);
    if (at[0].b >= 0) {
      const TcaSeq s = tca_seq(a, at[0].b);
      a.plan[kKvPlan * blockIdx.x + 2] = make_int4(s.begin, s.rows, 0, 0);
    }
  }
}

template <int D>
struct TcaCfg {
  static constexpr int OpQ = kTcaRows * D * 2, Op = kTcaTile * D * 2;   // bytes of the fp16 operand tiles
  static constexpr int OQ = 0, OK = 2 * OpQ, OV = OK + 2 * Op, ORing = OV + kTcaVStages * Op;
  static constexpr int OMeta = ORing + 2 * kTcaSlots * kTcaSlot;        // [steps][4] scales of 16 tokens each
  static constexpr int OCoef = OMeta + kTcaMeta * 4 * 16;               // [2][256] the rows' factors; a tile's units take turns
  static constexpr int OBar = OCoef + 2 * kTcaGroup * 4;
  static constexpr int Bars = 21 + 2 * kTcaVStages + 4 * kTcaSlots;
  static constexpr int Smem = 1024 + OBar + 8 * Bars + 64;
  static constexpr int Columns = 512;
  static constexpr int SlotFloats = kTcaGroup * (D + 1);
};

// tmQ: bf16 [N][Hq][D], box {D, G, rows of a slot / G} (not used where G does not divide those rows);
// tmK, tmV: uint8 [pages * H * P, D], box {D, min(P, 64)}; no swizzle.
template <int D>
__global__ void __launch_bounds__(kTcaThreads, 1)
kv_attn_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const KvAttnArgs a) {
  using C = TcaCfg<D>;
  constexpr int KB = D / 64;         // 64-value blocks of a row
  constexpr int Block = kTcaTile * 128, BlockQ = kTcaRows * 128;   // bytes of one block of K or V, of Q
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t bars = base + C::OBar;
  const uint32_t kfull = bars, kempty = bars + 16;                            // [2] stages
  const uint32_t qfull = bars + 32, qempty = bars + 48, sfull = bars + 64, sfree = bars + 80;   // [2] tiles
  const uint32_t pfull = bars + 96, pfree = bars + 128, drained = bars + 160;                // [2 tiles][2 places of P]
  const uint32_t vfull = bars + 168, vempty = vfull + 8 * kTcaVStages;                       // stages of V
  const uint32_t efull = vempty + 8 * kTcaVStages, eempty = efull + 16 * kTcaSlots;          // [2 rings] slots
  volatile int* sh = reinterpret_cast<volatile int*>(smem + C::OBar + 8 * C::Bars);
  const uint32_t tslot = base + C::OBar + 8 * C::Bars + 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull + 8 * i, 4);
      mbar_init(kempty + 8 * i, 2);   // both tiles' products
      mbar_init(qfull + 8 * i, 4);
      mbar_init(qempty + 8 * i, 1);
      mbar_init(sfull + 8 * i, 2);   // the product, and the issuing thread (it saw the step's scales)
      mbar_init(sfree + 8 * i, 4);
      mbar_init(pfull + 16 * i, 4);
      mbar_init(pfull + 16 * i + 8, 4);
      mbar_init(pfree + 16 * i, 1);
      mbar_init(pfree + 16 * i + 8, 1);
    }
    for (int i = 0; i < kTcaVStages; ++i) {
      mbar_init(vfull + 8 * i, 4);
      mbar_init(vempty + 8 * i, 2);
    }
    for (int i = 0; i < 2 * kTcaSlots; ++i) {
      mbar_init(efull + 8 * i, 32);   // every lane of warp 17, and the bytes of its tensor copies
      mbar_init(eempty + 8 * i, 4);
    }
    mbar_init(drained, 2);
    fence_mbarrier_init();
  }
  if (warp == 16) {
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
    regs_take<kTcaRegsRows>();
    const int tile = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // 32 lanes of tensor memory a warp
    const uint32_t ts = tmem + lanes + tile * 64, tp = tmem + lanes + 128 + tile * 64, to = tmem + lanes + 256 + tile * D;
    bool ok = true;
    int use = 0, step = 0, seg = 0;   // use: steps of this tile; P's place is use & 1
    int mine = 0;                     // units of this tile
    const uint32_t pfree_t = pfree + 16 * tile;
    // PV of use u has completed (its P is free, its O is there): u the last or the one before
    auto product = [&](int u) { return mbar_wait_warp(pfree_t + 8 * (u & 1), (u >> 1) & 1, kSiteKvAccum); };
    while (cur.left > 0 && ok) {
      const int n = cur.steps();
      const int row0 = cur.g * kTcaGroup;
      if (row0 + tile * kTcaRows < cur.s.rows) {
        const int row = row0 + tile * kTcaRows + r;
        const bool live = row < cur.s.rows;
        const int rr = min(row, cur.s.rows - 1);
        const int tok = kv_div_g(a, rr), hq = cur.h * a.G + rr - tok * a.G;
        const int pos = cur.s.len - cur.s.n + tok;
        const int hi = a.causal ? min(pos, cur.s.len - 1) : cur.s.len - 1;
        const int lo = a.window > 0 ? pos - a.window + 1 : 0;
        // steps in which no row of the warp has a masked token: [whole0, whole1)
        const int first_t = (cur.t0 + cur.z) * kTcaTile;
        const int whole0 = (max(0, __reduce_max_sync(0xFFFFFFFFu, lo) - first_t) + kTcaTile - 1) / kTcaTile;
        const int whole1 = (__reduce_min_sync(0xFFFFFFFFu, hi) + 1 - first_t) / kTcaTile;   // (below 0: none)
        float M = -INFINITY, l = 0.0f, coef = 0.0f, ref = 1.0f;
        bool there = false;   // S of the step has been seen complete
        for (int j = 0; j < n; ++j, ++use) {
          // S of this step also says that P's place is free: its arrival follows every product that
          // its thread issued before, PV of use - 2 among them.
          if (!there) ok = mbar_wait_warp(sfull + 8 * tile, use & 1, kSiteKvAccum);
          if (!ok) break;
          tc_fence_after();
          uint32_t v[2][32];
          tmem_ld_32x32b_x32(ts, v[0]);
          tmem_ld_32x32b_x32(ts + 32, v[1]);
          if (j == 0) coef = reinterpret_cast<const float*>(smem + C::OCoef)[(mine & 1) * kTcaGroup + tile * kTcaRows + r];
          const int t = (cur.t0 + cur.z + j) * kTcaTile;
          const KvScale* meta = reinterpret_cast<const KvScale*>(smem + C::OMeta) + ((step + j) % kTcaMeta) * 4;
          if (j == 0) ref = meta->ref;
          const bool whole = j >= whole0 && j < whole1;
          const bool unseen = M == -INFINITY && t <= hi && t + kTcaTile - 1 >= lo;   // the row's first tokens
          // a factor of 0 (all products are 0, or are to count as 0) becomes one that keeps -inf
          float ck[4], lv[4], iv[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const KvScale sc = meta[c];
            ck[c] = fmaxf(coef * sc.k, 1e-37f);
            lv[c] = sc.lv;
            iv[c] = sc.iv;
          }
          tmem_wait_ld();
          tmem_values(v[0]);
          tmem_values(v[1]);
          tc_fence_before();
          mbar_arrive_warp(sfree + 8 * tile);   // (the wait for the loads is the whole warp's)
          if (!whole) {
            const int first = lo - t, last = hi - t;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i < first || 32 * c + i > last) v[c][i] = 0xFF800000u;   // -inf
          }
          // ---- weights against the maximum of the steps before, their sum and their own maximum: the
          // comparisons run beside the exponentials. Where an exponent passes M by 2^15 (the unit's
          // first step, and rarely later) the maximum moves and the weights are formed again.
          float ls = 0.0f;
#pragma unroll 1
          for (bool again = j == 0;;) {
            if (again) {
              float mx = -INFINITY;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t* x = &v[c / 2][16 * (c % 2)];
                float m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  m[i] = fmaxf(fmaxf(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1])),
                               fmaxf(__uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3])));
                mx = fmaxf(mx, fmaf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), ck[c], lv[c]));
              }
              const float Mn = mx > M + (kKvBias + kKvLazy) ? mx - kKvBias : M;
              const float f = Mn == M ? 1.0f : ex2(M - Mn);   // 0 from nothing
              M = Mn;
              l *= f;
              if (j > 0) {
                ok = product(use - 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t u[16];
                  tmem_ld_32x32b_x16(to + 16 * c, u);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * f);
                  tmem_st_32x32b_x16(to + 16 * c, u);
                }
              }
            }
            const float Ms = M == -INFINITY ? 0.0f : M;
            ls = 0.0f;
            __half2 top[2] = {__half2half2(__ushort_as_half(0)), __half2half2(__ushort_as_half(0))};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t p[16];
#pragma unroll
              for (int hb = 0; hb < 2; ++hb) {
                const float o = lv[2 * c + hb] - Ms;
                const uint64_t ck2 = f32x2(ck[2 * c + hb], ck[2 * c + hb]), of2 = f32x2(o, o);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  const float2 e = f32x2_split(fma_f32x2(
                      f32x2(__uint_as_float(v[c][16 * hb + i]), __uint_as_float(v[c][16 * hb + i + 1])), ck2, of2));
                  const float x = ex2(e.x), y = ex2(e.y);
                  const uint32_t w = pack_f16x2(x, y);
                  p[8 * hb + i / 2] = w;
                  sum[(i / 2) & 1] = add_f32x2(sum[(i / 2) & 1], f32x2(x, y));
                  top[(i / 2) & 1] = __hmax2(top[(i / 2) & 1], *reinterpret_cast<const __half2*>(&w));
                }
                const float2 s2 = f32x2_split(add_f32x2(sum[0], sum[1]));
                ls = fmaf(s2.x + s2.y, iv[2 * c + hb], ls);
              }
              tmem_st_32x32b_x16(tp + 32 * (use & 1) + 16 * c, p);
              // the next step's S, looked at where the answer is not waited for
              if (c == 0) there = j + 1 < n && mbar_test_wait(sfull + 8 * tile, (use + 1) & 1);
            }
            // (after the maximum has moved no weight passes 2^15)
            const __half2 tt = __hmax2(top[0], top[1]);
            const float limit = 32768.0f;   // 2^(kKvBias + kKvLazy)
            there = __all_sync(0xFFFFFFFFu, there);
            again = !again && __any_sync(0xFFFFFFFFu, unseen || __low2float(tt) > limit || __high2float(tt) > limit);
            if (!again) break;
          }
          if (!ok) break;
          l += ls;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive_warp(pfull + 16 * tile + 8 * (use & 1));
        }
        if (ok) ok = product(use - 1);
        if (!ok) break;
        ++mine;
        tc_fence_after();
        const bool split = n < cur.tiles;
        float* slot = a.part + (static_cast<long long>(blockIdx.x) * 2 + (seg > 0 ? 1 : 0)) * C::SlotFloats;
        const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;   // a row that sees nothing is 0
        const float L = l == 0.0f ? -INFINITY : M + log2f(l) - log2f(ref);
        __nv_bfloat16* op = a.out + (cur.s.begin + tok) * a.ldo + static_cast<long long>(hq) * D;
        const bool wide = (reinterpret_cast<uintptr_t>(a.out) | (a.ldo * 2)) % 32 == 0;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          __syncwarp();   // absent rows skip the stores
          tmem_ld_32x32b_x32(to + 32 * c, v);
          tmem_wait_ld();
          tmem_values(v);
          if (!live) continue;
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * inv * ref);
          if (split) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              kv_put_partial(slot, kTcaGroup, row - row0, 32 * c + i,
                             make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]),
                                         __uint_as_float(v[i + 3])));
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k)
                w[k] = pack_bf16x2(__uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
              uint32_t* at = reinterpret_cast<uint32_t*>(op + 32 * c + i);
              if (wide) {
                st_global_v8(at, w);
              } else {
                reinterpret_cast<uint4*>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        }
        __syncwarp();
        tc_fence_before();
        if (live) {
          if (split)
            slot[kTcaGroup * D + row - row0] = L;
          else if (a.lse != nullptr)
            a.lse[(cur.s.begin + tok) * static_cast<long long>(a.Hq) + hq] = L * 0.693147180559945f;
        }
      }
      step += n;
      ++seg;
      cur.next(a);
    }
  } else if (warp < 16) {
    // ------------------------------------------------ codes to fp16
    regs_give<kTcaRegsCodes>();
    const int pt = (tid - 256) & 127, half = (warp - 8) >> 2;   // half: 0 tile 0 and K, 1 tile 1 and V
    bool ok = true;
    int mine = 0, slot = 0, ph_e = 0, stage = 0, ph_s = 1;   // mine: units of this half's tile
    const int stages = half ? kTcaVStages : 2;
    const uint32_t full_e = efull + 8 * kTcaSlots * half, empty_e = eempty + 8 * kTcaSlots * half;   // this half's ring
    const uint8_t* const ring = smem + C::ORing + half * kTcaSlots * kTcaSlot;
    auto take = [&]() {
      ok = ok && mbar_wait_warp(full_e + 8 * slot, ph_e, kSiteKvLoad);
      return ring + slot * kTcaSlot;
    };
    // the operand tile is written (and the slot's bytes are read): for the async proxy, then the next user
    auto give = [&](uint32_t full) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(empty_e + 8 * slot);
        if (full) mbar_arrive(full);
      }
      if (++slot == kTcaSlots) {
        slot = 0;
        ph_e ^= 1;
      }
    };
    auto widen = [&](uint8_t* to, const uint8_t* from) {
      constexpr int Pieces = D / 16;                 // 16-byte pieces of a token's codes
      constexpr int Per = kTcaTile * Pieces / 128;   // pieces of a thread
      constexpr int Step = 128 / Pieces;             // tokens between them
      const int c = pt % Pieces, tk = pt / Pieces;
      uint8_t* p = to + (c >> 2) * Block + (tk >> 3) * 1024 + (tk & 7) * 128;   // t & 7 = tk & 7
      const int a0 = ((2 * (c & 3)) ^ (tk & 7)) << 4;
#pragma unroll
      for (int i = 0; i < Per; ++i) {
        const uint4 w = reinterpret_cast<const uint4*>(from)[pt + 128 * i];
        const uint32_t x[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
        const uint4 lo = make_uint4(codes_f16x2<0>(x[0]), codes_f16x2<1>(x[0]), codes_f16x2<0>(x[1]), codes_f16x2<1>(x[1]));
        const uint4 hi = make_uint4(codes_f16x2<0>(x[2]), codes_f16x2<1>(x[2]), codes_f16x2<0>(x[3]), codes_f16x2<1>(x[3]));
        *reinterpret_cast<uint4*>(p + i * Step * 128 + a0) = lo;
        *reinterpret_cast<uint4*>(p + i * Step * 128 + (a0 ^ 16)) = hi;
      }
    };
    while (cur.left > 0 && ok) {
      const int n = cur.steps();
      // ---- queries: scaled by a power of two to fp16
      constexpr int L = D / 8, RE = kTcaSlot / (2 * D);   // pieces of a row, rows of a slot
      const int tile = half, row0 = cur.g * kTcaGroup;
      if (row0 + tile * kTcaRows < cur.s.rows) {
        // The last S of the tile's unit before is there, so its first step's rows have read the
        // factors of the one before that, and their place is free. (Counted over the tile's own
        // units: with a unit without this tile between, nothing says that they were read.)
        ok = mbar_wait_warp(qempty + 8 * tile, (mine & 1) ^ 1, kSiteKvFree);
#pragma unroll 1
        for (int r0 = 0; r0 < kTcaRows; r0 += RE) {
          const uint8_t* from = take();
          if (!ok) break;
          // TR threads a row, four pieces each: piece (i + row) % 4 * TR + c, so that the rows of eight
          // neighbouring lanes lie on different banks, read and written
          constexpr int TR = L / 4;
          const int r = r0 + pt / TR, c = pt % TR;
          uint4 w[4];
          uint32_t m2 = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = reinterpret_cast<const uint4*>(from)[pt / TR * L + ((i + r) & 3) * TR + c];
            m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu),
                                       __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu)));
          }
          uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
          for (int o = TR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          // (a row with an infinity or NaN is scaled as one of 2^127: its results are not finite anyway)
          const int e = max(-110, min(127, static_cast<int>(m >> 7) - 127));
          // a negative scale goes with the queries, so that the factors are not negative
          const float up = copysignf(__int_as_float((14 - e + 127) << 23), a.scale);
          uint8_t* qs = smem + C::OQ + tile * C::OpQ + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int piece = ((i + r) & 3) * TR + c;
            float f[8];
            bf16x8_to_f32(w[i], f);
            *reinterpret_cast<uint4*>(qs + (piece >> 3) * BlockQ + (((piece & 7) ^ (r & 7)) << 4)) =
                make_uint4(pack_f16x2(f[0] * up, f[1] * up), pack_f16x2(f[2] * up, f[3] * up),
                           pack_f16x2(f[4] * up, f[5] * up), pack_f16x2(f[6] * up, f[7] * up));
          }
          if (c == 0)
            reinterpret_cast<float*>(smem + C::OCoef)[(mine & 1) * kTcaGroup + tile * kTcaRows + r] =
                __int_as_float((e - 14 + 127) << 23) * fabsf(a.scale);
          give(r0 + RE >= kTcaRows ? qfull + 8 * tile : 0u);
        }
        ++mine;
      }
      // ---- codes
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j) {
        const uint8_t* from = take();
        const uint32_t full = (half ? vfull : kfull) + 8 * stage, empty = (half ? vempty : kempty) + 8 * stage;
        ok = ok && mbar_wait_warp(empty, ph_s, kSiteKvFree);
        if (!ok) break;
        widen(smem + (half ? C::OV : C::OK) + stage * C::Op, from);
        give(full);
        if (++stage == stages) {
          stage = 0;
          ph_s ^= 1;
        }
      }
      cur.next(a);
    }
  } else {
    regs_give<kTcaRegsLast>();
    if (warp == 17) {
      // ---------------------------------------------- the rings
      bool ok = true;
      int j = 0, step = 0, used0 = 0, used1 = 0;   // entries of ring 0 and 1 so far
      // the next slot of a ring, once it is free: 0 .. 2 * kTcaSlots - 1
      auto next_slot = [&](int ring) {
        const int used = ring ? used1 : used0;
        const int slot = ring * kTcaSlots + used % kTcaSlots;
        ok = mbar_wait_warp(eempty + 8 * slot, (used / kTcaSlots & 1) ^ 1, kSiteKvFree);
        return slot;
      };
      TcaCursor ahead = cur;   // the lookups' cursor; cur: the copies'
      int aj = 0, au = 0;        // its step of the unit, its unit
      int ref_u = -1;            // the unit that the last lookups ended in, and its ref
      float ref_last = 1.0f;
      while (cur.left > 0 && ok) {
        // ---- page ids and scales of eight steps: lane / 4, 16 tokens a lane
        int b = -1, h = 0, t = 0, unit = -1;
#pragma unroll 1
        for (int u = 0; u < 8 && ahead.left > 0; ++u) {
          if (lane >> 2 == u) {
            b = ahead.b;
            h = ahead.h;
            unit = au;
            t = (ahead.t0 + ahead.z + aj) * kTcaTile + 16 * (lane & 3);
            const int SP = min(a.c.P, kTcaTile);
            if (t >= ahead.s.len || (t & ~(SP - 1)) + SP <= ahead.low) b = -1;   // (pages behind the window may be gone)
          }
          if (++aj == ahead.steps()) {
            aj = 0;
            ++au;
            ahead.next(a);
          }
        }
        int row = -1;
        float ks = 0.0f, vs = 0.0f;
        if (b >= 0) {
          const int page = kv_page(a.c, b, t);
          if (page >= 0) {
            const int phd = page * a.c.H + h;
            row = phd * a.c.P + t % a.c.P;
            ks = a.c.k_scale[phd];
            vs = a.c.v_scale[phd];
          }
        }
        // a unit's ref, from the lookups it begins in
        float most = vs > 0.0f ? vs : 0.0f, ref = 0.0f;
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {
          const float m = __shfl_sync(0xFFFFFFFFu, most, 4 * u);
          if (__shfl_sync(0xFFFFFFFFu, unit, 4 * u) == unit) ref = fmaxf(ref, m);
        }
        if (unit == ref_u) ref = ref_last;
        else if (ref == 0.0f) ref = 1.0f;
        ref_u = __shfl_sync(0xFFFFFFFFu, unit, 31);
        ref_last = __shfl_sync(0xFFFFFFFFu, ref, 31);
        KvScale sc = kv_scale_of(ks, vs, ref);
        if (row < 0) sc.lv = -INFINITY;
        // a page's first 16 tokens name its copy; tokens of no page keep what the slot holds (finite codes)
        const int SP = min(a.c.P, kTcaTile);   // rows of a copy
        const bool boxes = row >= 0 && ((lane & 3) * 16) % SP == 0;
        // ---- copies, step by step
#pragma unroll 1
        for (int u = 0; u < 8 && cur.left > 0 && ok; ++u, ++step) {
          if (j == 0) {
            constexpr int L = D / 8, RE = kTcaSlot / (2 * D);
#pragma unroll 1
            for (int r0 = 0; r0 < kTcaGroup && ok; r0 += RE) {
              const int row0 = cur.g * kTcaGroup + r0;
              if (cur.g * kTcaGroup + (r0 & ~(kTcaRows - 1)) >= cur.s.rows) break;
              const int ring = r0 >= kTcaRows;   // the tile's
              const int slot = next_slot(ring);
              if (!ok) break;
              const uint32_t dst = base + C::ORing + slot * kTcaSlot;
              if (RE % a.G == 0) {   // whole tokens: rows behind the sequence are anybody's, and dead
                if (lane == 0) {
                  mbar_arrive_expect_tx(efull + 8 * slot, kTcaSlot);
                  tma_load_3d(dst, &tmQ, 0, cur.h * a.G, cur.s.begin + kv_div_g(a, row0), efull + 8 * slot);
                } else {
                  mbar_arrive(efull + 8 * slot);
                }
              } else {
                int tok = kv_div_g(a, row0 + lane / L), g = row0 + lane / L - tok * a.G;
                const int dt = kv_div_g(a, 32 / L), dg = 32 / L - dt * a.G;
#pragma unroll 1
                for (int i = 0; i < RE * L / 32; ++i) {
                  const bool in = tok < cur.s.n;
                  cp_async_16(dst + (32 * i + lane) * 16,
                              reinterpret_cast<const uint4*>(a.q + (cur.s.begin + (in ? tok : 0)) * a.ldq +
                                                             static_cast<long long>(cur.h * a.G + g) * D) + lane % L,
                              in);
                  tok += dt;
                  g += dg;
                  if (g >= a.G) {
                    g -= a.G;
                    ++tok;
                  }
                }
                cp_async_arrive(efull + 8 * slot);
              }
              (ring ? used1 : used0) += 1;
            }
          }
#pragma unroll 1
          for (int kv = 0; kv < 2 && ok; ++kv) {
            const int slot = next_slot(kv);
            if (!ok) break;
            const bool mine = boxes && lane >> 2 == u;
            if (kv == 0 && lane >> 2 == u)
              reinterpret_cast<KvScale*>(smem + C::OMeta)[(step % kTcaMeta) * 4 + (lane & 3)] = sc;
            if (mine) mbar_arrive_expect_tx(efull + 8 * slot, static_cast<uint32_t>(SP * D));
            if (mine)
              tma_load_2d(base + C::ORing + slot * kTcaSlot + (lane & 3) * 16 * D, kv == 0 ? &tmK : &tmV, 0, row, efull + 8 * slot);
            if (!mine) mbar_arrive(efull + 8 * slot);
            (kv ? used1 : used0) += 1;
          }
          if (++j == cur.steps()) {
            j = 0;
            cur.next(a);
          }
        }
      }
      // leave only once the last copies have landed, whatever became of the others
      for (int ring = 0; ring < 2; ++ring) {
        const int used = ring ? used1 : used0;
        for (int i = max(0, used - kTcaSlots); i < used; ++i)
          mbar_wait(efull + 8 * (ring * kTcaSlots + i % kTcaSlots), (i / kTcaSlots) & 1, kSiteKvLoad);
      }
    } else if ((warp == 16 || warp == 18) && elect_one()) {
      // ---------------------------------------------- tensor core, one thread a tile
      constexpr uint32_t is = umma_idesc_f16(kTcaRows, kTcaTile, false), io = umma_idesc_f16(kTcaRows, D, true);
      const int tile = (warp - 16) >> 1;
      const uint32_t ts = tmem + tile * 64, tp = tmem + 128 + tile * 64, to = tmem + 256 + tile * D;
      const uint64_t dq = umma_desc_sw128(base + C::OQ) + tile * (C::OpQ >> 4);   // addresses in 16 bytes
      const uint64_t dk = umma_desc_sw128(base + C::OK), dv = umma_desc_sw128_n(base + C::OV, Block);
      bool ok = true;
      uint32_t units = 0, scored = 0, used = 0;   // of this tile: units, S and PV issued
      // S of a step (of the piece; the unit's first or last)
      auto scores = [&](int step, bool mine, bool first, bool last) {
        const int st = step & 1;
        ok = mbar_wait(kfull + 8 * st, (step >> 1) & 1, kSiteKvLoad);
        if (!mine) {   // a unit without this tile: only K's stage is passed on
          if (ok) mbar_arrive(kempty + 8 * st);
          return;
        }
        if (first) {
          ok = ok && mbar_wait(qfull + 8 * tile, units & 1, kSiteKvLoad);
          ++units;
        }
        if (scored > 0) ok = ok && mbar_wait(sfree + 8 * tile, (scored - 1) & 1, kSiteKvAccum);   // the last S is read
        ++scored;
        if (!ok) return;
        tc_fence_after();
        const uint64_t dks = dk + st * (C::Op >> 4);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int k = 0; k < 4; ++k)   // (kind::f16; the descriptor says fp16)
            tc_mma_bf16(ts, dq + kb * (BlockQ >> 4) + 2 * k, dks + kb * (Block >> 4) + 2 * k, is, kb + k > 0);
        mbar_arrive(sfull + 8 * tile);
        tc_commit(sfull + 8 * tile);
        tc_commit(kempty + 8 * st);
        if (last) tc_commit(qempty + 8 * tile);
      };
      auto is_mine = [&]() { return cur.g * kTcaGroup + tile * kTcaRows < cur.s.rows; };
      int j = 0, n = cur.left > 0 ? cur.steps() : 0, vst = 0, ph_v = 0;
      bool mine = cur.left > 0 && is_mine();
      if (cur.left > 0) scores(0, mine, true, n == 1);
      for (int step = 0; cur.left > 0 && ok; ++step) {
        const bool now = mine, first = j == 0;
        if (++j == n) {   // the next step is the next unit's first
          cur.next(a);
          j = 0;
          if (cur.left > 0) {
            n = cur.steps();
            mine = is_mine();
          }
        }
        if (cur.left > 0) scores(step + 1, mine, j == 0, j == n - 1);
        ok = ok && mbar_wait(vfull + 8 * vst, ph_v, kSiteKvLoad);
        if (now) {
          const int pb = used & 1;
          ok = ok && mbar_wait(pfull + 16 * tile + 8 * pb, (used >> 1) & 1, kSiteKvAccum);
          if (!ok) break;
          ++used;
          tc_fence_after();
          const uint64_t dvs = dv + vst * (C::Op >> 4);
#pragma unroll
          for (int k = 0; k < kTcaTile / 16; ++k)
            tc_mma_f16_ta(to, tp + 32 * pb + 8 * k, dvs + 128 * k, io, !first || k > 0);
          tc_commit(pfree + 16 * tile + 8 * pb);
          tc_commit(vempty + 8 * vst);
        } else if (ok) {
          mbar_arrive(vempty + 8 * vst);
        }
        if (++vst == kTcaVStages) {
          vst = 0;
          ph_v ^= 1;
        }
      }
      // nothing issued here may still run when the tensor memory is given back
      tc_commit(drained);
      mbar_wait(drained, 0, kSiteKvAccum);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, C::Columns);
}

}  // namespace respin
