// The 8-bit key/value cache: pages of int8 codes with one fp32 scale for each
// page and head, written (quantized) and read back.
//
//   codes [pages][heads][P][D] int8, scales [pages][heads] fp32,
//   value = code * scale;  token t of sequence b is slot t % P of page
//   table[b][t / P].
//
// Writing. With a = max |x| over the finite new values of a page and head
// (binary32, every operation rounded to nearest even):
//   s = max(s_old, a / 127)     s_old: the page's scale if it holds earlier
//                               tokens of the sequence, else 0
//   s < 2^-126 -> 0
//   earlier codes c -> rint(c * (s_old / s)), left alone while s = s_old
//   new codes = clamp(rint(x * (1 / s)), -127, 127); NaN -> 0; all 0 for s = 0
// A page of a call's tokens belongs to one block per head and tensor, which
// sees all of them, so nothing depends on an order of blocks and a repeated
// call finds s = s_old and writes the same bytes again.
//
// Both directions are memory bound (3 bytes an element). Measured: 6906 tokens
// of 32 heads of 128 into pages of 16, 42 us (4.0 TB/s; a warp has no load on its
// way while it forms a unit's codes); 22006 tokens of 8
// heads read back, 28 us (5.1 TB/s).
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace respin {

// Device view of a cache and of a ragged batch of the last tokens of its
// sequences: rows cu[b] .. cu[b + 1] - 1 are the last ones of sequence b,
// whose length with them is kv_len[b]. cu == nullptr: `per` rows each.
struct KvView {
  int8_t* k;
  int8_t* v;
  float* k_scale;
  float* v_scale;
  int pages, P, H;
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int B, max_pages, N, per;
};

// Rows of sequence b: [begin, end) within [0, N), or an empty range, and its
// length. What does not fit the batch or the block table is recorded and
// taken as empty.
__device__ __forceinline__ bool kv_rows(const KvView& c, int b, int& begin, int& end, int& len) {
  begin = c.cu ? c.cu[b] : b * c.per;
  end = c.cu ? c.cu[b + 1] : begin + c.per;
  len = c.kv_len[b];
  if (begin == end) len = 0;   // no rows (a padded batch): its length is not looked at
  const bool ok = begin >= 0 && begin <= end && end <= c.N && len >= 0 &&
                  static_cast<long long>(len) <= static_cast<long long>(c.max_pages) * c.P;
  if (!ok) {
    record_status(kSiteKvLength);
    begin = end = 0;
    len = 0;
  }
  return ok;
}

// Sequence of row r, or B when no sequence holds it (rows behind the last
// one). Every lane of the warp calls it with the same r: 32 sequences are
// looked at in a step, so 32 take one and 1024 two round trips to memory.
__device__ __forceinline__ int kv_find(const KvView& c, int r) {
  if (c.cu == nullptr) return r / c.per;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = c.B;   // the first b with cu[b + 1] > r lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && c.cu[at + 1] <= r;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, below));
    if (n == 0) break;
    const int first = lo + (n - 1) * step + 1;
    hi = min(hi, lo + n * step);
    lo = first;
  }
  return lo;
}

// Page id of token t of sequence b, or -1 (recorded) outside the cache.
__device__ __forceinline__ int kv_page(const KvView& c, int b, int t) {
  const int id = c.table[static_cast<long long>(b) * c.max_pages + t / c.P];
  if (id >= 0 && id < c.pages) return id;
  record_status(kSiteKvPage);
  return -1;
}

constexpr int kKvPieces = 8;         // 16-byte pieces of new values a thread holds
constexpr int kKvAppendThreads = 256;

struct KvAppendArgs {
  KvView c;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long ldk, ldv;   // elements between tokens
  int rows;             // rows of a block
  int warps;            // of a unit (a head's K or V): P * D / 8 pieces at kKvPieces a lane, 1, 2, 4 or 8
};

// max |x| of eight bf16 values, finite ones only, as the bits of a bf16.
__device__ __forceinline__ uint32_t bf16x8_finite_amax(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    m = max(m, lo < 0x7F80u ? lo : 0u);
    m = max(m, hi < 0x7F80u ? hi : 0u);
  }
  return m;
}

// max |x| of eight bf16 values as the bits of a bf16, whatever they are
// (infinities and NaN lie above all finite ones).
__device__ __forceinline__ uint32_t bf16x8_amax(const uint4& v) {
  const uint32_t k = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
  return max(m & 0xFFFFu, m >> 16);
}

// Codes of four finite values with |x * inv| < 127.5: adding 1.5 * 2^23
// rounds to a whole number (ties to even) whose low byte is the code. (The
// conversion instruction has a quarter of the rate.)
__device__ __forceinline__ uint32_t kv_codes4(float a, float b, float c, float d, float inv) {
  const float k = 12582912.0f;
  const uint32_t x = __float_as_uint(__fadd_rn(__fmul_rn(a, inv), k)), y = __float_as_uint(__fadd_rn(__fmul_rn(b, inv), k));
  const uint32_t z = __float_as_uint(__fadd_rn(__fmul_rn(c, inv), k)), w = __float_as_uint(__fadd_rn(__fmul_rn(d, inv), k));
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t kv_code(float x, float inv) {
  const int q = __float2int_rn(__fmul_rn(x, inv));   // NaN -> 0, saturates
  return static_cast<uint32_t>(max(-127, min(127, q))) & 0xFFu;
}

// grid (row chunks, groups of units). The block's rows are cut at page
// boundaries and sequence ends; it owns the pages whose first new token is
// one of its rows. Its eight warps are shared out over units (a head's keys or
// values) and go from group to group of them, so a page's place is looked up
// once for many. The new values stay in registers between the maximum and the
// codes. (A block for each unit, with its own lookups: 122 us for 6906 tokens
// of 32 heads, 1.4 TB/s.)
template <int D>
__global__ void __launch_bounds__(kKvAppendThreads, 3) kv_append_kernel(const KvAppendArgs a) {
  constexpr int L = D / 8;   // 16-byte pieces of a token
  __shared__ uint32_t amax_warp[kKvAppendThreads / 32];
  const KvView& c = a.c;
  const int warp = threadIdx.x / 32;
  const int T = a.warps * 32, tid = threadIdx.x % T;   // threads of a unit
  const int units = 8 / a.warps;                       // of the block at a time

  grid_dep_wait();
  grid_dep_launch();
  int r = blockIdx.x * a.rows;
  const int stop = min(c.N, r + a.rows);
  while (r < stop) {
    const int b = kv_find(c, r);
    if (b >= c.B) break;
    int begin, end, len;
    if (!kv_rows(c, b, begin, end, len) || r < begin || r >= end) {
      ++r;   // (an unordered cu: nothing to rely on)
      continue;
    }
    const int start = len - (end - begin);          // position of the first new token
    if (start < 0) {                                // more new tokens than the sequence has
      record_status(kSiteKvLength);
      r = end;
      continue;
    }
    const int pos = start + (r - begin);
    const int slot = pos % c.P;
    const int n = min(end - r, c.P - slot);         // new tokens of this page from here on
    if (r != begin && slot != 0) {                  // another block owns this page
      r += n;
      continue;
    }
    const int page = kv_page(c, b, pos);
    for (int u0 = blockIdx.y * units; u0 < 2 * c.H; u0 += gridDim.y * units) {
      const int unit = u0 + warp / a.warps;   // head, K | V
      const bool on = unit < 2 * c.H;
      const int h = on ? unit >> 1 : 0;
      const bool is_v = unit & 1;
      const __nv_bfloat16* src = (is_v ? a.v : a.k) + static_cast<long long>(h) * D;
      const long long ld = is_v ? a.ldv : a.ldk;
      int8_t* const codes0 = is_v ? c.v : c.k;
      float* const scales0 = is_v ? c.v_scale : c.k_scale;
      const int pieces = on ? n * L : 0;
      uint4 buf[kKvPieces];
#pragma unroll
      for (int i = 0; i < kKvPieces; ++i) {
        const int p = tid + i * T;
        buf[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p < pieces) buf[i] = reinterpret_cast<const uint4*>(src + (r + p / L) * ld)[p % L];
      }
      const long long ph = static_cast<long long>(page < 0 ? 0 : page) * c.H + h;
      int8_t* codes = codes0 + ph * c.P * D;
      float* scale = scales0 + ph;
      const float s_old = slot > 0 && page >= 0 ? *scale : 0.0f;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kKvPieces; ++i) m = max(m, bf16x8_amax(buf[i]));
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      if (a.warps > 1) {
        if ((threadIdx.x & 31) == 0) amax_warp[warp] = m;
        __syncthreads();
        for (int w = 0; w < a.warps; ++w) m = max(m, amax_warp[warp / a.warps * a.warps + w]);
      }
      const bool finite = m < 0x7F80u;   // (of the unit)
      if (a.warps > 1 ? __syncthreads_or(!finite) : !finite) {   // once more over the finite values
        m = 0;
#pragma unroll
        for (int i = 0; i < kKvPieces; ++i) m = max(m, bf16x8_finite_amax(buf[i]));
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (a.warps > 1) {
          if ((threadIdx.x & 31) == 0) amax_warp[warp] = m;
          __syncthreads();
          for (int w = 0; w < a.warps; ++w) m = max(m, amax_warp[warp / a.warps * a.warps + w]);
        }
      }
      if (on && page >= 0) {
        float s = fmaxf(s_old, __fdiv_rn(__uint_as_float(m << 16), 127.0f));
        if (s < 1.17549435e-38f) s = 0.0f;
        const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
        const float ratio = s > 0.0f ? __fdiv_rn(s_old, s) : 0.0f;
#pragma unroll
        for (int i = 0; i < kKvPieces; ++i) {
          const int p = tid + i * T;
          if (p < pieces) {
            float x[8];
            bf16x8_to_f32(buf[i], x);
            uint2 w = make_uint2(0u, 0u);
            if (finite) {   // (s = 0 has inv = 0)
              w = make_uint2(kv_codes4(x[0], x[1], x[2], x[3], inv), kv_codes4(x[4], x[5], x[6], x[7], inv));
            } else if (s > 0.0f) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                w.x |= kv_code(x[j], inv) << (8 * j);
                w.y |= kv_code(x[4 + j], inv) << (8 * j);
              }
            }
            reinterpret_cast<uint2*>(codes + (slot + p / L) * D)[p % L] = w;
          }
        }
        if (slot > 0 && ratio != 1.0f) {   // the page's earlier tokens take the larger scale
          for (int p = tid; p < slot * (D / 16); p += T) {
            uint4* at = reinterpret_cast<uint4*>(codes) + p;
            const uint4 w = *at;
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 16; ++j)
              o[j / 4] |= kv_code(static_cast<float>(static_cast<int8_t>(in[j / 4] >> (8 * (j % 4)))), ratio) << (8 * (j % 4));
            *at = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      if (a.warps > 1) __syncthreads(); else __syncwarp();   // the unit has read its old scale and the maxima
      if (on && page >= 0 && tid == 0) {
        float s = fmaxf(s_old, __fdiv_rn(__uint_as_float(m << 16), 127.0f));
        *scale = s < 1.17549435e-38f ? 0.0f : s;
      }
    }
    r += n;
  }
}

struct KvReadArgs {
  KvView c;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  long long ldk, ldv;
  int heads;   // of a block
};

constexpr int kKvReadThreads = 128;

// grid (chunks of R rows, K | V, groups of heads). One search finds the first row's sequence;
// each row's lane walks on from there and looks its page up, so the rows'
// lookups run side by side. Then the block walks heads, rows and 8-byte
// pieces of codes (16 bytes out, so a warp's stores are whole lines): neighbouring rows of a page are neighbours in memory, so a
// head's rows are one run of codes.
template <int D, int R>
__global__ void __launch_bounds__(kKvReadThreads) kv_read_kernel(const KvReadArgs a) {
  constexpr int L = D / 8;   // 8-byte pieces of a token's codes
  __shared__ int page_of[R], slot_of[R];
  const KvView& c = a.c;
  const int tid = threadIdx.x;
  const bool is_v = blockIdx.y != 0;
  const int8_t* const codes = is_v ? c.v : c.k;
  const float* const scales = is_v ? c.v_scale : c.k_scale;
  __nv_bfloat16* const out = is_v ? a.v : a.k;
  const long long ld = is_v ? a.ldv : a.ldk;
  const int r0 = blockIdx.x * R;

  grid_dep_wait();
  grid_dep_launch();
  if (tid < 32) {
    int b = kv_find(c, r0);
    const int r = r0 + tid;
    int page = -1, slot = 0;
    if (tid < R && r < c.N) {
      if (c.cu == nullptr) b = r / c.per;
      else
        while (b < c.B && c.cu[b + 1] <= r) ++b;
      int begin, end, len;
      if (b < c.B && kv_rows(c, b, begin, end, len) && r >= begin && r < end) {
        const int pos = len - (end - r);
        if (pos >= 0) {
          page = kv_page(c, b, pos);
          slot = pos % c.P;
        } else {
          record_status(kSiteKvLength);
        }
      }
    }
    if (tid < R) {
      page_of[tid] = page;
      slot_of[tid] = slot;
    }
  }
  __syncthreads();
  // this block's heads
  const int h0 = blockIdx.z * a.heads, nh = min(a.heads, c.H - h0);
  const int total = nh * R * L;
  constexpr int U = 8;   // pieces of a thread in flight
  for (int p0 = tid; p0 < total; p0 += U * kKvReadThreads) {
    uint2 w[U];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + u * kKvReadThreads;
      const int row = (p / L) % R, h = h0 + p / (L * R);
      w[u] = make_uint2(0u, 0u);
      s[u] = 0.0f;
      if (p < total && page_of[row] >= 0) {
        const long long ph = static_cast<long long>(page_of[row]) * c.H + h;
        w[u] = reinterpret_cast<const uint2*>(codes + (ph * c.P + slot_of[row]) * D)[p % L];
        s[u] = scales[ph];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + u * kKvReadThreads;
      const int row = (p / L) % R, h = h0 + p / (L * R);
      if (p >= total || page_of[row] < 0) continue;
      const uint32_t in[2] = {w[u].x, w[u].y};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {   // (a bit trick in place of the conversion took more registers: 34 us against 30)
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(static_cast<float>(static_cast<int8_t>(in[i] >> (8 * j))), s[u]);
        o[2 * i] = pack_bf16x2(x[0], x[1]);
        o[2 * i + 1] = pack_bf16x2(x[2], x[3]);
      }
      reinterpret_cast<uint4*>(out + (r0 + row) * ld + static_cast<long long>(h) * D)[p % L] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace respin
