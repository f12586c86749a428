// Host side of the attention half of a layer (head norms and rotation, the
// 8-bit cache, attention over it): argument checks and launches. Included at
// the end of respin_lib.cu, whose error reporting and launch helpers it uses.
#pragma once

namespace {

bool kv_head_dim_ok(int d) { return d == 64 || d == 128; }

// Elements between tokens: whole 16-byte pieces, no overlap of tokens.
bool kv_ld_ok(long long ld, long long row) { return ld >= row && ld % 8 == 0; }

respin_status_t kv_check(const respin_kv_cache_t* c, const respin_kv_batch_t* b, KvView* v) {
  if (c == nullptr || b == nullptr) return fail(RESPIN_ERR_INVALID_ARG, "cache and batch must be non-NULL");
  if (!kv_head_dim_ok(c->head_dim))
    return fail(RESPIN_ERR_UNSUPPORTED, "head_dim=%d: need 64 or 128", c->head_dim);
  const int P = c->page_size;
  if (P != 16 && P != 32 && P != 64 && P != 128)
    return fail(RESPIN_ERR_UNSUPPORTED, "page_size=%d: need 16, 32, 64 or 128", P);
  if (c->kv_heads < 1 || c->kv_heads > 1024)
    return fail(RESPIN_ERR_UNSUPPORTED, "kv_heads=%d: need 1 .. 1024", c->kv_heads);
  if (c->num_pages < 1) return fail(RESPIN_ERR_INVALID_ARG, "num_pages=%d: need at least 1", c->num_pages);
  if (static_cast<long long>(c->num_pages) * c->kv_heads * P > 0x7FFFFFFFLL)
    return fail(RESPIN_ERR_UNSUPPORTED, "num_pages * kv_heads * page_size = %lld tokens: at most 2^31 - 1",
                static_cast<long long>(c->num_pages) * c->kv_heads * P);
  if (b->B < 0 || b->N < 0) return fail(RESPIN_ERR_INVALID_ARG, "B=%d and N=%d must not be negative", b->B, b->N);
  if (b->B > 65536) return fail(RESPIN_ERR_UNSUPPORTED, "B=%d: at most 65536 sequences", b->B);
  if (b->max_pages < 1 || static_cast<long long>(b->max_pages) * P > 0x7FFF0000LL)
    return fail(RESPIN_ERR_INVALID_ARG, "max_pages=%d: need at least 1, and max_pages * page_size at most 2^31 - 2^16", b->max_pages);
  if (b->N == 0 || b->B == 0) {
    if (b->N != 0) return fail(RESPIN_ERR_INVALID_ARG, "N=%d tokens of no sequence", b->N);
    return ok();
  }
  if (b->cu == nullptr && b->N % b->B)
    return fail(RESPIN_ERR_INVALID_ARG, "N=%d is not a multiple of B=%d: cu is needed", b->N, b->B);
  if (c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr ||
      b->kv_len == nullptr || b->block_table == nullptr)
    return fail(RESPIN_ERR_INVALID_ARG, "a required pointer of the cache or the batch is NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(RESPIN_ERR_ALIGNMENT, "the cache's codes must be 16-byte aligned");
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(b->cu, 4) || !aligned(b->kv_len, 4) ||
      !aligned(b->block_table, 4))
    return fail(RESPIN_ERR_ALIGNMENT, "scales, cu, kv_len and block_table must be 4-byte aligned");
  *v = KvView{c->k, c->v, c->k_scale, c->v_scale, c->num_pages, P, c->kv_heads, b->cu, b->kv_len, b->block_table,
              b->B, b->max_pages, b->N, b->N / b->B};
  return ok();
}

cudaError_t launch_dependent3(const void* fn, dim3 grid, int block, size_t smem, cudaStream_t s, void** args) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = grid;
  lc.blockDim = dim3(static_cast<unsigned>(block), 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelExC(&lc, fn, args);
}

struct KvAttnVariant {
  const void* fn;
  size_t smem;
  int threads;
  int rows;            // of a partial result
  long long slot;      // floats of one
};

template <int D, int NT>
KvAttnVariant kv_few() {
  using C = KvAttnCfg<D, NT>;
  return {reinterpret_cast<const void*>(&kv_attn_kernel<D, NT>), static_cast<size_t>(C::Smem), kKvThreads, C::RB,
          static_cast<long long>(C::SlotFloats)};
}

template <int D>
KvAttnVariant kv_many() {
  using C = TcaCfg<D>;
  return {reinterpret_cast<const void*>(&kv_attn_tc_kernel<D>), static_cast<size_t>(C::Smem), kTcaThreads, kTcaGroup,
          static_cast<long long>(C::SlotFloats)};
}

// 3-D tensor map over bf16 [N][heads][D] with ld elements between tokens, box
// {D, box_heads, box_tokens}; tokens past the end read as zeros.
bool make_tmap_heads(CUtensorMap* m, const void* ptr, int N, int heads, int D, long long ld, int box_heads, int box_tokens) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(N)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(box_heads),
                             static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kKvVariants = 6;

// Variants 0, 1: at most 8 rows a key head (single tokens: one n = 8 product)
// or kKvFewRows; 2: more (tensor memory). Then the same for head_dim 128.
KvAttnVariant kv_variant(int i) {
  switch (i) {
    case 0: return kv_few<64, 1>();
    case 1: return kv_few<64, 2>();
    case 2: return kv_many<64>();
    case 3: return kv_few<128, 1>();
    case 4: return kv_few<128, 2>();
    default: return kv_many<128>();
  }
}

struct KvDeviceInfo {
  bool ready = false;
  int sms = 0;
  int occ[kKvVariants] = {0, 0, 0, 0, 0, 0};   // resident blocks per SM
};

cudaError_t kv_prepare(int dev, KvDeviceInfo* info) {
  static std::mutex mu;
  static KvDeviceInfo infos[256];
  if (dev < 0 || dev >= 256) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  KvDeviceInfo& d = infos[dev];
  if (!d.ready) {
    cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    for (int i = 0; i < kKvVariants && e == cudaSuccess; ++i) {
      const KvAttnVariant v = kv_variant(i);
      e = cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(v.smem));
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.occ[i], v.fn, v.threads, v.smem);
      if (e == cudaSuccess && d.occ[i] < 1) e = cudaErrorInvalidConfiguration;
    }
    if (e != cudaSuccess) return e;
    d.ready = true;
  }
  *info = d;
  return cudaSuccess;
}

// What a call launches and how its workspace is laid out: the plans and the
// partial results of both kernels.
struct KvLayout {
  int few, many;          // variants; many < 0: not launched
  long long part_few, part_many, bytes;
};

KvLayout kv_layout(int D, long long rows) {
  KvLayout l;
  const int v0 = D == 64 ? 0 : 3;
  l.few = rows <= 8 ? v0 : v0 + 1;
  l.many = rows > kKvFewRows ? v0 + 2 : -1;
  l.part_few = 16LL * kKvPlan * (kKvMaxBlocks + kTcaMaxBlocks);
  l.part_many = l.part_few + 2LL * kKvMaxBlocks * kv_variant(l.few).slot * 4;
  l.bytes = l.part_many + (l.many < 0 ? 0 : 2LL * kTcaMaxBlocks * kv_variant(l.many).slot * 4);
  return l;
}

}  // namespace

extern "C" {

respin_status_t respin_qk_norm_rope(const void* q, const void* k, int N, int q_heads, int kv_heads, int head_dim,
                                    long long ld_q, long long ld_k, const void* q_weight, const void* k_weight,
                                    float eps, const int32_t* positions, const float* inv_freq, int rot_dim,
                                    int interleaved, void* q_out, void* k_out, long long ld_qo, long long ld_ko,
                                    void* stream) {
  t_last_error.clear();
  if (N < 0) return fail(RESPIN_ERR_INVALID_ARG, "N=%d is negative", N);
  if (!kv_head_dim_ok(head_dim)) return fail(RESPIN_ERR_UNSUPPORTED, "head_dim=%d: need 64 or 128", head_dim);
  if (q_heads < 0 || kv_heads < 0 || q_heads + kv_heads < 1 || q_heads > 1024 || kv_heads > 1024)
    return fail(RESPIN_ERR_UNSUPPORTED, "q_heads=%d, kv_heads=%d: need 0 .. 1024 and one at least", q_heads, kv_heads);
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16)
    return fail(RESPIN_ERR_UNSUPPORTED, "rot_dim=%d: need a multiple of 16 up to head_dim", rot_dim);
  if ((q_weight != nullptr || k_weight != nullptr) && !(eps >= 1e-20f && eps < 1e20f))
    return fail(RESPIN_ERR_INVALID_ARG, "eps=%g: need 1e-20 <= eps < 1e20", static_cast<double>(eps));
  if (N == 0) return ok();
  if ((q_heads > 0 && (q == nullptr || q_out == nullptr)) || (kv_heads > 0 && (k == nullptr || k_out == nullptr)) ||
      (rot_dim > 0 && (positions == nullptr || inv_freq == nullptr)))
    return fail(RESPIN_ERR_INVALID_ARG, "a required pointer is NULL");
  const long long rq = static_cast<long long>(q_heads) * head_dim, rk = static_cast<long long>(kv_heads) * head_dim;
  if (!kv_ld_ok(ld_q, rq) || !kv_ld_ok(ld_qo, rq) || !kv_ld_ok(ld_k, rk) || !kv_ld_ok(ld_ko, rk))
    return fail(RESPIN_ERR_INVALID_ARG, "token strides must be multiples of 8 elements and at least heads * head_dim");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16))
    return fail(RESPIN_ERR_ALIGNMENT, "q, k, their outputs and the weights must be 16-byte aligned");
  if (!aligned(positions, 4) || !aligned(inv_freq, 4))
    return fail(RESPIN_ERR_ALIGNMENT, "positions and inv_freq must be 4-byte aligned");
  if (fault_at("launch")) return fail(RESPIN_ERR_CUDA, "injected fault at launch");

  typedef __nv_bfloat16 bf16;
  RopeArgs a{static_cast<const bf16*>(q), static_cast<const bf16*>(k), static_cast<bf16*>(q_out), static_cast<bf16*>(k_out),
             static_cast<const bf16*>(q_weight), static_cast<const bf16*>(k_weight), positions, inv_freq,
             ld_q, ld_k, ld_qo, ld_ko, N, q_heads, kv_heads, rot_dim, 1, eps};
  // Many tokens: as many a block as make one wave of five blocks on each of 148 SMs, at most 8 (their
  // sines and cosines are formed once for all heads). Few: one, and its vectors go to several blocks.
  a.tokens = N < 592 ? 1 : N >= 8 * 740 ? 8 : (N + 739) / 740;
  const int V = kRopeThreads / (head_dim / 8);
  const int passes = (a.tokens * (q_heads + kv_heads) + V - 1) / V;
  const int y = N >= 592 ? 1 : passes;
  const dim3 grid(static_cast<unsigned>((N + a.tokens - 1) / a.tokens), static_cast<unsigned>(y), 1);
  const size_t smem = static_cast<size_t>(a.tokens) * (rot_dim / 2) * sizeof(float2);
  const void* fn = head_dim == 64 ? (interleaved ? reinterpret_cast<const void*>(&qk_norm_rope_kernel<64, true>)
                                                 : reinterpret_cast<const void*>(&qk_norm_rope_kernel<64, false>))
                                  : (interleaved ? reinterpret_cast<const void*>(&qk_norm_rope_kernel<128, true>)
                                                 : reinterpret_cast<const void*>(&qk_norm_rope_kernel<128, false>));
  void* args[] = {&a};
  cudaError_t e = launch_dependent3(fn, grid, kRopeThreads, smem, static_cast<cudaStream_t>(stream), args);
  if (e != cudaSuccess) return cuda_fail(e, "qk_norm_rope_kernel launch");
  return ok();
}

respin_status_t respin_kv_append(const respin_kv_cache_t* cache, const respin_kv_batch_t* batch, const void* k,
                                 const void* v, long long ld_k, long long ld_v, void* stream) {
  t_last_error.clear();
  KvAppendArgs a{};
  respin_status_t st = kv_check(cache, batch, &a.c);
  if (st != RESPIN_OK || batch->N == 0) return st;
  if (k == nullptr || v == nullptr) return fail(RESPIN_ERR_INVALID_ARG, "k and v must be non-NULL");
  const int D = cache->head_dim, P = cache->page_size;
  const long long row = static_cast<long long>(cache->kv_heads) * D;
  if (!kv_ld_ok(ld_k, row) || !kv_ld_ok(ld_v, row))
    return fail(RESPIN_ERR_INVALID_ARG, "token strides must be multiples of 8 elements and at least kv_heads * head_dim");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(RESPIN_ERR_ALIGNMENT, "k and v must be 16-byte aligned");
  if (fault_at("launch")) return fail(RESPIN_ERR_CUDA, "injected fault at launch");
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.ldk = ld_k;
  a.ldv = ld_v;
  // A block's rows: about one sequence's, at most a page, so that a decode
  // step has a block for each sequence and a prefill one for each page.
  const int per = batch->N / batch->B;
  a.rows = per < 1 ? 1 : per > P ? P : per;
  a.warps = P * D / 8 / (32 * kKvPieces);
  if (a.warps < 1) a.warps = 1;
  // Groups of units side by side until there are three blocks for each of 148 SMs; the rest in turn.
  const int units = 8 / a.warps, groups = (2 * cache->kv_heads + units - 1) / units;
  const int chunks = (batch->N + a.rows - 1) / a.rows;
  int y = (3 * 148 + chunks - 1) / chunks;
  if (y > groups) y = groups;
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(y), 1);
  void* args[] = {&a};
  cudaError_t e = launch_dependent3(D == 64 ? reinterpret_cast<const void*>(&kv_append_kernel<64>)
                                            : reinterpret_cast<const void*>(&kv_append_kernel<128>),
                                    grid, kKvAppendThreads, 0, static_cast<cudaStream_t>(stream), args);
  if (e != cudaSuccess) return cuda_fail(e, "kv_append_kernel launch");
  return ok();
}

respin_status_t respin_kv_read(const respin_kv_cache_t* cache, const respin_kv_batch_t* batch, void* k_out,
                               void* v_out, long long ld_k, long long ld_v, void* stream) {
  t_last_error.clear();
  KvReadArgs a{};
  respin_status_t st = kv_check(cache, batch, &a.c);
  if (st != RESPIN_OK || batch->N == 0) return st;
  if (k_out == nullptr || v_out == nullptr) return fail(RESPIN_ERR_INVALID_ARG, "k_out and v_out must be non-NULL");
  const long long row = static_cast<long long>(cache->kv_heads) * cache->head_dim;
  if (!kv_ld_ok(ld_k, row) || !kv_ld_ok(ld_v, row))
    return fail(RESPIN_ERR_INVALID_ARG, "token strides must be multiples of 8 elements and at least kv_heads * head_dim");
  if (!aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(RESPIN_ERR_ALIGNMENT, "k_out and v_out must be 16-byte aligned");
  if (fault_at("launch")) return fail(RESPIN_ERR_CUDA, "injected fault at launch");
  a.k = static_cast<__nv_bfloat16*>(k_out);
  a.v = static_cast<__nv_bfloat16*>(v_out);
  a.ldk = ld_k;
  a.ldv = ld_v;
  // 32 rows a block share the lookups; 8 where that leaves SMs without a block. A block takes as many
  // heads as make 2048 pieces of 8 bytes (16 a thread): more of them hide one another's lookups.
  const bool few = batch->N < 32 * 148;
  const void* fn = cache->head_dim == 64 ? (few ? reinterpret_cast<const void*>(&kv_read_kernel<64, 8>)
                                                : reinterpret_cast<const void*>(&kv_read_kernel<64, 32>))
                                         : (few ? reinterpret_cast<const void*>(&kv_read_kernel<128, 8>)
                                                : reinterpret_cast<const void*>(&kv_read_kernel<128, 32>));
  const int R = few ? 8 : 32;
  a.heads = 1024 / (R * cache->head_dim / 16);
  const dim3 grid(static_cast<unsigned>((batch->N + R - 1) / R), 2,
                  static_cast<unsigned>((cache->kv_heads + a.heads - 1) / a.heads));
  void* args[] = {&a};
  cudaError_t e = launch_dependent3(fn, grid, kKvReadThreads, 0, static_cast<cudaStream_t>(stream), args);
  if (e != cudaSuccess) return cuda_fail(e, "kv_read_kernel launch");
  return ok();
}

// Rows a key head has in the longest call: max_q tokens (0: unknown, N) of
// its query heads.
static long long kv_attn_rows(int N, int max_q, int G) {
  return static_cast<long long>(max_q > 0 && max_q < N ? max_q : N) * G;
}

respin_status_t respin_kv_attention_workspace(int q_heads, int kv_heads, int head_dim, int N, int max_q,
                                              long long* bytes) {
  t_last_error.clear();
  if (bytes == nullptr) return fail(RESPIN_ERR_INVALID_ARG, "bytes is NULL");
  if (!kv_head_dim_ok(head_dim)) return fail(RESPIN_ERR_UNSUPPORTED, "head_dim=%d: need 64 or 128", head_dim);
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || N < 0 || max_q < 0)
    return fail(RESPIN_ERR_INVALID_ARG, "q_heads=%d must be a positive multiple of kv_heads=%d, N=%d and max_q=%d not negative",
                q_heads, kv_heads, N, max_q);
  *bytes = kv_layout(head_dim, kv_attn_rows(N, max_q, q_heads / kv_heads)).bytes;
  return ok();
}

respin_status_t respin_kv_attention(const respin_kv_cache_t* cache, const respin_kv_batch_t* batch, const void* q,
                                    int q_heads, long long ld_q, int max_q, int causal, int window, float scale,
                                    void* out, long long ld_out, float* lse, void* workspace,
                                    long long workspace_bytes, void* stream) {
  t_last_error.clear();
  KvAttnArgs a{};
  respin_status_t st = kv_check(cache, batch, &a.c);
  if (st != RESPIN_OK) return st;
  const int D = cache->head_dim, H = cache->kv_heads;
  if (q_heads < 1 || q_heads > 1024 || q_heads % H)
    return fail(RESPIN_ERR_UNSUPPORTED, "q_heads=%d: need a multiple of kv_heads=%d up to 1024", q_heads, H);
  if (max_q < 0 || window < 0) return fail(RESPIN_ERR_INVALID_ARG, "max_q=%d and window=%d must not be negative", max_q, window);
  if (window > 0 && !causal) return fail(RESPIN_ERR_INVALID_ARG, "a window needs causal");
  if (!(scale > -1e30f && scale < 1e30f)) return fail(RESPIN_ERR_INVALID_ARG, "scale must be finite (below 1e30)");
  if (batch->N == 0) return ok();
  if (static_cast<long long>(batch->N) * (q_heads / H) > 0x7FFFFFFFLL)
    return fail(RESPIN_ERR_UNSUPPORTED, "N * q_heads / kv_heads = %lld rows: at most 2^31 - 1",
                static_cast<long long>(batch->N) * (q_heads / H));
  // Tiles of 64 tokens (a unit's fixed cost aside) in both kernels' lines of work at most: a sequence has
  // one row group of few rows, or one for each 256 rows and a part. A block's piece is counted in 32 bits;
  // both kernels have 128 blocks at least.
  const long long line = H * (batch->B + static_cast<long long>(batch->N) * (q_heads / H) / kTcaGroup) *
                         (static_cast<long long>(batch->max_pages) * cache->page_size / kKvTile + 1 + kTcaUnitCost);
  if (line > 1LL << 38)
    return fail(RESPIN_ERR_UNSUPPORTED, "kv_heads * (B + rows / 256) * max_pages * page_size / 64 = %lld: at most 2^38", line);
  if (batch->cu == nullptr) max_q = batch->N / batch->B;   // what it is, whatever was given
  if (q == nullptr || out == nullptr || workspace == nullptr)
    return fail(RESPIN_ERR_INVALID_ARG, "q, out and workspace must be non-NULL");
  const long long row = static_cast<long long>(q_heads) * D;
  if (!kv_ld_ok(ld_q, row) || !kv_ld_ok(ld_out, row))
    return fail(RESPIN_ERR_INVALID_ARG, "token strides must be multiples of 8 elements and at least q_heads * head_dim");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16))
    return fail(RESPIN_ERR_ALIGNMENT, "q, out and workspace must be 16-byte aligned");
  if (!aligned(lse, 4)) return fail(RESPIN_ERR_ALIGNMENT, "lse must be 4-byte aligned");
  long long need = 0;
  st = respin_kv_attention_workspace(q_heads, H, D, batch->N, max_q, &need);
  if (st != RESPIN_OK) return st;
  if (workspace_bytes < need)
    return fail(RESPIN_ERR_INVALID_ARG, "workspace of %lld bytes: need %lld", workspace_bytes, need);
  if (fault_at("launch")) return fail(RESPIN_ERR_CUDA, "injected fault at launch");

  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  KvDeviceInfo info;
  e = kv_prepare(dev, &info);
  if (e != cudaSuccess) return cuda_fail(e, "preparing kv_attn_kernel");
  const int G = q_heads / H;
  const long long most = kv_attn_rows(batch->N, max_q, G);
  const KvLayout lay = kv_layout(D, most);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.ldq = ld_q;
  a.ldo = ld_out;
  a.Hq = q_heads;
  a.G = G;
  a.causal = causal != 0;
  a.window = window < static_cast<long long>(batch->max_pages) * cache->page_size ? window : 0;   // else it hides nothing
  a.scale = scale * 1.44269504088896340736f;
  a.div_g = G == 1 ? 0ull : ~0ull / static_cast<unsigned long long>(G) + 1ull;
  a.few_rows = most < kKvFewRows ? static_cast<int>(most) : kKvFewRows;
  a.others = lay.many >= 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  // Sequences of many rows, then those of few; a uniform batch has one kind.
  KvJoin few{reinterpret_cast<int4*>(ws), reinterpret_cast<float*>(ws + lay.part_few), 0, kv_variant(lay.few).rows, 0};
  KvJoin many{reinterpret_cast<int4*>(ws + 16 * kKvPlan * kKvMaxBlocks), reinterpret_cast<float*>(ws + lay.part_many), 0, kTcaGroup, 0};
  const uint64_t rows = static_cast<uint64_t>(cache->num_pages) * H * cache->page_size;
  const uint32_t box = cache->page_size < kKvTile ? cache->page_size : kKvTile;   // both kernels' 64-token tiles
  CUtensorMap tmK, tmV;
  if (lay.many >= 0) {
    const KvAttnVariant v = kv_variant(lay.many);
    many.blocks = info.sms < kTcaMaxBlocks ? info.sms : kTcaMaxBlocks;
    if (!make_tmap_u8(&tmK, cache->k, rows, D, box, D) || !make_tmap_u8(&tmV, cache->v, rows, D, box, D))
      return fail(RESPIN_ERR_CUDA, "cuTensorMapEncodeTiled failed for the cache");
    const int slot_rows = kTcaSlot / (2 * D);
    CUtensorMap tmQ;
    if (!make_tmap_heads(&tmQ, q, batch->N, q_heads, D, ld_q, slot_rows % G ? 1 : G, slot_rows % G ? 1 : slot_rows / G))
      return fail(RESPIN_ERR_CUDA, "cuTensorMapEncodeTiled failed for the queries");
    a.plan = const_cast<int4*>(many.plan);
    a.part = const_cast<float*>(many.part);
    void* args[] = {&tmQ, &tmK, &tmV, &a};
    e = launch_dependent3(v.fn, dim3(static_cast<unsigned>(many.blocks), 1, 1), v.threads, v.smem, s, args);
    if (e != cudaSuccess) return cuda_fail(e, "kv_attn_tc_kernel launch");
  }
  if (lay.many < 0 || batch->cu != nullptr) {
    const KvAttnVariant v = kv_variant(lay.few);
    few.blocks = info.occ[lay.few] * info.sms < kKvMaxBlocks ? info.occ[lay.few] * info.sms : kKvMaxBlocks;
    const CUtensorMapSwizzle swz = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!make_tmap_u8(&tmK, cache->k, rows, D, box, D, swz) || !make_tmap_u8(&tmV, cache->v, rows, D, box, D, swz))
      return fail(RESPIN_ERR_CUDA, "cuTensorMapEncodeTiled failed for the cache");
    a.plan = const_cast<int4*>(few.plan);
    a.part = const_cast<float*>(few.part);
    void* args[] = {&tmK, &tmV, &a};
    e = launch_dependent3(v.fn, dim3(static_cast<unsigned>(few.blocks), 1, 1), v.threads, v.smem, s, args);
    if (e != cudaSuccess) return cuda_fail(e, "kv_attn_kernel launch");
  }
  few.parts = few.rows * D / 4 / 64;   // 4 or 8 at head_dim 128, 2 or 4 at 64
  many.parts = D / 8;
  const int joins = (few.blocks > 0 ? (few.blocks - 1) * few.parts : 0) + (many.blocks > 0 ? (many.blocks - 1) * many.parts : 0);
  if (joins > 0) {
    void* args[] = {&a, &few, &many};
    e = launch_dependent3(D == 64 ? reinterpret_cast<const void*>(&kv_combine_kernel<64>)
                                  : reinterpret_cast<const void*>(&kv_combine_kernel<128>),
                          dim3(static_cast<unsigned>(joins), 1, 1), kKvJoinThreads, 0, s, args);
    if (e != cudaSuccess) return cuda_fail(e, "kv_combine_kernel launch");
  }
  return ok();
}

}  // extern "C"
