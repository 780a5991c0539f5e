// C entry points around a verification round: sampling, truncation and the paged cache.
// Argument checks and launches.
#pragma once

namespace specv {

// ---------------------------------------------------------------------------
// Sampling and truncation.
// ---------------------------------------------------------------------------

// CTAs per row: one where the rows cover the SMs, else as many as do, each with some
// thousand entries.
constexpr size_t kSampleRunBytes = 16384;
inline int sample_cluster(const SampleParams& p, size_t es, int sms) {
  int c = 1;
  while (c < kSampleMaxCluster && (long long)p.rows * c < sms &&
         (size_t)p.V * es >= 2 * c * kSampleRunBytes)
    c *= 2;
  return c;
}

template <typename TIn>
spec_status_t sample_run(const SampleParams& p, cudaStream_t stream) {
  DeviceInfo* d = nullptr;
  if (device_info(&d) != cudaSuccess) return SPEC_ERR_CUDA;
  const int c = sample_cluster(p, sizeof(TIn), d->sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.rows * c));
  cfg.blockDim = dim3(kSampleThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<TIn>, p) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

inline spec_status_t sample_entry(const char* name, const void* logits, spec_dtype_t dtype,
                                  int rows, int V, int group, const float* temperature,
                                  const int32_t* top_k, const float* top_p, const float* min_p,
                                  const float* uniforms, int32_t* tokens, bool want_tokens,
                                  void* kept, bool want_kept, void* stream) {
  if (rows < 1 || V < 1 || group < 1) return SPEC_ERR_INVALID_ARG;
  if (rows > SPEC_MAX_ROWS || V > SPEC_MAX_V) return SPEC_ERR_UNSUPPORTED;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (!logits || !temperature || (want_tokens && (!tokens || !uniforms)) || (want_kept && !kept))
    return SPEC_ERR_INVALID_ARG;
  const size_t es = dtype == SPEC_F32 ? 4 : 2;
  if (!aligned(logits, es) || !aligned(kept, es)) return SPEC_ERR_INVALID_ARG;
  const size_t n4 = (size_t)rows * 4, g4 = ((size_t)rows + group - 1) / group * 4;
  const struct {
    const void* p;
    size_t n;
  } in[5] = {{temperature, g4}, {top_k, g4}, {top_p, g4}, {min_p, g4}, {uniforms, n4}};
  const size_t nl = (size_t)rows * V * es;
  for (const auto& b : in) {
    if (!aligned(b.p, 4)) return SPEC_ERR_INVALID_ARG;
    if (b.p && (overlap(tokens, tokens ? n4 : 0, b.p, b.n) ||
                overlap(kept, kept ? nl : 0, b.p, b.n)))
      return SPEC_ERR_INVALID_ARG;
  }
  if (!aligned(tokens, 4) || overlap(tokens, tokens ? n4 : 0, logits, nl) ||
      overlap(tokens, tokens ? n4 : 0, kept, kept ? nl : 0))
    return SPEC_ERR_INVALID_ARG;
  if (kept && kept != logits && overlap(kept, nl, logits, nl)) return SPEC_ERR_INVALID_ARG;
  NvtxRange r(name);
  DeviceOf on_device(logits);
  if (!on_device.ok()) return SPEC_ERR_CUDA;
  if (!on_device.device()) return SPEC_ERR_INVALID_ARG;
  SampleParams p = {};
  p.logits = logits;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.uniforms = uniforms;
  p.tokens = tokens;
  p.kept = kept;
  p.rows = rows;
  p.V = V;
  p.group = group;
  p.unit_bits = sample_unit_bits(V);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == SPEC_F32 ? sample_run<float>(p, s) : sample_run<uint16_t>(p, s);
}

// ---------------------------------------------------------------------------
// The paged cache.
// ---------------------------------------------------------------------------

// Bytes from a cache's base to behind its last entry; 0: strides that do not fit.
inline size_t cache_extent(const spec_paged_cache_t& c, long long page, long long slot,
                           long long head) {
  const long long most = 1ll << 38;
  for (long long s : {page, slot, head})
    if (s < c.width || s > most || s % 8 != 0) return 0;
  const unsigned __int128 n = (unsigned __int128)(c.num_pages - 1) * (uint64_t)page +
                              (unsigned __int128)(c.page_size - 1) * (uint64_t)slot +
                              (unsigned __int128)(c.kv_heads - 1) * (uint64_t)head + c.width;
  return n > ((unsigned __int128)1 << 46) ? 0 : (size_t)n * 2;
}

// A copy of the caller's description, checked; strides of what there is only one of
// do not matter and are set to the width.
inline spec_status_t cache_check(const spec_paged_cache_t* in, spec_dtype_t dtype, int rows,
                                 spec_paged_cache_t* out, size_t* k_bytes, size_t* v_bytes) {
  if (!in) return SPEC_ERR_INVALID_ARG;
  spec_paged_cache_t c = *in;
  if (rows < 1 || c.B < 1 || c.num_pages < 1 || c.page_size < 1 || c.kv_heads < 1 || c.width < 1 ||
      c.max_pages < 1)
    return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_BF16 || rows > SPEC_MAX_ROWS || c.B > SPEC_MAX_B || c.page_size < 8 ||
      c.page_size > 1024 || (c.page_size & (c.page_size - 1)) != 0 || c.kv_heads > 1024 ||
      (c.width != 64 && c.width != 128) || (long long)c.max_pages * c.page_size > (1 << 30))
    return SPEC_ERR_UNSUPPORTED;
  if (!c.k_cache || !c.v_cache || !c.page_table || !c.new_start || !c.kv_len)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(c.k_cache, 16) || !aligned(c.v_cache, 16) || !aligned(c.page_table, 4) ||
      !aligned(c.new_start, 4) || !aligned(c.kv_len, 4))
    return SPEC_ERR_INVALID_ARG;
  if (c.num_pages == 1) c.k_page = c.v_page = c.width;
  if (c.kv_heads == 1) c.k_head = c.v_head = c.width;
  *k_bytes = cache_extent(c, c.k_page, c.k_slot, c.k_head);
  *v_bytes = cache_extent(c, c.v_page, c.v_slot, c.v_head);
  if (*k_bytes == 0 || *v_bytes == 0) return SPEC_ERR_INVALID_ARG;
  *out = c;
  return SPEC_OK;
}

// Whether [a, a + na) shares a byte with the cache or its tables.
inline bool meets_tables(const spec_paged_cache_t& c, const void* a, size_t na) {
  return overlap(a, na, c.page_table, (size_t)c.B * c.max_pages * 4) ||
         overlap(a, na, c.new_start, ((size_t)c.B + 1) * 4) ||
         overlap(a, na, c.kv_len, (size_t)c.B * 4);
}

inline bool row_stride_ok(long long stride, long long row) {
  return stride >= row && stride % 8 == 0 && stride <= (1ll << 38);
}

inline bool attn_sizes_ok(int rows, int heads, int kv_heads, int width) {
  return rows >= 1 && heads >= 1 && kv_heads >= 1 && rows <= SPEC_MAX_ROWS && heads <= 1024 &&
         heads % kv_heads == 0 && (width == 64 || width == 128) &&
         (long long)rows * heads <= (1 << 30);
}

struct AttnLayout {
  size_t ctas, met, stats, parts, total;
  int slot_rows;
};
inline AttnLayout attn_layout(int rows, int heads, int kv_heads, int width) {
  AttnLayout l;
  l.slot_rows = (int)std::min<long long>(kAtUnitRows, (long long)rows * (heads / kv_heads));
  l.ctas = align256(sizeof(WsHeader));
  l.met = l.ctas + align256(kAtMaxCtas * sizeof(AtCta));
  l.stats = l.met + align256(kAtMaxCtas * sizeof(int));
  l.parts = l.stats + align256((size_t)2 * kAtMaxCtas * l.slot_rows * sizeof(float2));
  l.total = l.parts + align256((size_t)2 * kAtMaxCtas * l.slot_rows * width * sizeof(float));
  return l;
}

// Tensor map of a cache: [pages, heads, slots, width] in boxes of up to 128 slots x 64 entries
// with the 128-byte swizzle.
inline bool attn_map(CUtensorMap* m, const spec_paged_cache_t& c, void* base, long long page,
                     long long slot, long long head) {
  EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)c.width, (cuuint64_t)c.page_size,
                              (cuuint64_t)c.kv_heads, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)slot * 2, (cuuint64_t)head * 2, (cuuint64_t)page * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)std::min(c.page_size, kAtTile), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline cudaError_t attn_prepare(DeviceInfo* d) {
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (d->attn_ready) return cudaSuccess;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(paged_attention_kernel<64>, attr, at_smem<64>())) != cudaSuccess)
    return e;
  if ((e = cudaFuncSetAttribute(paged_attention_kernel<128>, attr, at_smem<128>())) != cudaSuccess)
    return e;
  d->attn_ready = true;
  return cudaSuccess;
}

template <int D>
spec_status_t attn_run(const PagedParams& p, unsigned char* ws, cudaStream_t s) {
  DeviceInfo* d = nullptr;
  if (device_info(&d) != cudaSuccess || attn_prepare(d) != cudaSuccess) return SPEC_ERR_CUDA;
  const AttnLayout lay = attn_layout(p.rows, p.heads, p.c.kv_heads, D);
  AtParams a = {};
  a.p = p;
  a.p.header = reinterpret_cast<WsHeader*>(ws);
  a.group = p.heads / p.c.kv_heads;
  int bits = 0;
  while ((1 << bits) < a.group) ++bits;
  a.shift = 31 + bits;
  a.magic = (uint32_t)(((1ull << a.shift) + a.group - 1) / a.group);
  while ((1 << a.page_bits) < p.c.page_size) ++a.page_bits;
  a.slot_rows = lay.slot_rows;
  a.scale2 = p.scale * kLog2e;
  a.ctas = reinterpret_cast<AtCta*>(ws + lay.ctas);
  a.met = reinterpret_cast<int*>(ws + lay.met);
  a.stats = reinterpret_cast<float2*>(ws + lay.stats);
  a.parts = reinterpret_cast<float*>(ws + lay.parts);
  a.main_ctas = std::min(d->sms, kAtMaxCtas);
  AtMaps maps;
  if (!attn_map(&maps.k, p.c, p.c.k_cache, p.c.k_page, p.c.k_slot, p.c.k_head) ||
      !attn_map(&maps.v, p.c, p.c.v_cache, p.c.v_page, p.c.v_slot, p.c.v_head))
    return SPEC_ERR_CUDA;
  // A warp of the join per row of a part, up to 8 CTAs of them.
  a.join_share = std::min(8, (lay.slot_rows + kAtJoinThreads / 32 - 1) / (kAtJoinThreads / 32));
  if (launch(paged_attention_kernel<D>, dim3((unsigned)a.main_ctas), dim3(kAtThreads), at_smem<D>(),
             s, true, maps, a) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return launch(paged_join_kernel<D>, dim3((unsigned)(a.main_ctas * a.join_share)),
                dim3(kAtJoinThreads), 0, s, true, a) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace specv

extern "C" {

spec_status_t spec_sample(const void* logits, spec_dtype_t dtype, int rows, int V, int group,
                          const float* temperature, const int32_t* top_k, const float* top_p,
                          const float* min_p, const float* uniforms, int32_t* tokens, void* kept,
                          void* stream) {
  return sample_entry("spec_sample", logits, dtype, rows, V, group, temperature, top_k, top_p, min_p,
                      uniforms, tokens, true, kept, false, stream);
}

spec_status_t spec_truncate(const void* logits, spec_dtype_t dtype, int rows, int V, int group,
                            const float* temperature, const int32_t* top_k, const float* top_p,
                            const float* min_p, void* kept, void* stream) {
  return sample_entry("spec_truncate", logits, dtype, rows, V, group, temperature, top_k, top_p,
                      min_p, nullptr, nullptr, false, kept, true, stream);
}

spec_status_t spec_kv_append(const spec_paged_cache_t* cache, spec_dtype_t dtype,
                             const void* k_new, const void* v_new, int rows, long long k_stride,
                             long long v_stride, void* stream) {
  PagedParams p = {};
  size_t nk = 0, nv = 0;
  const spec_status_t st = cache_check(cache, dtype, rows, &p.c, &nk, &nv);
  if (st != SPEC_OK) return st;
  const long long row = (long long)p.c.kv_heads * p.c.width;
  if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16)) return SPEC_ERR_INVALID_ARG;
  if (rows == 1) k_stride = v_stride = row;
  if (!row_stride_ok(k_stride, row) || !row_stride_ok(v_stride, row)) return SPEC_ERR_INVALID_ARG;
  const size_t kn = ((size_t)(rows - 1) * k_stride + row) * 2;
  const size_t vn = ((size_t)(rows - 1) * v_stride + row) * 2;
  for (const auto& o : {std::make_pair((const void*)p.c.k_cache, nk),
                        std::make_pair((const void*)p.c.v_cache, nv)})
    if (overlap(o.first, o.second, k_new, kn) || overlap(o.first, o.second, v_new, vn) ||
        meets_tables(p.c, o.first, o.second))
      return SPEC_ERR_INVALID_ARG;
  // One cache in both places.  (Interleaved ones share a range, but no entry.)
  const uintptr_t ka = reinterpret_cast<uintptr_t>(p.c.k_cache);
  const uintptr_t va = reinterpret_cast<uintptr_t>(p.c.v_cache);
  if ((ka > va ? ka - va : va - ka) < (uintptr_t)p.c.width * 2) return SPEC_ERR_INVALID_ARG;
  NvtxRange r("spec_kv_append");
  DeviceOf on_device(p.c.k_cache);
  if (!on_device.ok()) return SPEC_ERR_CUDA;
  if (!on_device.device()) return SPEC_ERR_INVALID_ARG;
  p.rows = rows;
  p.k_new = static_cast<const uint16_t*>(k_new);
  p.v_new = static_cast<const uint16_t*>(v_new);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  const long long n = (long long)rows * (row / 8);
  const long long blocks = blocks_of(n, kAppendThreads);
  if (blocks > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  return launch(kv_append_kernel, dim3((unsigned)blocks), dim3(kAppendThreads), 0,
                static_cast<cudaStream_t>(stream), true, p) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

size_t spec_paged_attention_workspace_bytes(int rows, int heads, int kv_heads, int width) {
  if (!attn_sizes_ok(rows, heads, kv_heads, width)) return 0;
  return attn_layout(rows, heads, kv_heads, width).total;
}

spec_status_t spec_paged_attention(const spec_paged_cache_t* cache, spec_dtype_t dtype,
                                   const void* q, int rows, int heads, long long q_stride,
                                   int causal, int window, float scale, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  PagedParams p = {};
  size_t nk = 0, nv = 0;
  const spec_status_t st = cache_check(cache, dtype, rows, &p.c, &nk, &nv);
  if (st != SPEC_OK) return st;
  if (heads < 1 || heads % p.c.kv_heads != 0) return SPEC_ERR_INVALID_ARG;
  if (!attn_sizes_ok(rows, heads, p.c.kv_heads, p.c.width)) return SPEC_ERR_UNSUPPORTED;
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal) ||
      !(scale > 0.0f && scale * kLog2e <= FLT_MAX))
    return SPEC_ERR_INVALID_ARG;
  const long long row = (long long)heads * p.c.width;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return SPEC_ERR_INVALID_ARG;
  if (rows == 1) q_stride = row;
  if (!row_stride_ok(q_stride, row)) return SPEC_ERR_INVALID_ARG;
  const size_t nq = ((size_t)(rows - 1) * q_stride + row) * 2, no = (size_t)rows * row * 2;
  const size_t nl = lse ? (size_t)rows * heads * 4 : 0;
  const size_t nw = attn_layout(rows, heads, p.c.kv_heads, p.c.width).total;
  for (const auto& o : {std::make_pair((const void*)out, no), std::make_pair((const void*)lse, nl)})
    if (overlap(o.first, o.second, q, nq) || overlap(o.first, o.second, p.c.k_cache, nk) ||
        overlap(o.first, o.second, p.c.v_cache, nv) || meets_tables(p.c, o.first, o.second))
      return SPEC_ERR_INVALID_ARG;
  if (overlap(out, no, lse, nl)) return SPEC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < nw) return SPEC_ERR_WORKSPACE;
  if (overlap(workspace, nw, q, nq) || overlap(workspace, nw, out, no) ||
      overlap(workspace, nw, lse, nl) || overlap(workspace, nw, p.c.k_cache, nk) ||
      overlap(workspace, nw, p.c.v_cache, nv) || meets_tables(p.c, workspace, nw))
    return SPEC_ERR_INVALID_ARG;
  NvtxRange r("spec_paged_attention");
  DeviceOf on_device(workspace);
  if (!on_device.ok()) return SPEC_ERR_CUDA;
  if (!on_device.device()) return SPEC_ERR_INVALID_ARG;
  p.rows = rows;
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.heads = heads;
  p.causal = causal;
  p.window = std::min(window, 1 << 30);  // (as good as none: see max_pages)
  p.scale = scale;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p.c.width == 64 ? attn_run<64>(p, ws, s) : attn_run<128>(p, ws, s);
}

}  // extern "C"
