// C entry points of the drafter-training operators: argument checks and launches.
#pragma once

namespace specv {

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na != 0 && nb != 0 && x < y + nb && y < x + na;
}

// ---------------------------------------------------------------------------
// Linear cross entropy.
// ---------------------------------------------------------------------------

inline bool ce_sizes_ok(int N, int V, int D) {
  return N <= kCeMaxTokens && V <= SPEC_MAX_V && D <= kCeMaxWidth && D % 8 == 0;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Tensor map of a row-major bf16 matrix [rows, cols], rows `ld` entries apart, in
// boxes of box_rows x 64 with the 128-byte swizzle.  What lies outside the matrix
// reads as 0 and is not written.
inline bool ce_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld,
                   int box_rows) {
  EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t one[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of floats [slices, rows, cols] in boxes of 1 x 32 x 32.
inline bool ce_map3(CUtensorMap* m, void* base, long long slices, long long rows, long long cols) {
  EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)slices};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 4, (cuuint64_t)(cols * rows) * 4};
  const cuuint32_t box[3] = {32, 32, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline cudaError_t ce_prepare(DeviceInfo* d) {
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (d->ce_ready) return cudaSuccess;
  cudaError_t e;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute(ce_mma_kernel<kCeLoss, true>, attr, kMmSmem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(ce_mma_kernel<kCeDz, false>, attr, kMmSmem)) != cudaSuccess)
    return e;
  if ((e = cudaFuncSetAttribute(ce_mma_kernel<kCeDz, true>, attr, kMmSmem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(ce_mma_kernel<kCeGrads, false>, attr, kMmSmem)) != cudaSuccess)
    return e;
  if ((e = cudaFuncSetAttribute(ce_mma_kernel<kCeGrads, true>, attr, kMmSmem)) != cudaSuccess)
    return e;
  // The small kernels between the products take the same split of L1, so that no SM has
  // to be idle to change it.
  for (const void* k : {(const void*)ce_finish_kernel, (const void*)ce_round_kernel,
                        (const void*)ce_label_kernel})
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout,
                                  cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
      return e;
  d->ce_ready = true;
  return cudaSuccess;
}

template <CeMode M, bool kChunks>
cudaError_t launch_ce(const DeviceInfo* d, const CeMaps& maps, CeParams& p, long long tiles,
                      cudaStream_t stream) {
  const long long pairs = std::max<long long>(1, std::min<long long>(tiles, d->sms / 2));
  if (M == kCeGrads)
    p.deal = ce_deal(p.dh_units, p.dw_units, p.split_iters, (p.N + kMmK - 1) / kMmK, (int)pairs);
  else
    p.z_tiles = (int)tiles;
  return launch(ce_mma_kernel<M, kChunks>, dim3((unsigned)(2 * pairs)), dim3(kMmThreads), kMmSmem, stream,
                true, maps, p);
}

inline CeParams ce_params(const int32_t* labels, int N, int V, int D, const CeLayout& lay,
                          unsigned char* ws) {
  CeParams p = {};
  p.labels = labels;
  p.N = N;
  p.V = V;
  p.D = D;
  p.parts = lay.parts;
  p.m_blocks = (N + kMmM - 1) / kMmM;
  p.a_rows = N < kMmHalf ? (N + 7) / 8 * 8 : kMmHalf;
  p.partials = reinterpret_cast<float2*>(ws + lay.partials);
  p.piece = lay.piece;
  p.dh_acc = reinterpret_cast<float*>(ws + lay.dh_acc);
  p.resid = reinterpret_cast<float*>(ws + lay.resid);
  p.in_rows = reinterpret_cast<uint32_t*>(ws + lay.in_rows);
  p.label_sums = reinterpret_cast<float*>(ws + lay.label_sums);
  p.header = reinterpret_cast<WsHeader*>(ws);
  return p;
}

inline long long blocks_of(long long n, int b) { return (n + b - 1) / b; }

inline spec_status_t ce_loss(const void* hidden, const void* weight, const int32_t* labels, int N,
                             int V, int D, float* nll, float* lse, unsigned char* ws,
                             cudaStream_t s) {
  NvtxRange r("spec_linear_ce");
  DeviceInfo* d = nullptr;
  if (device_info(&d) != cudaSuccess || ce_prepare(d) != cudaSuccess) return SPEC_ERR_CUDA;
  const CeLayout lay = ce_layout(N, V, D, false);
  CeParams p = ce_params(labels, N, V, D, lay, ws);
  p.h = static_cast<const uint16_t*>(hidden);
  p.w = static_cast<const uint16_t*>(weight);
  p.check = 1;
  p.group = 32;
  if (N <= kCeFewTokens) {
    while (p.group / 2 >= N) p.group /= 2;
    p.a_rows = 32;
  }
  CeMaps maps = {};
  if (!ce_map(&maps.h_k, hidden, N, D, D, p.a_rows) ||
      !ce_map(&maps.w_k, weight, V, D, D, kMmHalf))
    return SPEC_ERR_CUDA;
  if (launch_ce<kCeLoss, true>(d, maps, p, blocks_of(N, kMmM) * lay.tiles, s) != cudaSuccess)
    return SPEC_ERR_CUDA;
  // Tokens of a CTA of the join: a sector's worth of partials (4), more only where the CTAs
  // still cover the SMs, so that the labels' logits are formed by many at once (512 tokens,
  // D = 2048: 8 us with 4 a CTA, 14 with 32; 2048 tokens, D = 4096: 12 with 16, 17
  // with 32).
  int tokens = 1;
  while (tokens < 32 && tokens < N && (tokens < 4 || blocks_of(N, tokens) > d->sms)) tokens *= 2;
  if (launch(ce_finish_kernel, dim3((unsigned)blocks_of(N, tokens)), dim3(kCeFinishThreads), 0, s,
             true, p, tokens, nll, lse) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

inline spec_status_t ce_grad(const void* hidden, const void* weight, const int32_t* labels,
                             const float* nll, const float* lse, const float* grad_nll, int N,
                             int V, int D, void* d_hidden, void* d_weight, unsigned char* ws, cudaStream_t s) {
  NvtxRange r("spec_linear_ce_grad");
  DeviceInfo* d = nullptr;
  if (device_info(&d) != cudaSuccess || ce_prepare(d) != cudaSuccess) return SPEC_ERR_CUDA;
  const CeLayout lay = ce_layout(N, V, D, true);
  CeParams p = ce_params(labels, N, V, D, lay, ws);
  p.h = static_cast<const uint16_t*>(hidden);
  p.w = static_cast<const uint16_t*>(weight);
  p.nll = nll;
  p.lse = lse;
  p.g = grad_nll;
  p.splits = lay.splits;
  p.dh_direct = lay.direct;
  void* dz = ws + lay.dz;
  CeMaps maps = {};
  if (!ce_map(&maps.h_k, hidden, N, D, D, p.a_rows) ||
      !ce_map(&maps.w_k, weight, V, D, D, kMmHalf) ||
      !ce_map(&maps.h_mn, hidden, N, D, D, 64) || !ce_map(&maps.w_mn, weight, V, D, D, 64))
    return SPEC_ERR_CUDA;
  if (d_weight != nullptr && !ce_map(&maps.dw_out, d_weight, V, D, D, 32)) return SPEC_ERR_CUDA;
  if (d_hidden != nullptr && !(lay.direct ? ce_map(&maps.dh_out, d_hidden, N, D, D, 32)
                                          : ce_map3(&maps.acc, p.dh_acc, p.splits, N, D)))
    return SPEC_ERR_CUDA;
  const long long mb = blocks_of(N, kMmM), db = blocks_of(D, kMmN);
  for (int v0 = 0; v0 < V; v0 += lay.piece) {
    p.v0 = v0;
    p.nv = std::min(lay.piece, V - v0);
    p.first = v0 == 0;
    p.check = p.first;
    p.split_iters = (int)blocks_of(blocks_of(p.nv, kMmK), p.splits);
    p.dh_units = d_hidden != nullptr ? (int)(mb * db * p.splits) : 0;
    p.dw_units = d_weight != nullptr ? (int)(blocks_of(p.nv, kMmM) * db) : 0;
    // dZ's own extent: what its last tile has past the vocabulary is not written,
    // and reads as 0.
    if (!ce_map(&maps.dz_k, dz, N, p.nv, lay.piece, p.a_rows) ||
        !ce_map(&maps.dz_mn, dz, N, p.nv, lay.piece, 64) ||
        !ce_map(&maps.dz_out, dz, N, p.nv, lay.piece, 32))
      return SPEC_ERR_CUDA;
    const long long z_tiles = mb * blocks_of(p.nv, kMmN);
    if ((D > kMmChunk * kMmK ? launch_ce<kCeDz, true>(d, maps, p, z_tiles, s)
                             : launch_ce<kCeDz, false>(d, maps, p, z_tiles, s)) != cudaSuccess)
      return SPEC_ERR_CUDA;
    p.check = 0;  // the header is written once a call, or a timeout in dZ would be lost
    // Once, beside the first piece's dZ; only labels of more tokens than kCeFixes need it.
    if (p.first && d_weight != nullptr && N > kCeFixes &&
        launch(ce_label_kernel,
               dim3((unsigned)blocks_of(N, kCeLabelThreads / 32), (unsigned)blocks_of(D, kCeLabelCols)),
               dim3(kCeLabelThreads), 0, s, true, p) != cudaSuccess)
      return SPEC_ERR_CUDA;
    const long long units = (long long)p.dh_units + p.dw_units;
    const bool chunks = (p.dh_units > 0 && p.split_iters > kMmGradChunk) ||
                        (p.dw_units > 0 && N > kMmGradChunk * kMmK);
    if ((chunks ? launch_ce<kCeGrads, true>(d, maps, p, units, s)
                : launch_ce<kCeGrads, false>(d, maps, p, units, s)) != cudaSuccess)
      return SPEC_ERR_CUDA;
  }
  if (d_hidden != nullptr && !lay.direct) {
    const long long n = (long long)N * D;
    if (launch(ce_round_kernel, dim3((unsigned)blocks_of(n, 256)), dim3(256), 0, s, true, p, static_cast<uint16_t*>(d_hidden)) != cudaSuccess)
      return SPEC_ERR_CUDA;
  }
  return SPEC_OK;
}

// ---------------------------------------------------------------------------
// Mixture-loss gradient.
// ---------------------------------------------------------------------------

// CTAs per position.  Rows go through shared memory where eight CTAs or fewer can
// share them at kOgSliceBytes each, so that three fit an SM (a CTA's own
// variables and what the system keeps are in the difference to a third of 228 KB).
// Longer ones are read from memory in every pass, one CTA per 4096 entries up to eight
// (measured, before the passes over shared memory came to 313 us: 128 requests of up to 16
// rows of 151936 bf16 336 us, 453 us without; 32 requests in float, which would leave one
// CTA per SM, 241 and 193 us; 60 requests of 32000 bf16 41 and 58 us).
constexpr int kOgSliceBytes = 76000;

inline size_t opd_grad_slice(int V, int cs, size_t es) {
  const long long wins = V / 8;  // at most: the entries before the first window are less
  return (size_t)((wins + cs - 1) / cs) * 8 * es * 2 + 16;
}

inline cudaError_t opd_grad_prepare(DeviceInfo* d) {
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (d->opd_grad_ready) return cudaSuccess;
  for (const void* k : {(const void*)opd_grad_smem_kernel<float>,
                        (const void*)opd_grad_smem_kernel<uint16_t>}) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kOgSliceBytes);
    if (e != cudaSuccess) return e;
  }
  d->opd_grad_ready = true;
  return cudaSuccess;
}

template <typename TIn>
spec_status_t opd_grad_typed(OpdGradParams p, cudaStream_t stream) {
  NvtxRange r("spec_opd_grad");
  DeviceInfo* d = nullptr;
  if (device_info(&d) != cudaSuccess || opd_grad_prepare(d) != cudaSuccess) return SPEC_ERR_CUDA;
  int cs = 1;
  while (cs < kOgMaxCluster && opd_grad_slice(p.V, cs, sizeof(TIn)) > kOgSliceBytes) cs *= 2;
  const size_t bytes = opd_grad_slice(p.V, cs, sizeof(TIn));
  const bool smem = p.draft_vec && p.target_vec && bytes <= kOgSliceBytes;
  if (!smem) {
    cs = 1;
    while (cs < kOgMaxCluster && (long long)cs * 4096 < p.V) cs *= 2;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.B * p.k * cs));
  cfg.blockDim = dim3(kOgThreads);
  cfg.dynamicSmemBytes = smem ? bytes : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = smem ? cudaLaunchKernelEx(&cfg, opd_grad_smem_kernel<TIn>, p)
                             : cudaLaunchKernelEx(&cfg, opd_grad_kernel<TIn>, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Gradient norm and clipping.
// ---------------------------------------------------------------------------

constexpr int kNormMaxTensors = 1 << 20;
constexpr int kNormMaxCtas = 1024;  // partials a launch may leave, whatever the device

inline size_t grad_norm_ws(int count) {
  const size_t launches = ((size_t)count + kNormTensors - 1) / kNormTensors;
  return align256(launches * kNormMaxCtas * sizeof(NormPartial));
}

// Tensors from t on that are not empty, up to a launch's number: their descriptors.
// Returns how many units they have.
template <int kN>
int norm_fill(NormBatch<kN>& batch, const void* const* grads, void* const* outs,
              const long long* sizes, const int* dtypes, int count, bool clip, int& t) {
  batch.count = 0;
  int units = 0;
  batch.first_unit[0] = 0;
  for (; t < count && batch.count < kN; ++t) {
    if (sizes[t] == 0) continue;
    const int c = batch.count;
    const int es = dtypes[t] == SPEC_BF16 ? 2 : 4;
    void* out = clip ? (outs != nullptr ? outs[t] : const_cast<void*>(grads[t])) : nullptr;
    batch.in[c] = grads[t];
    batch.out[c] = out;
    batch.n[c] = sizes[t];
    batch.bf16[c] = es == 2;
    units += (int)norm_units(grads[t], out, sizes[t], es);
    batch.first_unit[++batch.count] = units;
  }
  return units;
}

template <int kN>
spec_status_t norm_launches(const void* const* grads, void* const* outs, const long long* sizes,
                            const int* dtypes, int count, float max_norm, float* norm,
                            NormPartial* partials, cudaStream_t s, bool clip, int most) {
  NormBatch<kN> batch;
  int parts = 0;
  for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
    int t = 0;
    do {  // (the norm of nothing is 0)
      const int units = norm_fill(batch, grads, outs, sizes, dtypes, count, clip, t);
      const int grid = std::max(1, std::min(units, most));
      if (pass == 0) {
        if (launch(grad_norm_kernel<kN>, dim3(grid), dim3(kNormThreads), 0, s, true, batch,
                   partials + parts) != cudaSuccess)
          return SPEC_ERR_CUDA;
        parts += grid;
      } else if (launch(clip_kernel<kN>, dim3(grid), dim3(kNormThreads), 0, s, true, batch,
                        (const NormPartial*)partials, parts, max_norm, norm) != cudaSuccess) {
        return SPEC_ERR_CUDA;
      }
    } while (t < count);
  }
  if (!clip && launch(grad_norm_finish_kernel, dim3(1), dim3(kNormThreads), 0, s, true,
                      (const NormPartial*)partials, parts, norm) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

inline spec_status_t norm_run(const void* const* grads, void* const* outs, const long long* sizes,
                              const int* dtypes, int count, long long units, float max_norm,
                              float* norm, void* workspace, cudaStream_t s, bool clip) {
  NvtxRange r(clip ? "spec_clip_grad_norm" : "spec_grad_norm");
  DeviceInfo* d = nullptr;
  if (device_info(&d) != cudaSuccess) return SPEC_ERR_CUDA;
  NormPartial* partials = static_cast<NormPartial*>(workspace);
  const int most = std::min(kNormMaxCtas, d->sms * kNormCtasPerSm);
  if (count <= kNormFewTensors && units <= kNormFewUnits) {
    NormBatch<kNormFewTensors> batch;
    int t = 0;
    norm_fill(batch, grads, outs, sizes, dtypes, count, clip, t);
    return launch(clip_few_kernel, dim3(kNormCluster), dim3(kNormThreads), 0, s, true, batch,
                  max_norm, clip, norm) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
  }
  if (count <= kNormFewTensors)
    return norm_launches<kNormFewTensors>(grads, outs, sizes, dtypes, count, max_norm, norm,
                                          partials, s, clip, most);
  return norm_launches<kNormTensors>(grads, outs, sizes, dtypes, count, max_norm, norm, partials, s,
                                     clip, most);
}

// The byte ranges of a clip's tensors: no output may share a byte with another
// tensor's input or output (its own input, exactly, is the in-place form).
inline bool norm_ranges_ok(const void* const* grads, void* const* outs, const long long* sizes,
                           const int* dtypes, int count) {
  struct Range {
    uintptr_t a, b;
    int t;
    bool out;
  };
  std::vector<Range> rs;
  rs.reserve(2 * (size_t)count);
  for (int t = 0; t < count; ++t) {
    if (sizes[t] == 0) continue;
    const size_t bytes = (size_t)sizes[t] * (dtypes[t] == SPEC_BF16 ? 2 : 4);
    const uintptr_t a = reinterpret_cast<uintptr_t>(grads[t]);
    const uintptr_t o = outs != nullptr ? reinterpret_cast<uintptr_t>(outs[t]) : a;
    rs.push_back({o, o + bytes, t, true});
    if (o != a) rs.push_back({a, a + bytes, t, false});
  }
  std::sort(rs.begin(), rs.end(), [](const Range& x, const Range& y) { return x.a < y.a; });
  // Inputs may share bytes among themselves; an output with nothing.
  uintptr_t end_any = 0, end_out = 0;
  for (const Range& r : rs) {
    if (r.a < (r.out ? end_any : end_out)) return false;
    end_any = std::max(end_any, r.b);
    if (r.out) end_out = std::max(end_out, r.b);
  }
  return true;
}

inline spec_status_t norm_entry(const void* const* grads, void* const* outs,
                                const long long* sizes, const int* dtypes, int count,
                                float max_norm, float* norm, void* workspace,
                                size_t workspace_bytes, void* stream, bool clip) {
  if (count < 1 || !grads || !sizes || !dtypes || !norm || !aligned(norm, 4))
    return SPEC_ERR_INVALID_ARG;
  if (count > kNormMaxTensors) return SPEC_ERR_UNSUPPORTED;
  if (clip && !(max_norm > 0.0f && max_norm <= FLT_MAX)) return SPEC_ERR_INVALID_ARG;
  long long units = 0;
  for (int t = 0; t < count; ++t) {
    if (dtypes[t] != SPEC_F32 && dtypes[t] != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
    if (sizes[t] < 0) return SPEC_ERR_INVALID_ARG;
    if (sizes[t] > (1LL << 40)) return SPEC_ERR_UNSUPPORTED;
    const size_t es = dtypes[t] == SPEC_F32 ? 4 : 2;
    if (sizes[t] > 0 && (!grads[t] || !aligned(grads[t], es))) return SPEC_ERR_INVALID_ARG;
    if (sizes[t] > 0 && outs != nullptr && (!outs[t] || !aligned(outs[t], es)))
      return SPEC_ERR_INVALID_ARG;
    units += norm_units(grads[t], outs != nullptr ? outs[t] : nullptr, sizes[t], (int)es);
    if (sizes[t] > 0 && overlap(norm, 4, grads[t], (size_t)sizes[t] * es))
      return SPEC_ERR_INVALID_ARG;
    if (sizes[t] > 0 && outs != nullptr && overlap(norm, 4, outs[t], (size_t)sizes[t] * es))
      return SPEC_ERR_INVALID_ARG;
  }
  if (units > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  try {  // the check sorts ranges in host memory it allocates
    if (clip && !norm_ranges_ok(grads, outs, sizes, dtypes, count)) return SPEC_ERR_INVALID_ARG;
  } catch (...) {
    return SPEC_ERR_INTERNAL;
  }
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < grad_norm_ws(count))
    return SPEC_ERR_WORKSPACE;
  DeviceOf on_device(norm);
  if (!on_device.ok()) return SPEC_ERR_CUDA;
  return norm_run(grads, outs, sizes, dtypes, count, units, max_norm, norm, workspace,
                  static_cast<cudaStream_t>(stream), clip);
}

}  // namespace specv

extern "C" {

size_t spec_linear_ce_workspace_bytes(int N, int V, int D) {
  if (N < 1 || V < 1 || D < 1 || !ce_sizes_ok(N, V, D)) return 0;
  return ce_layout(N, V, D, false).total;
}

size_t spec_linear_ce_grad_workspace_bytes(int N, int V, int D) {
  if (N < 1 || V < 1 || D < 1 || !ce_sizes_ok(N, V, D)) return 0;
  return ce_layout(N, V, D, true).total;
}

spec_status_t spec_linear_ce(const void* hidden, const void* weight, spec_dtype_t dtype,
                             const int32_t* labels, int N, int V, int D, float* nll, float* lse,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (N < 1 || V < 1 || D < 1) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_BF16 || !ce_sizes_ok(N, V, D)) return SPEC_ERR_UNSUPPORTED;
  if (!hidden || !weight || !labels || !nll || !lse) return SPEC_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(labels, 4) || !aligned(nll, 4) ||
      !aligned(lse, 4))
    return SPEC_ERR_INVALID_ARG;
  const size_t n4 = (size_t)N * 4, nh = (size_t)N * D * 2, nw = (size_t)V * D * 2;
  for (const void* o : {(const void*)nll, (const void*)lse})
    if (overlap(o, n4, hidden, nh) || overlap(o, n4, weight, nw) || overlap(o, n4, labels, n4))
      return SPEC_ERR_INVALID_ARG;
  if (overlap(nll, n4, lse, n4)) return SPEC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < spec_linear_ce_workspace_bytes(N, V, D))
    return SPEC_ERR_WORKSPACE;
  DeviceOf on_device(weight);
  if (!on_device.ok()) return SPEC_ERR_CUDA;
  return ce_loss(hidden, weight, labels, N, V, D, nll, lse, static_cast<unsigned char*>(workspace),
                 static_cast<cudaStream_t>(stream));
}

spec_status_t spec_linear_ce_grad(const void* hidden, const void* weight, spec_dtype_t dtype,
                                  const int32_t* labels, const float* nll, const float* lse,
                                  const float* grad_nll, int N, int V, int D, void* d_hidden,
                                  void* d_weight,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (N < 1 || V < 1 || D < 1) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_BF16 || !ce_sizes_ok(N, V, D)) return SPEC_ERR_UNSUPPORTED;
  if (!hidden || !weight || !labels || !nll || !lse || !grad_nll || (!d_hidden && !d_weight))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(labels, 4) || !aligned(nll, 4) ||
      !aligned(lse, 4) || !aligned(grad_nll, 4) || !aligned(d_hidden, 16) || !aligned(d_weight, 16))
    return SPEC_ERR_INVALID_ARG;
  const size_t n4 = (size_t)N * 4, nh = (size_t)N * D * 2, nw = (size_t)V * D * 2;
  const void* outs[2] = {d_hidden, d_weight};
  const size_t out_bytes[2] = {d_hidden ? nh : 0, d_weight ? nw : 0};
  for (int o = 0; o < 2; ++o)
    if (overlap(outs[o], out_bytes[o], hidden, nh) || overlap(outs[o], out_bytes[o], weight, nw) ||
        overlap(outs[o], out_bytes[o], labels, n4) || overlap(outs[o], out_bytes[o], lse, n4) ||
        overlap(outs[o], out_bytes[o], nll, n4) ||
        overlap(outs[o], out_bytes[o], grad_nll, n4))
      return SPEC_ERR_INVALID_ARG;
  if (overlap(d_hidden, out_bytes[0], d_weight, out_bytes[1])) return SPEC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < spec_linear_ce_grad_workspace_bytes(N, V, D))
    return SPEC_ERR_WORKSPACE;
  DeviceOf on_device(weight);
  if (!on_device.ok()) return SPEC_ERR_CUDA;
  return ce_grad(hidden, weight, labels, nll, lse, grad_nll, N, V, D, d_hidden, d_weight,
                 static_cast<unsigned char*>(workspace), static_cast<cudaStream_t>(stream));
}

spec_status_t spec_opd_grad(const void* target_logits, const void* draft_logits,
                            spec_dtype_t dtype, const int32_t* lengths, const float* grad_loss,
                            int B, int k, int V, float delta, float alpha, void* d_draft,
                            void* stream) {
  if (B < 1 || k < 1 || V < 1) return SPEC_ERR_INVALID_ARG;
  if (!sizes_ok(B, k, V)) return SPEC_ERR_UNSUPPORTED;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (!(delta > 0.0f && delta <= FLT_MAX) || !(alpha >= 0.0f && alpha <= 1.0f))
    return SPEC_ERR_INVALID_ARG;
  if (!target_logits || !draft_logits || !lengths || !grad_loss || !d_draft)
    return SPEC_ERR_INVALID_ARG;
  const size_t es = dtype == SPEC_F32 ? 4 : 2;
  if (!aligned(target_logits, es) || !aligned(draft_logits, es) || !aligned(lengths, 4) ||
      !aligned(grad_loss, 4) || !aligned(d_draft, es))
    return SPEC_ERR_INVALID_ARG;
  const size_t nd = (size_t)B * k * V * es, nt = (size_t)B * (k + 1) * V * es;
  if (overlap(d_draft, nd, draft_logits, nd) || overlap(d_draft, nd, target_logits, nt) ||
      overlap(d_draft, nd, lengths, (size_t)B * 4) || overlap(d_draft, nd, grad_loss, (size_t)B * 4))
    return SPEC_ERR_INVALID_ARG;
  {
    bool direct = false;
    const void* t = target_logits;
    const void* d = draft_logits;
    if (!resolve_logits(&t, &d, &direct) || direct) return SPEC_ERR_INVALID_ARG;
  }
  DeviceOf on_device(target_logits);
  if (!on_device.ok()) return SPEC_ERR_CUDA;
  OpdGradParams p = {};
  p.target = target_logits;
  p.draft = draft_logits;
  p.lengths = lengths;
  p.grad_loss = grad_loss;
  p.out = d_draft;
  p.B = B;
  p.k = k;
  p.V = V;
  p.draft_vec = aligned(draft_logits, 16) && aligned(d_draft, 16);
  p.target_vec = aligned(target_logits, 16);
  p.delta = delta;
  p.alpha = alpha;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == SPEC_F32 ? opd_grad_typed<float>(p, s) : opd_grad_typed<uint16_t>(p, s);
}

size_t spec_grad_norm_workspace_bytes(int count) {
  if (count < 1 || count > kNormMaxTensors) return 0;
  return grad_norm_ws(count);
}

spec_status_t spec_grad_norm(const void* const* grads, const long long* sizes, const int* dtypes,
                             int count, float* norm, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return norm_entry(grads, nullptr, sizes, dtypes, count, 0.0f, norm, workspace, workspace_bytes,
                    stream, false);
}

spec_status_t spec_clip_grad_norm(const void* const* grads, void* const* outs,
                                  const long long* sizes, const int* dtypes, int count,
                                  float max_norm, float* norm, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return norm_entry(grads, outs, sizes, dtypes, count, max_norm, norm, workspace, workspace_bytes,
                    stream, true);
}

}  // extern "C"
