// Global gradient norm over many tensors, and clipping to a largest norm.
//
//   norm  = sqrt(sum over every tensor and entry of x^2)
//   out_t = x_t * min(1, max_norm / norm)
//
// The tensors are cut into units of at most kNormUnitVecs 16-byte vectors; a
// launch takes the descriptors of up to kNormTensors tensors as kernel
// parameters (no table in memory, nothing to upload), and each CTA works on one
// run of units.  The second pass goes through a CTA's run backwards: what the
// first read last is still in L2.  A few units are done by one cluster of CTAs in one
// launch, with the sums exchanged through distributed shared memory (12 tensors of
// 20000 entries in all: 8.5 to 11 us, 11.8 as two launches).  The order of every addition is
// fixed by sizes and alignments alone, so two calls on the same tensors give the
// same bits.
//
// Range.  x^2 overflows single precision from |x| = 2^64 and vanishes below
// 2^-75, both inside the range of bfloat16 and float gradients.  A thread sums
// its share of a unit in single precision; if that sum is above 2^100 (or not
// finite) it sums the share again with x scaled by 2^-100, if it is tiny (below 2^-100,
// but some entry is not zero) with x scaled by 2^100.  So shares have room to be added:
// 2^27 of them in each kind, where a block has at most 2^23 (280 GB over 456 blocks).
// The three kinds of sums are carried apart, as float-float pairs, and joined in double
// precision at the end.
// Infinities and NaN, which a float-float pair cannot carry, go into a plain sum
// of their own: where an entry is one, the norm is, and every tensor stays as it is.  (A sum of
// finite entries whose root is above the largest float gives an infinite norm, and the
// tensors are scaled all the same.)
//
// Tensors are read by plain loads, here and in the other training kernels: the read-only
// path is for data that nobody writes while the kernel lives, and a clip in place
// writes what it has read; a kernel launched ahead of its predecessor's end also lives
// while that one still writes.
//
// Bound by memory: 0.4 G bf16 entries are summed at 85 % of the DRAM's peak and
// scaled into other tensors at 74 % (reading and writing); 0.8 G in 835 us, 60 M of 290
// tensors in 87 us.
#pragma once

#include "opd.cuh"

namespace specv {

constexpr int kNormThreads = 256;
constexpr int kNormVecsPerThread = 8;
constexpr int kNormUnitVecs = kNormThreads * kNormVecsPerThread;  // 32 KB of a tensor
constexpr int kNormTensors = 512;     // per launch
constexpr int kNormFewTensors = 32;   // per launch, where there are no more
constexpr int kNormCtasPerSm = 3;
constexpr int kNormCluster = 8;       // CTAs that do a few units in one launch
constexpr int kNormFewUnits = 2 * kNormCluster;

template <int kN>
struct NormBatch {
  const void* in[kN];
  void* out[kN];           // clip only
  long long n[kN];         // entries
  int first_unit[kN + 1];  // units before this tensor, in this launch
  unsigned char bf16[kN];
  int count;
};

// One CTA's sums: normal, scaled down (large entries), scaled up (small ones).
struct __align__(16) NormPartial {
  FF s[3];
  float bad;  // sum of what is not finite (0 when everything is)
  float pad;
};

// The scale is pre * scale: pre is 2^-100 where the scale alone would be
// subnormal (entries near the top of the range, a small largest norm) and would
// have lost bits, else 1.
struct NormResult {
  float norm;
  float pre, scale;
};

constexpr float kNormDown = 7.888609052210118e-31f;  // 2^-100
constexpr float kNormUp = 1.2676506002282294e30f;    // 2^100

// What a unit of a tensor covers: `vecs` vectors from `v`, and for the
// tensor's first unit the entries before its first and after its last vector.
// Tensors whose input and output lie differently in a 16-byte line have no
// vectors: their units are cut in entries.
struct NormUnit {
  int t;
  long long e0;   // first entry of the unit's body
  int ne;         // entries in the body (a multiple of a vector's when vec)
  int head;       // first unit: entries [0, head) as well
  long long tail0;  // first unit: entries [tail0, n) as well
  bool vec;
};

__host__ __device__ inline int norm_head(const void* p, long long n, int esize) {
  const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
  const long long h = off ? (16 - off) / esize : 0;
  return (int)(h < n ? h : n);
}

__host__ __device__ inline bool norm_vec_ok(const void* in, const void* out) {
  return out == nullptr || ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
}

// Units a tensor is cut into (at least one, so that short tensors are seen).
__host__ __device__ inline long long norm_units(const void* in, const void* out, long long n,
                                                int esize) {
  if (n <= 0) return 0;
  const int epv = 16 / esize;
  const long long body = norm_vec_ok(in, out) ? (n - norm_head(in, n, esize)) / epv * epv : n;
  const long long per = (long long)kNormUnitVecs * epv;
  const long long u = (body + per - 1) / per;
  return u < 1 ? 1 : u;
}

// The tensor with first_unit[t] <= u < first_unit[t + 1].
template <int kN>
__device__ __forceinline__ int norm_tensor(const NormBatch<kN>& b, int u) {
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first_unit[mid] <= u) lo = mid;
    else hi = mid;
  }
  return (int)SPEC_CHECKED(lo, b.count, kSiteNormUnit);
}

template <int kN>
__device__ __forceinline__ NormUnit norm_unit(const NormBatch<kN>& b, int t, int u) {
  NormUnit r;
  r.t = t;
  const int es = b.bf16[t] ? 2 : 4, epv = 16 / es;
  const long long n = b.n[t], per = (long long)kNormUnitVecs * epv;
  const int j = u - b.first_unit[t];
  r.vec = norm_vec_ok(b.in[t], b.out[t]);
  const int head = r.vec ? norm_head(b.in[t], n, es) : 0;
  const long long body = r.vec ? (n - head) / epv * epv : n;
  r.e0 = head + j * per;
  const long long left = body - j * per;
  r.ne = (int)(left < per ? (left > 0 ? left : 0) : per);
  r.head = j == 0 ? head : 0;
  r.tail0 = j == 0 ? head + body : n;
  return r;
}

// CTA c's run of units.
__device__ __forceinline__ int norm_run_start(int units, int c, int ctas) {
  return (int)((long long)units * c / ctas);
}

template <typename TIn>
__device__ __forceinline__ float sum_squares(const uint4 (&v)[kNormVecsPerThread], float k) {
  using Tr = ElemTraits<TIn>;
  float2 a[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  const float2 kk = make_float2(k, k);
#pragma unroll
  for (int i = 0; i < kNormVecsPerThread; ++i) {
    float x[Tr::kPerVec];
    Tr::unpack(v[i], x);
#pragma unroll
    for (int e = 0; e < Tr::kPerVec; e += 2) {
      float2 y = make_float2(x[e], x[e + 1]);
      if (k != 1.0f) y = f32x2_mul(y, kk);
      a[(e >> 1) & 1] = f32x2_fma(y, y, a[(e >> 1) & 1]);
    }
  }
  const float2 t = f32x2_add(a[0], a[1]);
  return __fadd_rn(t.x, t.y);
}

// Whether a share's plain sum has to be taken again, and with which scale:
// 0 keep it, 1 scale down (above 2^100, not only where it overflows itself: the shares
// are added up), 2 scale up.
__device__ __forceinline__ int norm_class(float s, bool any) {
  if (!(s <= kNormUp)) return 1;
  return (any && s < kNormDown) ? 2 : 0;
}

__device__ __forceinline__ void norm_add(NormPartial& p, int cls, float s) {
  if (!(s <= FLT_MAX)) {
    p.bad = __fadd_rn(p.bad, s);
    return;
  }
#pragma unroll
  for (int c = 0; c < 3; ++c)
    if (c == cls) p.s[c] = ff_add_f(p.s[c], s);
}

__device__ __forceinline__ NormPartial norm_zero() {
  NormPartial p;
#pragma unroll
  for (int c = 0; c < 3; ++c) p.s[c] = FF{0.0f, 0.0f};
  p.bad = p.pad = 0.0f;
  return p;
}

// The lanes' sums in every lane; the first `levels` powers of two of the lanes have some.
template <int levels = 5>
__device__ __forceinline__ void norm_warp_sum(NormPartial& p) {
  p.s[0] = group_sum_ff(p.s[0], levels);
  // Seldom: some entry was very large, very small or not finite.
  if (!__any_sync(0xffffffffu, p.s[1].hi != 0.0f || p.s[2].hi != 0.0f || p.bad != 0.0f)) return;
#pragma unroll
  for (int c = 1; c < 3; ++c) p.s[c] = group_sum_ff(p.s[c], levels);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    p.bad = __fadd_rn(p.bad, __shfl_xor_sync(0xffffffffu, p.bad, off));
}

__device__ __forceinline__ void norm_add1(NormPartial& p, float x) {
  const float s = __fmul_rn(x, x);
  const int cls = norm_class(s, x != 0.0f);
  const float k = cls == 1 ? kNormDown : cls == 2 ? kNormUp : 1.0f;
  const float y = __fmul_rn(x, k);
  norm_add(p, cls, __fmul_rn(y, y));
}

template <typename TIn, int kN>
__device__ __forceinline__ void norm_unit_sum(const NormBatch<kN>& b, const NormUnit& u,
                                              NormPartial& p) {
  using Tr = ElemTraits<TIn>;
  const TIn* x = static_cast<const TIn*>(b.in[u.t]);
  if (u.vec) {
    const uint4* xv = reinterpret_cast<const uint4*>(x + u.e0);
    const int nv = u.ne / Tr::kPerVec;
    uint4 v[kNormVecsPerThread];
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kNormVecsPerThread; ++i) {
      const int at = threadIdx.x + i * kNormThreads;
      v[i] = at < nv ? xv[at] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kNormVecsPerThread; ++i) any |= v[i].x | v[i].y | v[i].z | v[i].w;
    any &= sizeof(TIn) == 2 ? 0x7fff7fffu : 0xffffffffu;
    float s = sum_squares<TIn>(v, 1.0f);
    // A float word of only sign bits is -0: its square is 0 as well.
    const int cls = norm_class(s, any != 0);
    if (cls == 1) s = sum_squares<TIn>(v, kNormDown);
    if (cls == 2) s = sum_squares<TIn>(v, kNormUp);
    norm_add(p, cls, s);
  } else {
    for (int e = threadIdx.x; e < u.ne; e += kNormThreads) norm_add1(p, Tr::to_float(x[u.e0 + e]));
  }
  if ((int)threadIdx.x < u.head) norm_add1(p, Tr::to_float(x[threadIdx.x]));
  if (u.tail0 + threadIdx.x < b.n[u.t]) norm_add1(p, Tr::to_float(x[u.tail0 + threadIdx.x]));
}

// A CTA's sum over its run of units, in thread 0.
template <int kN>
__device__ __forceinline__ NormPartial norm_cta_sum(const NormBatch<kN>& b, int u0, int u1) {
  NormPartial p = norm_zero();
  if (u0 < u1) {
    int t = norm_tensor(b, u0);
    for (int u = u0; u < u1; ++u) {
      while (u >= b.first_unit[t + 1]) ++t;
      const NormUnit nu = norm_unit(b, t, u);
      if (b.bf16[t]) norm_unit_sum<uint16_t>(b, nu, p);
      else norm_unit_sum<float>(b, nu, p);
    }
  }
  __shared__ NormPartial warp_sum[kNormThreads / 32];
  norm_warp_sum(p);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = p;
  __syncthreads();
  if (threadIdx.x < 32) {
    p = threadIdx.x < kNormThreads / 32 ? warp_sum[threadIdx.x] : norm_zero();
    norm_warp_sum<3>(p);
  }
  return p;
}

// Sums of squares: partials[blockIdx.x].
template <int kN>
__global__ void __launch_bounds__(kNormThreads, kNormCtasPerSm)
    grad_norm_kernel(const __grid_constant__ NormBatch<kN> b, NormPartial* partials) {
  pdl_wait();
  pdl_launch_dependents();
  const int units = b.first_unit[b.count];
  const NormPartial p = norm_cta_sum(b, norm_run_start(units, blockIdx.x, gridDim.x),
                                     norm_run_start(units, blockIdx.x + 1, gridDim.x));
  if (threadIdx.x == 0) partials[blockIdx.x] = p;
}

// The norm from the CTAs' partials, the same in every thread: added in a fixed
// order, in double precision (2^200 and 2^-200 undo the scaling of the squares).
// Called by whole CTAs.
__device__ __forceinline__ NormResult norm_result(const NormPartial* partials, int n,
                                                  float max_norm) {
  __shared__ double sums[kNormThreads / 32];
  __shared__ float bads[kNormThreads / 32];
  double t = 0.0;
  float bad = 0.0f;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kNormThreads) {
    const NormPartial p = partials[i];
    t += ((double)p.s[0].hi + (double)p.s[0].lo) +
         ((double)p.s[1].hi + (double)p.s[1].lo) * 1.6069380442589903e60 +
         ((double)p.s[2].hi + (double)p.s[2].lo) * 6.223015277861142e-61;
    bad = __fadd_rn(bad, p.bad);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t += __shfl_xor_sync(0xffffffffu, t, o);
    bad = __fadd_rn(bad, __shfl_xor_sync(0xffffffffu, bad, o));
  }
  if ((threadIdx.x & 31) == 0) {
    sums[threadIdx.x >> 5] = t;
    bads[threadIdx.x >> 5] = bad;
  }
  __syncthreads();
  t = sums[0];
  bad = bads[0];
#pragma unroll
  for (int w = 1; w < kNormThreads / 32; ++w) {
    t += sums[w];
    bad = __fadd_rn(bad, bads[w]);
  }
  NormResult r;
  const double norm = sqrt(t);
  r.norm = bad == 0.0f ? (float)norm : bad;
  r.pre = r.scale = 1.0f;
  if (bad == 0.0f && norm > (double)max_norm) {
    const double scale = (double)max_norm / norm;
    const bool small = scale < 7.888609052210118e-31;
    r.pre = small ? kNormDown : 1.0f;
    r.scale = (float)(small ? scale * 1.2676506002282294e30 : scale);
  }
  return r;
}

__global__ void __launch_bounds__(kNormThreads)
    grad_norm_finish_kernel(const NormPartial* partials, int n, float* norm) {
  pdl_wait();
  const NormResult r = norm_result(partials, n, FLT_MAX);
  if (threadIdx.x == 0) *norm = r.norm;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <typename TIn>
__device__ __forceinline__ uint4 pack_vec(const float* x);
template <>
__device__ __forceinline__ uint4 pack_vec<float>(const float* x) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}
template <>
__device__ __forceinline__ uint4 pack_vec<uint16_t>(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store_elem(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_elem(uint16_t* p, float x) {
  *p = (uint16_t)pack_bf16(x, 0.0f);
}

__device__ __forceinline__ float norm_scaled(float x, const NormResult& r) {
  return __fmul_rn(__fmul_rn(x, r.pre), r.scale);
}

template <typename TIn, int kN>
__device__ __forceinline__ void clip_unit(const NormBatch<kN>& b, const NormUnit& u, const NormResult& r) {
  using Tr = ElemTraits<TIn>;
  const TIn* x = static_cast<const TIn*>(b.in[u.t]);
  TIn* y = static_cast<TIn*>(b.out[u.t]);
  if (u.vec) {
    const uint4* xv = reinterpret_cast<const uint4*>(x + u.e0);
    uint4* yv = reinterpret_cast<uint4*>(y + u.e0);
    const int nv = u.ne / Tr::kPerVec;
    uint4 v[kNormVecsPerThread];
#pragma unroll
    for (int i = 0; i < kNormVecsPerThread; ++i) {
      const int at = threadIdx.x + i * kNormThreads;
      if (at < nv) v[i] = __ldcs(xv + at);
    }
#pragma unroll
    for (int i = 0; i < kNormVecsPerThread; ++i) {
      const int at = threadIdx.x + i * kNormThreads;
      if (at >= nv) continue;
      float e[Tr::kPerVec];
      Tr::unpack(v[i], e);
#pragma unroll
      for (int j = 0; j < Tr::kPerVec; ++j) e[j] = norm_scaled(e[j], r);
      __stcs(yv + at, pack_vec<TIn>(e));
    }
  } else {
    for (int e = threadIdx.x; e < u.ne; e += kNormThreads)
      store_elem(y + u.e0 + e, norm_scaled(Tr::to_float(x[u.e0 + e]), r));
  }
  if ((int)threadIdx.x < u.head)
    store_elem(y + threadIdx.x, norm_scaled(Tr::to_float(x[threadIdx.x]), r));
  if (u.tail0 + threadIdx.x < b.n[u.t])
    store_elem(y + u.tail0 + threadIdx.x,
               norm_scaled(Tr::to_float(x[u.tail0 + threadIdx.x]), r));
}

// A CTA's run of units, scaled, backwards.
template <int kN>
__device__ __forceinline__ void clip_run(const NormBatch<kN>& b, int u0, int u1,
                                         const NormResult& r) {
  if (u0 >= u1) return;
  int t = norm_tensor(b, u1 - 1);
  for (int u = u1 - 1; u >= u0; --u) {
    while (u < b.first_unit[t]) --t;
    // In place and within the norm: the tensor is what it has to be.
    if (r.scale == 1.0f && r.pre == 1.0f && b.in[t] == b.out[t]) continue;
    const NormUnit nu = norm_unit(b, t, u);
    if (b.bf16[t]) clip_unit<uint16_t>(b, nu, r);
    else clip_unit<float>(b, nu, r);
  }
}

template <int kN>
__global__ void __launch_bounds__(kNormThreads, kNormCtasPerSm)
    clip_kernel(const __grid_constant__ NormBatch<kN> b, const NormPartial* partials, int n,
                float max_norm, float* norm) {
  pdl_wait();
  pdl_launch_dependents();
  const NormResult r = norm_result(partials, n, max_norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = r.norm;
  const int units = b.first_unit[b.count];
  clip_run(b, norm_run_start(units, blockIdx.x, gridDim.x),
           norm_run_start(units, blockIdx.x + 1, gridDim.x), r);
}

// A few units: norm and clip (or the norm alone) by one cluster.
__global__ void __cluster_dims__(kNormCluster, 1, 1) __launch_bounds__(kNormThreads)
    clip_few_kernel(const __grid_constant__ NormBatch<kNormFewTensors> b, float max_norm, bool clip,
                    float* norm) {
  __shared__ NormPartial all[kNormCluster];
  pdl_wait();
  pdl_launch_dependents();
  cluster_sync();  // every CTA runs before any writes to another's shared memory
  const int rank = (int)cluster_rank(), units = b.first_unit[b.count];
  const int u0 = norm_run_start(units, rank, kNormCluster);
  const int u1 = norm_run_start(units, rank + 1, kNormCluster);
  const NormPartial p = norm_cta_sum(b, u0, u1);
  if (threadIdx.x == 0)
    for (int c = 0; c < kNormCluster; ++c) {
      const uint32_t to = dsmem_map(&all[rank], c);
      dsmem_st4(to, make_float4(p.s[0].hi, p.s[0].lo, p.s[1].hi, p.s[1].lo));
      dsmem_st4(to + 16, make_float4(p.s[2].hi, p.s[2].lo, p.bad, 0.0f));
    }
  cluster_sync();
  const NormResult r = norm_result(all, kNormCluster, clip ? max_norm : FLT_MAX);
  if (rank == 0 && threadIdx.x == 0) *norm = r.norm;
  if (clip) clip_run(b, u0, u1, r);
}

}  // namespace specv
