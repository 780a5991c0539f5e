// Global gradient norm over many tensors, and clipping to a largest norm.
//
//   norm  = sqrt(sum over every tensor and entry of x^2)
//   out_t = x_t * min(1, max_norm / norm)
//
// The tensors are cut into units of at most kNormUnitVecs 16-byte vectors; a
// launch takes the descriptors of up to kNormTensors tensors as kernel
// parameters (no table in memory, nothing to upload), and CTA c works on units
// c, c + grid, ...  The order of every addition is fixed by the sizes alone, so
// two calls on the same tensors give the same bits.
//
// Range.  x^2 overflows single precision from |x| = 2^64 and vanishes below
// 2^-75, both inside the range of bfloat16 and float gradients.  A thread sums
// its share of a unit in single precision; if that sum is not finite it sums
// the share again with x scaled by 2^-100, if it is tiny (below 2^-100, but
// some entry is not zero) with x scaled by 2^100.  The three kinds of sums are
// carried apart, as float-float pairs, and joined in double precision at the end.
// Infinities and NaN, which a float-float pair cannot carry, go into a plain sum
// of their own; a norm that is not finite leaves every tensor as it is.
#pragma once

#include "common.cuh"

namespace specv {

constexpr int kNormThreads = 256;
constexpr int kNormVecsPerThread = 8;
constexpr int kNormUnitVecs = kNormThreads * kNormVecsPerThread;  // 32 KB of a tensor
constexpr int kNormTensors = 512;                                 // per launch
constexpr int kNormCtasPerSm = 4;

struct NormBatch {
  const void* in[kNormTensors];
  void* out[kNormTensors];           // clip only
  long long n[kNormTensors];         // entries
  int first_unit[kNormTensors + 1];  // units before this tensor, in this launch
  unsigned char bf16[kNormTensors];
  int count;
};

// One CTA's sums: normal, scaled down (large entries), scaled up (small ones).
struct NormPartial {
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

__device__ __forceinline__ NormUnit norm_unit(const NormBatch& b, int u) {
  int lo = 0, hi = b.count;  // the tensor with first_unit[t] <= u < first_unit[t + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.first_unit[mid] <= u) lo = mid;
    else hi = mid;
  }
  NormUnit r;
  r.t = lo;
  const int es = b.bf16[lo] ? 2 : 4, epv = 16 / es;
  const long long n = b.n[lo], per = (long long)kNormUnitVecs * epv;
  const int j = u - b.first_unit[lo];
  r.vec = norm_vec_ok(b.in[lo], b.out[lo]);
  const int head = r.vec ? norm_head(b.in[lo], n, es) : 0;
  const long long body = r.vec ? (n - head) / epv * epv : n;
  r.e0 = head + j * per;
  const long long left = body - j * per;
  r.ne = (int)(left < per ? (left > 0 ? left : 0) : per);
  r.head = j == 0 ? head : 0;
  r.tail0 = j == 0 ? head + body : n;
  return r;
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
// 0 keep it, 1 scale down, 2 scale up.
__device__ __forceinline__ int norm_class(float s, bool any) {
  if (!(s <= FLT_MAX)) return 1;
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

__device__ __forceinline__ void norm_merge(NormPartial& p, const NormPartial& q) {
#pragma unroll
  for (int c = 0; c < 3; ++c) p.s[c] = ff_add(p.s[c], q.s[c]);
  p.bad = __fadd_rn(p.bad, q.bad);
}

__device__ __forceinline__ NormPartial norm_zero() {
  NormPartial p;
#pragma unroll
  for (int c = 0; c < 3; ++c) p.s[c] = FF{0.0f, 0.0f};
  p.bad = p.pad = 0.0f;
  return p;
}

__device__ __forceinline__ void norm_warp_sum(NormPartial& p) {
#pragma unroll
  for (int c = 0; c < 3; ++c) p.s[c] = warp_sum_ff(p.s[c]);
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

template <typename TIn>
__device__ __forceinline__ void norm_unit_sum(const NormBatch& b, const NormUnit& u,
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
      v[i] = at < nv ? __ldg(xv + at) : make_uint4(0, 0, 0, 0);
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
    for (int e = threadIdx.x; e < u.ne; e += kNormThreads) norm_add1(p, Tr::load(x, u.e0 + e));
  }
  if ((int)threadIdx.x < u.head) norm_add1(p, Tr::load(x, threadIdx.x));
  if (u.tail0 + threadIdx.x < b.n[u.t]) norm_add1(p, Tr::load(x, u.tail0 + threadIdx.x));
}

// Sums of squares: partials[blockIdx.x].
__global__ void __launch_bounds__(kNormThreads)
    grad_norm_kernel(const __grid_constant__ NormBatch b, NormPartial* partials) {
  pdl_wait();
  pdl_launch_dependents();
  NormPartial p = norm_zero();
  const int units = b.first_unit[b.count];
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const NormUnit nu = norm_unit(b, u);
    if (b.bf16[nu.t]) norm_unit_sum<uint16_t>(b, nu, p);
    else norm_unit_sum<float>(b, nu, p);
  }
  __shared__ NormPartial warp_sum[kNormThreads / 32];
  norm_warp_sum(p);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = p;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kNormThreads / 32; ++w) norm_merge(p, warp_sum[w]);
    partials[blockIdx.x] = p;
  }
}

// The norm from the CTAs' partials, the same in every thread that asks: warp 0
// adds them in a fixed order.  Called by whole CTAs.
__device__ __forceinline__ NormResult norm_result(const NormPartial* partials, int n,
                                                  float max_norm) {
  __shared__ NormResult r;
  if (threadIdx.x < 32) {
    NormPartial p = norm_zero();
    for (int i = threadIdx.x; i < n; i += 32) norm_merge(p, partials[i]);
    norm_warp_sum(p);
    if (threadIdx.x == 0) {
      // 2^200 and 2^-200 undo the scaling of the squares.
      const double t = ((double)p.s[0].hi + (double)p.s[0].lo) +
                       ((double)p.s[1].hi + (double)p.s[1].lo) * 1.6069380442589903e60 +
                       ((double)p.s[2].hi + (double)p.s[2].lo) * 6.223015277861142e-61;
      const double norm = sqrt(t);
      r.norm = p.bad == 0.0f ? (float)norm : p.bad;
      const bool clip = p.bad == 0.0f && norm > (double)max_norm;
      const double scale = clip ? (double)max_norm / norm : 1.0;
      const bool small = scale < 7.888609052210118e-31;
      r.pre = small ? kNormDown : 1.0f;
      r.scale = (float)(small ? scale * 1.2676506002282294e30 : scale);
    }
  }
  __syncthreads();
  return r;
}

__global__ void grad_norm_finish_kernel(const NormPartial* partials, int n, float* norm) {
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

template <typename TIn>
__device__ __forceinline__ void clip_unit(const NormBatch& b, const NormUnit& u, const NormResult& r) {
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
      if (at < nv) v[i] = xv[at];
    }
#pragma unroll
    for (int i = 0; i < kNormVecsPerThread; ++i) {
      const int at = threadIdx.x + i * kNormThreads;
      if (at >= nv) continue;
      float e[Tr::kPerVec];
      Tr::unpack(v[i], e);
#pragma unroll
      for (int j = 0; j < Tr::kPerVec; ++j) e[j] = norm_scaled(e[j], r);
      yv[at] = pack_vec<TIn>(e);
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

__global__ void __launch_bounds__(kNormThreads)
    clip_kernel(const __grid_constant__ NormBatch b, const NormPartial* partials, int n,
                float max_norm, float* norm) {
  pdl_wait();
  const NormResult r = norm_result(partials, n, max_norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = r.norm;
  const int units = b.first_unit[b.count];
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const NormUnit nu = norm_unit(b, u);
    // In place and within the norm: the tensor is what it has to be.
    if (r.scale == 1.0f && b.in[nu.t] == b.out[nu.t]) continue;
    if (b.bf16[nu.t]) clip_unit<uint16_t>(b, nu, r);
    else clip_unit<float>(b, nu, r);
  }
}

}  // namespace specv
