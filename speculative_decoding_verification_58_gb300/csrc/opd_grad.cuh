// Gradient of the mixture distillation loss (AdaFlash Section 3.1) with
// respect to the draft logits.
//
// For a verified position i < L_b, with p and q the softmax of the target and
// draft rows (temperature 1), t_v = log q_v - log p_v, f_v = q_v t_v and x* the
// target's argmax, the loss of spec_opd_stats is
//   alpha (-log q_{x*}) + (1 - alpha) sum_v min{f_v, delta},
// averaged over the L_b positions.  An entry with f_v >= delta adds a constant,
// any other one q_v log(q_v / p_v); with u_v = t_v + 1 where f_v < delta and 0
// elsewhere, and d q_v / d z_j = q_v ([v = j] - q_j),
//   d loss / d z_j = (1 / L_b) [ alpha (q_j - [j = x*])
//                              + (1 - alpha) q_j (u_j - sum_v q_v u_v) ].
//
// Three passes over a row pair: the softmax normalisers and the argmax, the sum
// over q u, the gradient.  A cluster of CTAs owns one position, each CTA one
// part of the vocabulary; partials are exchanged through distributed shared
// memory, and the second and third pass find the rows in L2.
#pragma once

#include "grad_norm.cuh"
#include "opd.cuh"

namespace specv {

constexpr int kOgThreads = 256;
constexpr int kOgMaxCluster = 8;

struct OpdGradParams {
  const void* target;      // [B, k+1, V]
  const void* draft;       // [B, k, V]
  const int32_t* lengths;  // [B]
  const float* grad_loss;  // [B]
  void* out;               // [B, k, V]
  int B, k, V;
  int slice;   // entries of a row per CTA of a cluster (a multiple of 8)
  int vec_ok;  // rows 16-byte aligned
  float delta, alpha;
};

// Softmax partial: s = sum 2^((z - m) log2 e).  The maximum is taken off before
// the scaling (unlike the row sweep's single fused step), so that a row at the
// lowest value of its type, whose product with log2 e overflows, is still the
// uniform distribution it stands for.
struct OgAcc {
  float m, s;
};

__device__ __forceinline__ float og_exp(float z, float m) {
  return ex2(__fmul_rn(__fsub_rn(z, m), kLog2e));
}

__device__ __forceinline__ void og_add8(OgAcc& a, const float* x) {
  float gm = x[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) gm = fmaxf(gm, x[e]);
  if (gm > a.m) {
    a.s = __fmul_rn(a.s, og_exp(a.m, gm));
    a.m = gm;
  }
  float t = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) t = __fadd_rn(t, og_exp(x[e], a.m));
  a.s = __fadd_rn(a.s, t);
}

__device__ __forceinline__ void og_merge(OgAcc& a, const OgAcc& b) {
  const float m = fmaxf(a.m, b.m);
  a.s = __fadd_rn(__fmul_rn(a.s, og_exp(a.m, m)), __fmul_rn(b.s, og_exp(b.m, m)));
  a.m = m;
}

__device__ __forceinline__ void og_warp_reduce(OgAcc& a) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    og_merge(a, OgAcc{__shfl_xor_sync(0xffffffffu, a.m, off), __shfl_xor_sync(0xffffffffu, a.s, off)});
}

struct OgSoft {
  OgAcc t, d;
  float argv;
  int argi;
  float pad[2];
};

struct OgSmem {
  OgSoft warp[kOgThreads / 32];
  OgSoft part[kOgMaxCluster];
  float2 warp_c[kOgThreads / 32];
  float2 part_c[kOgMaxCluster];
};

// Eight entries from e of a row, as floats; entries past the part's end are -inf.
template <typename TIn>
__device__ __forceinline__ void og_load(const TIn* row, int e, int n, bool vec, float* x) {
  using Tr = ElemTraits<TIn>;
  if (vec && e + 8 <= n) {
#pragma unroll
    for (int j = 0; j < 8; j += Tr::kPerVec)
      Tr::unpack(__ldg(reinterpret_cast<const uint4*>(row + e + j)), x + j);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = e + j < n ? Tr::load(row, e + j) : -INFINITY;
  }
}

template <typename TIn>
__device__ __forceinline__ void og_store(TIn* row, int e, int n, bool vec, const float* x) {
  using Tr = ElemTraits<TIn>;
  if (vec && e + 8 <= n) {
#pragma unroll
    for (int j = 0; j < 8; j += Tr::kPerVec)
      *reinterpret_cast<uint4*>(row + e + j) = pack_vec<TIn>(x + j);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + j < n) store_elem(row + e + j, x[j]);
  }
}

template <typename TIn>
__device__ __forceinline__ void og_fill(TIn* row, int n, bool vec, float v) {
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = v;
  for (int e = threadIdx.x * 8; e < n; e += kOgThreads * 8) og_store<TIn>(row, e, n, vec, x);
}

__device__ __forceinline__ void og_merge(OgSoft& a, const OgSoft& b) {
  og_merge(a.t, b.t);
  og_merge(a.d, b.d);
  ArgAcc g = {a.argv, a.argi};
  arg_merge(g, ArgAcc{b.argv, b.argi});
  a.argv = g.v;
  a.argi = g.i;
}

// u of one entry: t + 1 below the clip, 0 above it.  Infinite logits need no
// case of their own: z_d = -inf gives q = 0 and q t = NaN, z_t = -inf gives
// t = +inf (q t = +inf, or NaN where q vanished), and the comparison is false
// for all of them.
__device__ __forceinline__ float og_u(float q, float t, float delta) {
  return __fmul_rn(q, t) < delta ? __fadd_rn(t, 1.0f) : 0.0f;
}

template <typename TIn>
__global__ void __launch_bounds__(kOgThreads) opd_grad_kernel(OpdGradParams p) {
  __shared__ OgSmem sm;
  const uint32_t rank = cluster_rank(), cs = cluster_size();
  const long long pos = blockIdx.x / cs;  // one cluster per position
  const int b = (int)(pos / p.k), i = (int)(pos - (long long)b * p.k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s0 = (int)rank * p.slice;
  const int n = max(0, min(p.slice, p.V - s0));
  const long long row = SPEC_CHECKED(pos, (long long)p.B * p.k, kSiteOpdGradRow);
  TIn* out = static_cast<TIn*>(p.out) + (size_t)row * p.V + s0;
  const bool vec = p.vec_ok != 0;
  const int L = __ldg(&p.lengths[b]);
  // The same decision in every CTA of the cluster: none is left at a barrier.
  if (L < 1 || L > p.k || i >= L) {
    og_fill<TIn>(out, n, vec, (L < 1 || L > p.k) ? __int_as_float(0x7fc00000) : 0.0f);
    return;
  }
  cluster_sync();  // every CTA runs before any writes to another's shared memory
  const TIn* zt = static_cast<const TIn*>(p.target) + ((size_t)b * (p.k + 1) + i) * (size_t)p.V + s0;
  const TIn* zd = static_cast<const TIn*>(p.draft) + (size_t)row * p.V + s0;

  // Pass 1: normalisers of both rows, argmax of the target.
  OgAcc at = {-FLT_MAX, 0.0f}, ad = at;
  ArgAcc ag;
  arg_init(ag);
  for (int e = threadIdx.x * 8; e < n; e += kOgThreads * 8) {
    float a[8], d[8];
    og_load<TIn>(zt, e, n, vec, a);
    og_load<TIn>(zd, e, n, vec, d);
    og_add8(at, a);
    og_add8(ad, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) arg_add(ag, a[j], s0 + e + j);
  }
  og_warp_reduce(at);
  og_warp_reduce(ad);
  arg_warp_reduce(ag);
  if (lane == 0) sm.warp[warp] = OgSoft{at, ad, ag.v, ag.i};
  __syncthreads();
  if (threadIdx.x < cs) {  // every CTA sends its sum to all, itself included
    OgSoft s = sm.warp[0];
    for (int w = 1; w < kOgThreads / 32; ++w) og_merge(s, sm.warp[w]);
    const uint32_t to = dsmem_map(&sm.part[rank], threadIdx.x);
    dsmem_st4(to, make_float4(s.t.m, s.t.s, s.d.m, s.d.s));
    dsmem_st4(to + 16, make_float4(s.argv, __int_as_float(s.argi), 0.0f, 0.0f));
  }
  cluster_sync();
  OgSoft s = sm.part[0];
  for (uint32_t r = 1; r < cs; ++r) og_merge(s, sm.part[r]);
  // A row without finite mass: its position is NaN.
  const bool ok = s.t.m <= FLT_MAX && s.d.m <= FLT_MAX && s.t.s > 0.0f && s.t.s <= FLT_MAX &&
                  s.d.s > 0.0f && s.d.s <= FLT_MAX;
  // log q_v = (z_v - m) - log S, with the maximum taken off first: the
  // difference of nearby logits is exact however large they are.
  const float l2d = log2f(s.d.s), cdt = __fmul_rn(__fsub_rn(l2d, log2f(s.t.s)), kLn2f);
  const float md = s.d.m, mt = s.t.m;

  // Pass 2: the sum over q u.
  float c = 0.0f;
  if (ok) {
    for (int e = threadIdx.x * 8; e < n; e += kOgThreads * 8) {
      float a[8], d[8];
      og_load<TIn>(zt, e, n, vec, a);
      og_load<TIn>(zd, e, n, vec, d);
      float g = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xd = __fsub_rn(d[j], md);
        const float q = ex2(fmaf(xd, kLog2e, -l2d));
        const float t = __fsub_rn(__fsub_rn(xd, __fsub_rn(a[j], mt)), cdt);
        g = fmaf(q, og_u(q, t, p.delta), g);
      }
      c = __fadd_rn(c, g);
    }
  }
  FF cf = warp_sum_ff(FF{c, 0.0f});
  if (lane == 0) sm.warp_c[warp] = make_float2(cf.hi, cf.lo);
  __syncthreads();
  if (threadIdx.x < cs) {
    cf = FF{0.0f, 0.0f};
    for (int w = 0; w < kOgThreads / 32; ++w) cf = ff_add(cf, FF{sm.warp_c[w].x, sm.warp_c[w].y});
    const uint32_t to = dsmem_map(&sm.part_c[rank], threadIdx.x);
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(cf.hi), "f"(cf.lo)
                 : "memory");
  }
  cluster_sync();
  cf = FF{0.0f, 0.0f};
  for (uint32_t r = 0; r < cs; ++r) cf = ff_add(cf, FF{sm.part_c[r].x, sm.part_c[r].y});
  const float C = ff_to_float(cf);
  if (!ok) {
    og_fill<TIn>(out, n, vec, __int_as_float(0x7fc00000));
    return;
  }

  // Pass 3: the gradient.
  const float g0 = __fdiv_rn(__ldg(&p.grad_loss[b]), (float)L);
  const float al = p.alpha, be = __fsub_rn(1.0f, p.alpha);
  const float base = fmaf(-be, C, al);  // alpha - (1 - alpha) C
  const int hit = s.argi - s0;
  for (int e = threadIdx.x * 8; e < n; e += kOgThreads * 8) {
    float a[8], d[8], y[8];
    og_load<TIn>(zt, e, n, vec, a);
    og_load<TIn>(zd, e, n, vec, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float xd = __fsub_rn(d[j], md);
      const float q = ex2(fmaf(xd, kLog2e, -l2d));
      const float t = __fsub_rn(__fsub_rn(xd, __fsub_rn(a[j], mt)), cdt);
      float v = __fmul_rn(q, fmaf(be, og_u(q, t, p.delta), base));
      if (e + j == hit) v = __fsub_rn(v, al);
      y[j] = __fmul_rn(v, g0);
    }
    og_store<TIn>(out, e, n, vec, y);
  }
}

}  // namespace specv
