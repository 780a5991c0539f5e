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
// A cluster of CTAs owns one position, each CTA one part of the vocabulary, which it
// copies into shared memory once (bulk copies, in pieces, so that the first pass
// starts with the first of them); partials go through distributed shared memory.
//   1. Softmax sums, the target's argmax, and A = sum e^(z_d - m_d) ((z_d - m_d)
//      - (z_t - m_t)), which gives sum_v q_v (t_v + 1) over all entries.
//   2. The clipped entries' part of it, to be taken off: q t >= delta needs
//      q >= delta / max t, so that most windows are passed over after one look at
//      the draft's logits, and all of them where no q is that large.
//   3. The gradient.
// What is taken off has to be small, or the difference keeps its roundings alone: where
// some t_v is above kOgMaxT (a target that masks entries with -1e9, say, which the drafter
// does not), and where an infinite logit makes A useless (0 x inf), the position
// sums q u entry by entry in its second pass.  Rows too long for shared memory, or not on 16-byte
// lines at their buffer's base, are read from memory in every pass (the later
// ones from L2), by the plain kernel below.
//
// Rows are worked on in windows of eight entries that start on a 16-byte line of
// the draft row (and of the gradient's, which lies alike): a vocabulary that is not a
// multiple of eight only leaves a few entries before the first and after the last
// window of each row.  The target row, which then lies differently, is read as the
// aligned blocks around a window and shifted into place.
//
// Measured: 128 requests of up to 16 rows of 151936 bf16, 313 to 335 us on several boxes
// (1.28 GB read and written once: 189 us; 370 us where every position sums entry by
// entry); DRAM at 45 % and issue at 56 % of their peaks: a third of the
// time lies between the passes (copies, cluster barriers), which three CTAs an SM
// overlap in part.  Where 256 threads a CTA took 311 us, 192, 224, 288 or 320 took 319 to 327
// (352 and more, 375 and up), 16-CTA clusters 394 to 409, resident clusters that copy ahead 359, three
// passes over L2 453.
#pragma once

#include "grad_norm.cuh"
#include "opd.cuh"

namespace specv {

constexpr int kOgThreads = 256;
constexpr int kOgMaxCluster = 8;
constexpr int kOgPieces = 4;
constexpr int kOgSmemCtas = 3;  // CTAs per SM, rows in shared memory

struct OpdGradParams {
  const void* target;      // [B, k+1, V]
  const void* draft;       // [B, k, V]
  const int32_t* lengths;  // [B]
  const float* grad_loss;  // [B]
  void* out;               // [B, k, V]
  int B, k, V;
  // Bases of draft and gradient on 16-byte lines / of the target: windows by
  // vectors, else entry by entry.
  int draft_vec, target_vec;
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

// One window: eight entries, in pairs.
struct OgWin {
  float2 x[4];
};

__device__ __forceinline__ float2 dup2(float x) { return make_float2(x, x); }

__device__ __forceinline__ float og_win_max(const OgWin& w) {
  float m = fmaxf(w.x[0].x, w.x[0].y);
#pragma unroll
  for (int e = 1; e < 4; ++e) m = fmaxf(m, fmaxf(w.x[e].x, w.x[e].y));
  return m;
}

__device__ __forceinline__ void og_add(OgAcc& a, const OgWin& w, float gm) {
  if (gm > a.m) {
    a.s = __fmul_rn(a.s, og_exp(a.m, gm));
    a.m = gm;
  }
  const float2 nm = dup2(-a.m), l2 = dup2(kLog2e);
  float2 t[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) t[e] = ex2x2(f32x2_mul(f32x2_add(w.x[e], nm), l2));
  const float2 r = f32x2_add(f32x2_add(t[0], t[1]), f32x2_add(t[2], t[3]));
  a.s = __fadd_rn(a.s, __fadd_rn(r.x, r.y));
}

__device__ __forceinline__ void og_add1(OgAcc& a, float x) {
  if (x > a.m) {
    a.s = __fmul_rn(a.s, og_exp(a.m, x));
    a.m = x;
  }
  a.s = __fadd_rn(a.s, og_exp(x, a.m));
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
  float warp_c[kOgThreads / 32];
  float part_c[kOgMaxCluster];
};

__device__ __forceinline__ OgWin og_unpack(const uint32_t* r, uint16_t) {
  OgWin w;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w.x[e] = make_float2(__uint_as_float(r[e] << 16), __uint_as_float(r[e] & 0xffff0000u));
  return w;
}
__device__ __forceinline__ OgWin og_unpack(const uint32_t* r, float) {
  OgWin w;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w.x[e] = make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
  return w;
}

// How a row's windows are read: as they lie on 16-byte lines, `shift` bytes off
// them, or entry by entry.
struct OgRow {
  const void* p;  // the row's first entry
  int shift;      // -1: entry by entry
};

// Words of an aligned window's blocks and one more, `shift` bytes into them.
template <int NB>
__device__ __forceinline__ void og_shift(uint32_t (&r)[4 * NB + 4], int shift) {
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 4 * NB + 2; ++i) r[i] = r[i + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 4 * NB + 1; ++i) r[i] = r[i + 1];
  }
  const int bits = (shift & 2) * 8;
#pragma unroll
  for (int i = 0; i < 4 * NB; ++i) r[i] = __funnelshift_r(r[i], r[i + 1], bits);
}

// The window at entry e.  A shifted one takes the aligned blocks around it (one
// more than it has itself); the caller sees to it that they lie in the buffer.
template <typename TIn>
__device__ __forceinline__ OgWin og_load(const OgRow& row, int e) {
  constexpr int NB = 8 * sizeof(TIn) / 16;  // blocks of an aligned window
  const TIn* at = static_cast<const TIn*>(row.p) + e;
  if (row.shift == 0) {
    uint32_t r[4 * NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      *reinterpret_cast<uint4*>(r + 4 * b) = reinterpret_cast<const uint4*>(at)[b];
    return og_unpack(r, TIn());
  }
  if (row.shift > 0) {
    uint32_t r[4 * NB + 4];
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(at) - row.shift);
#pragma unroll
    for (int b = 0; b <= NB; ++b) *reinterpret_cast<uint4*>(r + 4 * b) = q[b];
    og_shift<NB>(r, row.shift);
    return og_unpack(r, TIn());
  }
  OgWin w;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w.x[j] = make_float2(ElemTraits<TIn>::to_float(at[2 * j]),
                         ElemTraits<TIn>::to_float(at[2 * j + 1]));
  return w;
}

template <typename TIn>
__device__ __forceinline__ void og_store(TIn* at, bool vec, const OgWin& w) {
  using Tr = ElemTraits<TIn>;
  const float x[8] = {w.x[0].x, w.x[0].y, w.x[1].x, w.x[1].y,
                      w.x[2].x, w.x[2].y, w.x[3].x, w.x[3].y};
  if (vec) {
#pragma unroll
    for (int j = 0; j < 8; j += Tr::kPerVec)
      *reinterpret_cast<uint4*>(at + j) = pack_vec<TIn>(x + j);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) store_elem(at + j, x[j]);
  }
}

// Largest of the lanes' values (NaN is passed over), in one instruction.
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// The warp's 32 partials as one, in every lane: the maxima first, so that each
// sum is rescaled once; equal target maxima leave the lowest index.
__device__ __forceinline__ OgSoft og_warp(const OgSoft& a) {
  OgSoft r;
  r.t.m = warp_max(a.t.m);
  r.d.m = warp_max(a.d.m);
  r.t.s = warp_sum(__fmul_rn(a.t.s, og_exp(a.t.m, r.t.m)));
  r.d.s = warp_sum(__fmul_rn(a.d.s, og_exp(a.d.m, r.d.m)));
  r.argv = warp_max(a.argv);
  r.argi = __reduce_min_sync(0xffffffffu, a.argv == r.argv ? a.argi : INT32_MAX);
  return r;
}

__device__ __forceinline__ OgSoft og_none() {
  return OgSoft{{-FLT_MAX, 0.0f}, {-FLT_MAX, 0.0f}, -INFINITY, INT32_MAX, {0.0f, 0.0f}};
}

// q, u of entries with x_d = z_d - m_d and x_t = z_t - m_t: t = x_d - x_t - c and
// u = t + 1 below the clip, 0 above it.  Infinite logits need no case of their
// own: z_d = -inf gives q = 0 and q t = NaN, z_t = -inf gives t = +inf
// (q t = +inf, or NaN where q vanished), and the comparison is false for all of them.
struct OgTerms {
  float md, mt, l2d, cdt, delta;
};

__device__ __forceinline__ void og_terms(const OgTerms& k, float2 zt, float2 zd, float2& q,
                                         float2& u) {
  const float2 xd = f32x2_add(zd, dup2(-k.md)), xt = f32x2_add(zt, dup2(-k.mt));
  q = ex2x2(f32x2_fma(xd, dup2(kLog2e), dup2(-k.l2d)));
  const float2 t = f32x2_add(f32x2_fma(xt, dup2(-1.0f), xd), dup2(-k.cdt));
  const float2 f = f32x2_mul(q, t);
  u = f32x2_add(t, dup2(1.0f));
  u.x = f.x < k.delta ? u.x : 0.0f;
  u.y = f.y < k.delta ? u.y : 0.0f;
}

// What a CTA has of its position.
template <typename TIn>
struct OgPart {
  uint32_t rank, cs;
  int b, L;
  bool active;        // a verified position (the same in every CTA of the cluster)
  const TIn *zt, *zd;  // the rows
  TIn* out;
  int head;           // entries before the row's first window
  int w0, w1;         // this CTA's windows
  int edge;           // this thread's entry outside the windows (-1: none)
  int shift;          // bytes the target's windows lie off 16-byte lines
};

template <typename TIn>
__device__ __forceinline__ OgPart<TIn> og_part(const OpdGradParams& p) {
  OgPart<TIn> g;
  g.rank = cluster_rank();
  g.cs = cluster_size();
  const int pos = (int)(blockIdx.x / g.cs);  // one cluster per position
  g.b = pos / p.k;
  const int i = pos - g.b * p.k;
  const long long row = SPEC_CHECKED(pos, (long long)p.B * p.k, kSiteOpdGradRow);
  g.out = static_cast<TIn*>(p.out) + (size_t)row * p.V;
  g.zt = static_cast<const TIn*>(p.target) + ((size_t)row + g.b) * (size_t)p.V;
  g.zd = static_cast<const TIn*>(p.draft) + (size_t)row * p.V;
  g.head = p.draft_vec ? min(p.V, (int)(((16 - (reinterpret_cast<uintptr_t>(g.zd) & 15)) & 15) /
                                        sizeof(TIn)))
                       : 0;
  g.shift = (int)((reinterpret_cast<uintptr_t>(g.zt) + g.head * sizeof(TIn)) & 15);
  const int wins = (p.V - g.head) / 8, tail = g.head + wins * 8;
  const int per = (wins + (int)g.cs - 1) / (int)g.cs;
  g.w0 = min(wins, (int)g.rank * per);
  g.w1 = min(wins, g.w0 + per);
  // At most seven entries before the windows and seven after them: the first CTA's.
  g.edge = -1;
  if (g.rank == 0) {
    const int th = threadIdx.x;
    if (th < g.head) g.edge = th;
    else if (tail + th - g.head < p.V) g.edge = tail + th - g.head;
  }
  g.L = p.lengths[g.b];
  g.active = g.L >= 1 && g.L <= p.k && i < g.L;
  return g;
}

// Positions that are not verified get 0, those of a request with an invalid length NaN.
template <typename TIn>
__device__ __forceinline__ bool og_inactive(const OpdGradParams& p, const OgPart<TIn>& g) {
  if (g.active) return false;
  const float v = (g.L < 1 || g.L > p.k) ? __int_as_float(0x7fc00000) : 0.0f;
  OgWin x;
#pragma unroll
  for (int e = 0; e < 4; ++e) x.x[e] = dup2(v);
  for (int w = g.w0 + threadIdx.x; w < g.w1; w += kOgThreads)
    og_store<TIn>(g.out + g.head + w * 8, p.draft_vec != 0, x);
  if (g.edge >= 0) store_elem(g.out + g.edge, v);
  return true;
}

// Rows from memory in every pass.
template <typename TIn>
__global__ void __launch_bounds__(kOgThreads, 5) opd_grad_kernel(OpdGradParams p) {
  using Tr = ElemTraits<TIn>;
  __shared__ OgSmem sm;
  pdl_wait();
  pdl_launch_dependents();
  const OgPart<TIn> g = og_part<TIn>(p);
  const float nan = __int_as_float(0x7fc00000);
  if (og_inactive(p, g)) return;
  const uint32_t rank = g.rank, cs = g.cs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = g.head, w0 = g.w0, w1 = g.w1, edge = g.edge;
  const bool vec = p.draft_vec != 0;
  const OgRow rd = {g.zd, vec ? 0 : -1}, rt = {g.zt, p.target_vec ? g.shift : -1};
  cluster_sync();  // every CTA runs before any writes to another's shared memory

  // Pass 1: normalisers of both rows, argmax of the target.
  OgAcc at = {-FLT_MAX, 0.0f}, ad = at;
  ArgAcc ag;
  arg_init(ag);
  for (int w = w0 + threadIdx.x; w < w1; w += kOgThreads) {
    const int e = head + w * 8;
    const OgWin a = og_load<TIn>(rt, e), d = og_load<TIn>(rd, e);
    const float gm = og_win_max(a);
    og_add(at, a, gm);
    og_add(ad, d, og_win_max(d));
    if (gm > ag.v) {  // the window's first entry that is its maximum
      ag.v = gm;
#pragma unroll
      for (int j = 7; j >= 0; --j)
        if (((j & 1) ? a.x[j >> 1].y : a.x[j >> 1].x) == gm) ag.i = e + j;
    }
  }
  float et = 0.0f, ed = 0.0f;  // the entry outside the windows
  if (edge >= 0) {
    et = Tr::to_float(g.zt[edge]);
    ed = Tr::to_float(g.zd[edge]);
    og_add1(at, et);
    og_add1(ad, ed);
    arg_merge(ag, ArgAcc{et == et ? et : -INFINITY, et > -INFINITY ? edge : INT32_MAX});
  }
  OgSoft s = og_warp(OgSoft{at, ad, ag.v, ag.i, {0.0f, 0.0f}});
  if (lane == 0) sm.warp[warp] = s;
  __syncthreads();
  if (warp == 0) {
    s = og_warp(lane < kOgThreads / 32 ? sm.warp[lane] : og_none());
    if (lane < (int)cs) {  // to every CTA, this one included
      const uint32_t to = dsmem_map(&sm.part[rank], lane);
      dsmem_st4(to, make_float4(s.t.m, s.t.s, s.d.m, s.d.s));
      dsmem_st4(to + 16, make_float4(s.argv, __int_as_float(s.argi), 0.0f, 0.0f));
    }
  }
  cluster_sync();
  s = og_warp(lane < (int)cs ? sm.part[lane] : og_none());
  // A row without finite mass: its position is NaN.
  const bool ok = s.t.m <= FLT_MAX && s.d.m <= FLT_MAX && s.t.s > 0.0f && s.t.s <= FLT_MAX &&
                  s.d.s > 0.0f && s.d.s <= FLT_MAX;
  // log q_v = (z_v - m) - log S, with the maximum taken off first: the
  // difference of nearby logits is exact however large they are.
  OgTerms k;
  k.md = s.d.m;
  k.mt = s.t.m;
  k.l2d = log2f(s.d.s);
  k.cdt = __fmul_rn(__fsub_rn(k.l2d, log2f(s.t.s)), kLn2f);
  k.delta = p.delta;

  // Pass 2: the sum over q u.
  float2 c = dup2(0.0f);
  if (ok) {
    for (int w = w0 + threadIdx.x; w < w1; w += kOgThreads) {
      const int e = head + w * 8;
      const OgWin a = og_load<TIn>(rt, e), d = og_load<TIn>(rd, e);
      float2 sum = dup2(0.0f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 q, u;
        og_terms(k, a.x[j], d.x[j], q, u);
        sum = f32x2_fma(q, u, sum);
      }
      c = f32x2_add(c, sum);
    }
    if (edge >= 0) {
      float2 q, u;
      og_terms(k, dup2(et), dup2(ed), q, u);
      c.x = fmaf(q.x, u.x, c.x);
    }
  }
  float cw = warp_sum(__fadd_rn(c.x, c.y));
  if (lane == 0) sm.warp_c[warp] = cw;
  __syncthreads();
  if (warp == 0) {
    cw = warp_sum(lane < kOgThreads / 32 ? sm.warp_c[lane] : 0.0f);
    if (lane < (int)cs)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dsmem_map(&sm.part_c[rank], lane)),
                   "f"(cw)
                   : "memory");
  }
  cluster_sync();
  const float C = warp_sum(lane < (int)cs ? sm.part_c[lane] : 0.0f);

  // Pass 3: the gradient, q (beta u + base) less alpha at the argmax, all times
  // g / L.
  const float g0 = ok ? __fdiv_rn(p.grad_loss[g.b], (float)g.L) : nan;
  const float al = __fmul_rn(p.alpha, g0), be = __fmul_rn(__fsub_rn(1.0f, p.alpha), g0);
  const float base = fmaf(-be, C, al);
  const float2 be2 = dup2(be), base2 = dup2(base);
  for (int w = w0 + threadIdx.x; w < w1; w += kOgThreads) {
    const int e = head + w * 8;
    const OgWin a = og_load<TIn>(rt, e), d = og_load<TIn>(rd, e);
    OgWin y;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 q, u;
      og_terms(k, a.x[j], d.x[j], q, u);
      y.x[j] = f32x2_mul(q, f32x2_fma(be2, u, base2));
    }
    const int hit = s.argi - e;
    if (hit >= 0 && hit < 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (hit == 2 * j) y.x[j].x = __fsub_rn(y.x[j].x, al);
        if (hit == 2 * j + 1) y.x[j].y = __fsub_rn(y.x[j].y, al);
      }
    }
    og_store<TIn>(g.out + e, vec, y);
  }
  if (edge >= 0) {
    float2 q, u;
    og_terms(k, dup2(et), dup2(ed), q, u);
    const float y = __fmul_rn(q.x, fmaf(be, u.x, base));
    store_elem(g.out + edge, s.argi == edge ? __fsub_rn(y, al) : y);
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void og_qf(const OgTerms& k, float2 zt, float2 zd, float2& q, float2& f) {
  const float2 xd = f32x2_add(zd, dup2(-k.md)), xt = f32x2_add(zt, dup2(-k.mt));
  q = ex2x2(f32x2_fma(xd, dup2(kLog2e), dup2(-k.l2d)));
  const float2 t = f32x2_add(f32x2_fma(xt, dup2(-1.0f), xd), dup2(-k.cdt));
  f = f32x2_mul(q, t);
}

// What an entry changes in the second pass's sum: clipped entries' q (t + 1) comes
// off a sum over all of them (`off`), or q u is summed.
__device__ __forceinline__ float2 og_clip_part(const OgTerms& k, float2 zt, float2 zd, bool off) {
  float2 q, f;
  og_qf(k, zt, zd, q, f);
  const float2 v = f32x2_add(f, q);
  const bool bx = f.x < k.delta, by = f.y < k.delta;
  return off ? make_float2(bx ? 0.0f : -v.x, by ? 0.0f : -v.y)
             : make_float2(bx ? v.x : 0.0f, by ? v.y : 0.0f);
}

// ---------------------------------------------------------------------------
// Rows in shared memory.
// ---------------------------------------------------------------------------

// A thread's sums over its windows, relative to the warp's references mt, md:
// logits of the first windows, raised only when a logit lies more than kOgAhead
// above them (a sum then has terms up to e^40, which single precision holds as well as
// any), so that the rescaling almost never runs.
constexpr float kOgAhead = 40.0f;
// Largest t_v with which the sum over all entries is used.  The clipped entries' part
// of it is at most (kOgMaxT + 1) sum q, and the sums are good to about 2^-22 of their
// terms: 2^-17 of C's own size.
constexpr float kOgMaxT = 32.0f;
struct OgSums {
  float mt, md;
  float2 st, sd, a;  // sums of e^(z_t - m_t), e^(z_d - m_d) and of A's terms
  float dmax;        // largest (z_d - m_d) - (z_t - m_t)
  float best;        // the thread's largest target logit, and the window it is in
  int best_w;
  float dtop;        // the thread's largest draft logit
};

// The references to include gt, gd of the warp's lanes.
__device__ __forceinline__ void og_raise(OgSums& s, float gt, float gd) {
  if (!__any_sync(0xffffffffu, gt > __fadd_rn(s.mt, kOgAhead) || gd > __fadd_rn(s.md, kOgAhead)))
    return;
  const float nt = fmaxf(s.mt, warp_max(gt)), nd = fmaxf(s.md, warp_max(gd));
  const float ft = og_exp(s.mt, nt), fd = og_exp(s.md, nd);
  // A's terms are relative to both references: each moves by the difference of the moves.
  const float move = __fsub_rn(__fsub_rn(s.md, nd), __fsub_rn(s.mt, nt));
  if (s.sd.x != 0.0f || s.sd.y != 0.0f) {  // else there is nothing to move
    s.a = f32x2_mul(f32x2_fma(s.sd, dup2(move), s.a), dup2(fd));
    s.dmax = __fadd_rn(s.dmax, move);
  }
  s.st = f32x2_mul(s.st, dup2(ft));
  s.sd = f32x2_mul(s.sd, dup2(fd));
  s.mt = nt;
  s.md = nd;
}

// A window's terms (`gt`, `gd`: its largest logits).
__device__ __forceinline__ void og_window(OgSums& s, const OgWin& t, const OgWin& d, float gt,
                                          float gd, int w) {
  s.dtop = fmaxf(s.dtop, gd);
  const bool top = gt > s.best;
  s.best = top ? gt : s.best;
  s.best_w = top ? w : s.best_w;
  const float2 nt = dup2(-s.mt), nd = dup2(-s.md), l2 = dup2(kLog2e);
  float2 et[4], ed[4], a = dup2(0.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 xt = f32x2_add(t.x[j], nt), xd = f32x2_add(d.x[j], nd);
    et[j] = ex2x2(f32x2_mul(xt, l2));
    ed[j] = ex2x2(f32x2_mul(xd, l2));
    const float2 diff = f32x2_fma(xt, dup2(-1.0f), xd);
    a = j == 0 ? f32x2_mul(ed[j], diff) : f32x2_fma(ed[j], diff, a);
    s.dmax = fmaxf(s.dmax, fmaxf(diff.x, diff.y));
  }
  s.st = f32x2_add(s.st, f32x2_add(f32x2_add(et[0], et[1]), f32x2_add(et[2], et[3])));
  s.sd = f32x2_add(s.sd, f32x2_add(f32x2_add(ed[0], ed[1]), f32x2_add(ed[2], ed[3])));
  s.a = f32x2_add(s.a, a);
}

// A position's partial: a warp's, a CTA's, the cluster's.
struct OgPos {
  float mt, st, md, sd, a, dmax, argv;
  int argi;
  float dtop;
};

__device__ __forceinline__ OgPos og_none_pos() {
  return OgPos{-FLT_MAX, 0.0f,      -FLT_MAX,  0.0f,      0.0f,
               -INFINITY, -INFINITY, INT32_MAX, -INFINITY};
}

// The lanes' partials as one, in every lane.
__device__ __forceinline__ OgPos og_warp(const OgPos& x) {
  OgPos r;
  r.mt = warp_max(x.mt);
  r.md = warp_max(x.md);
  const float move = __fsub_rn(__fsub_rn(x.md, r.md), __fsub_rn(x.mt, r.mt));
  const float fd = og_exp(x.md, r.md);
  const bool any = x.sd != 0.0f;  // empty partials have maxima that mean nothing
  r.st = warp_sum(__fmul_rn(x.st, og_exp(x.mt, r.mt)));
  r.sd = warp_sum(__fmul_rn(x.sd, fd));
  r.a = warp_sum(any ? __fmul_rn(fmaf(x.sd, move, x.a), fd) : 0.0f);
  r.dmax = warp_max(any ? __fadd_rn(x.dmax, move) : -INFINITY);
  r.argv = warp_max(x.argv);
  r.argi = __reduce_min_sync(0xffffffffu, x.argv == r.argv ? x.argi : INT32_MAX);
  r.dtop = warp_max(x.dtop);
  return r;
}

// e^-x, x >= 0, with the rounding of x log2 e made good.
__device__ __forceinline__ float og_exp_down(float x) {
  const float y = __fmul_rn(x, kLog2e), rest = fmaf(x, kLog2e, -y);
  return __fmul_rn(ex2(-y), fmaf(rest, -kLn2f, 1.0f));
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// A window at a shared address; kShift: `shift` bytes into the blocks there.
template <typename TIn, bool kShift>
__device__ __forceinline__ OgWin og_smem(uint32_t addr, int shift) {
  constexpr int NB = 8 * sizeof(TIn) / 16;
  uint32_t r[4 * NB + 4];
#pragma unroll
  for (int b = 0; b < NB + (kShift ? 1 : 0); ++b) {
    const uint4 v = ld_shared16(addr + 16 * b);
    r[4 * b] = v.x;
    r[4 * b + 1] = v.y;
    r[4 * b + 2] = v.z;
    r[4 * b + 3] = v.w;
  }
  if (kShift) og_shift<NB>(r, shift);
  return og_unpack(r, TIn());
}

// The largest entry of an aligned window.
template <typename TIn>
__device__ __forceinline__ float og_smem_max(uint32_t addr) {
  uint4 v[8 * sizeof(TIn) / 16];
#pragma unroll
  for (int b = 0; b < (int)(8 * sizeof(TIn) / 16); ++b) v[b] = ld_shared16(addr + 16 * b);
  return batch_max<TIn>(v);
}

struct OgShared {
  OgPos warp[kOgThreads / 32];
  OgPos part[kOgMaxCluster];
  float warp_c[kOgThreads / 32];
  float part_c[kOgMaxCluster];
  uint64_t full[kOgPieces];  // pieces of the copies
  int abort_flag;
};

template <typename TIn, bool kShift>
__device__ __forceinline__ void og_passes(const OpdGradParams& p, const OgPart<TIn>& g, OgShared& sm,
                                          uint32_t buf, int piece) {
  using Tr = ElemTraits<TIn>;
  constexpr int kWin = 8 * sizeof(TIn);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, th = threadIdx.x;
  const int nw = g.w1 - g.w0, e0 = g.head + 8 * g.w0;
  const uint32_t bd = buf, bt = buf + nw * kWin;
  const float nan = __int_as_float(0x7fc00000);

  // Pass 1.  Whole rounds first, then one in which only some threads have a window,
  // then the entries outside the windows (the first CTA's first warp has them).
  OgSums s;
  s.mt = s.md = -FLT_MAX;
  s.st = s.sd = s.a = dup2(0.0f);
  s.dmax = s.best = s.dtop = -INFINITY;
  s.best_w = 0;
  int have = 0, ready = 0;  // pieces known to have arrived, their windows
  bool late = false;
  const int whole = nw / kOgThreads * kOgThreads;
  for (int r = 0; r < whole; r += kOgThreads) {
    for (; ready < r + kOgThreads && have < kOgPieces; ready += piece)
      late |= !mbar_sleep(&sm.full[have++], 0, &sm.abort_flag);
    const int w = r + th;
    const OgWin t = og_smem<TIn, kShift>(bt + w * kWin, g.shift);
    const OgWin d = og_smem<TIn, false>(bd + w * kWin, 0);
    const float gt = og_win_max(t), gd = og_win_max(d);
    og_raise(s, gt, gd);
    og_window(s, t, d, gt, gd, w);
  }
  // Every piece is waited for before the CTA can end; a copy that never came (a
  // bounded wait that ran out) leaves the position NaN.
  while (have < kOgPieces) late |= !mbar_sleep(&sm.full[have++], 0, &sm.abort_flag);
  __syncwarp();
  if (whole < nw) {
    const int w = whole + th;
    const bool mine = w < nw;
    OgWin t, d;
    if (mine) {
      t = og_smem<TIn, kShift>(bt + w * kWin, g.shift);
      d = og_smem<TIn, false>(bd + w * kWin, 0);
    }
    const float gt = mine ? og_win_max(t) : -INFINITY, gd = mine ? og_win_max(d) : -INFINITY;
    og_raise(s, gt, gd);
    if (mine) og_window(s, t, d, gt, gd, w);
  }
  // The thread's argmax: its best window's first entry with that value.
  ArgAcc arg = {s.best, INT32_MAX};
  if (s.best > -INFINITY) {
    const OgWin t = og_smem<TIn, kShift>(bt + s.best_w * kWin, g.shift);
#pragma unroll
    for (int j = 7; j >= 0; --j)
      if (((j & 1) ? t.x[j >> 1].y : t.x[j >> 1].x) == s.best) arg.i = e0 + s.best_w * 8 + j;
  }
  float et = 0.0f, ed = 0.0f;
  if (g.rank == 0 && warp == 0) {
    const bool mine = g.edge >= 0;
    if (mine) {
      et = Tr::to_float(g.zt[g.edge]);
      ed = Tr::to_float(g.zd[g.edge]);
    }
    og_raise(s, mine ? et : -INFINITY, mine ? ed : -INFINITY);
    if (mine) {
      if (et > arg.v || (et == arg.v && g.edge < arg.i)) arg = ArgAcc{et, g.edge};
      s.dtop = fmaxf(s.dtop, ed);
      const float xt = __fsub_rn(et, s.mt), xd = __fsub_rn(ed, s.md);
      const float e = og_exp(ed, s.md), diff = __fsub_rn(xd, xt);
      s.st.x = __fadd_rn(s.st.x, og_exp(et, s.mt));
      s.sd.x = __fadd_rn(s.sd.x, e);
      s.a.x = fmaf(e, diff, s.a.x);
      s.dmax = fmaxf(s.dmax, diff);
    }
  }
  OgPos r = {s.mt, __fadd_rn(s.st.x, s.st.y), s.md, __fadd_rn(s.sd.x, s.sd.y),
             __fadd_rn(s.a.x, s.a.y), s.dmax, arg.v, arg.i,
             s.dtop};
  if (late) r.sd = nan;
  r = og_warp(r);
  if (lane == 0) sm.warp[warp] = r;
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the peers run
  if (warp == 0) {
    r = og_warp(lane < kOgThreads / 32 ? sm.warp[lane] : og_none_pos());
    if (lane < (int)g.cs) {  // to every CTA, this one included
      const uint32_t to = dsmem_map(&sm.part[g.rank], lane);
      const float v[9] = {r.mt, r.st,   r.md,   r.sd, r.a,
                          r.dmax, r.argv, __int_as_float(r.argi), r.dtop};
#pragma unroll
      for (int e = 0; e < 9; ++e)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * e), "f"(v[e]) : "memory");
    }
  }
  cluster_sync();
  r = og_warp(lane < (int)g.cs ? sm.part[lane] : og_none_pos());
  // A row without finite mass: its position is NaN.
  const bool ok = r.mt <= FLT_MAX && r.md <= FLT_MAX && r.st > 0.0f && r.st <= FLT_MAX &&
                  r.sd > 0.0f && r.sd <= FLT_MAX;
  // From the references to the rows' maxima, where the large probabilities have
  // small exponents.
  const float up_d = __fsub_rn(r.dtop, r.md), up_t = __fsub_rn(r.argv, r.mt);
  const float shift = __fsub_rn(up_d, up_t);
  OgTerms k;
  k.md = r.dtop;
  k.mt = r.argv;
  k.l2d = log2f(__fmul_rn(r.sd, og_exp_down(up_d)));
  k.cdt = __fmul_rn(__fsub_rn(k.l2d, log2f(__fmul_rn(r.st, og_exp_down(up_t)))), kLn2f);
  k.delta = p.delta;

  // Pass 2.  `sums`: A is used, and only clipped entries are looked for; q t >= delta
  // with t <= tmax needs z_d - m_d >= least (lowered by more than the roundings).
  const float tmax = __fsub_rn(__fsub_rn(r.dmax, shift), k.cdt);
  const bool sums = ok && fabsf(r.a) <= FLT_MAX && tmax <= kOgMaxT;
  const float least = tmax > 0.0f ? __fadd_rn(__fmul_rn(__fadd_rn(log2f(__fdiv_rn(p.delta, tmax)), k.l2d),
                                                        kLn2f),
                                              -0.01f)
                                  : INFINITY;
  float C = sums ? __fadd_rn(__fsub_rn(__fsub_rn(__fdiv_rn(r.a, r.sd), shift), k.cdt), 1.0f) : 0.0f;
  // The same in every CTA of the cluster.
  if (ok && !(sums && least > 0.0f)) {
    const float from = sums ? least : -INFINITY;
    float2 c = dup2(0.0f);
    for (int w = th; w < nw; w += kOgThreads) {
      if (!(__fsub_rn(og_smem_max<TIn>(bd + w * kWin), k.md) >= from)) continue;
      const OgWin d = og_smem<TIn, false>(bd + w * kWin, 0);
      const OgWin t = og_smem<TIn, kShift>(bt + w * kWin, g.shift);
#pragma unroll
      for (int j = 0; j < 4; ++j) c = f32x2_add(c, og_clip_part(k, t.x[j], d.x[j], sums));
    }
    if (g.edge >= 0) c.x = __fadd_rn(c.x, og_clip_part(k, dup2(et), dup2(ed), sums).x);
    float cw = warp_sum(__fadd_rn(c.x, c.y));
    if (lane == 0) sm.warp_c[warp] = cw;
    __syncthreads();
    if (warp == 0) {
      cw = warp_sum(lane < kOgThreads / 32 ? sm.warp_c[lane] : 0.0f);
      if (lane < (int)g.cs)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dsmem_map(&sm.part_c[g.rank], lane)),
                     "f"(cw)
                     : "memory");
    }
    cluster_sync();
    C = __fadd_rn(C, warp_sum(lane < (int)g.cs ? sm.part_c[lane] : 0.0f));
  }

  // Pass 3: q (beta u + base), less alpha at the argmax, all times g / L.  With
  // f = q t this is beta f + (beta + base) q below the clip, base q above.
  const float g0 = ok ? __fdiv_rn(p.grad_loss[g.b], (float)g.L) : nan;
  const float al = __fmul_rn(p.alpha, g0), be = __fmul_rn(__fsub_rn(1.0f, p.alpha), g0);
  const float base = fmaf(-be, C, al);
  const float2 be2 = dup2(be), low2 = dup2(__fadd_rn(be, base));
  TIn* out = g.out + e0;
  const int hit = r.argi - e0;  // relative to this CTA's first entry
  for (int w = th; w < nw; w += kOgThreads) {
    const OgWin t = og_smem<TIn, kShift>(bt + w * kWin, g.shift);
    const OgWin d = og_smem<TIn, false>(bd + w * kWin, 0);
    OgWin y;
    float2 q[4], f[4];
    float fm = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      og_qf(k, t.x[j], d.x[j], q[j], f[j]);
      y.x[j] = f32x2_fma(f[j], be2, f32x2_mul(q[j], low2));
      fm = max_nan(fm, max_nan(f[j].x, f[j].y));
    }
    if (!(fm < k.delta)) {  // some entry is clipped, or has q = 0 and an infinite t
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!(f[j].x < k.delta)) y.x[j].x = __fmul_rn(q[j].x, base);
        if (!(f[j].y < k.delta)) y.x[j].y = __fmul_rn(q[j].y, base);
      }
    }
    if (hit >> 3 == w) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if ((hit & 7) == 2 * j) y.x[j].x = __fsub_rn(y.x[j].x, al);
        if ((hit & 7) == 2 * j + 1) y.x[j].y = __fsub_rn(y.x[j].y, al);
      }
    }
    og_store<TIn>(out + w * 8, true, y);
  }
  if (g.edge >= 0) {
    float2 q, f;
    og_qf(k, dup2(et), dup2(ed), q, f);
    const float y = f.x < k.delta ? fmaf(f.x, be, __fmul_rn(q.x, low2.x)) : __fmul_rn(q.x, base);
    store_elem(g.out + g.edge, r.argi == g.edge ? __fsub_rn(y, al) : y);
  }
}

template <typename TIn>
__global__ void __launch_bounds__(kOgThreads, kOgSmemCtas) opd_grad_smem_kernel(OpdGradParams p) {
  __shared__ OgShared sm;
  extern __shared__ __align__(128) unsigned char og_buf[];
  pdl_wait();
  pdl_launch_dependents();
  const OgPart<TIn> g = og_part<TIn>(p);
  if (og_inactive(p, g)) return;  // the whole cluster
  // The draft's windows, then the aligned blocks around the target's (the last
  // window ends within the row, and the block it shares with what follows lies
  // in the next row, which always exists).
  constexpr int kWin = 8 * sizeof(TIn);
  const int nw = g.w1 - g.w0, piece = max(1, (nw + kOgPieces - 1) / kOgPieces);
  const uint32_t more = g.shift > 0 ? 16 : 0;
  if (threadIdx.x == 0) {
    for (int c = 0; c < kOgPieces; ++c) mbar_init(&sm.full[c], 1);
    sm.abort_flag = 0;
    fence_mbar_init();
    const char* gd = reinterpret_cast<const char*>(g.zd + g.head) + (size_t)g.w0 * kWin;
    const char* gt = reinterpret_cast<const char*>(g.zt + g.head) + (size_t)g.w0 * kWin - g.shift;
    unsigned char* st = og_buf + (size_t)nw * kWin;
    const uint64_t pol = l2_policy_evict_first();
    for (int c = 0; c < kOgPieces; ++c) {
      const int a = min(nw, c * piece), n = min(nw, a + piece) - a;
      // A shifted target's first piece takes one block more, the others start
      // behind it.
      const uint32_t bytes = n * kWin, skip = c > 0 ? more : 0;
      const uint32_t tt = n > 0 ? bytes + more - skip : 0;
      mbar_arrive_expect_tx(&sm.full[c], bytes + tt);
      if (n > 0) {
        bulk_g2s_hint(og_buf + (size_t)a * kWin, gd + (size_t)a * kWin, bytes, &sm.full[c], pol);
        bulk_g2s_hint(st + (size_t)a * kWin + skip, gt + (size_t)a * kWin + skip, tt, &sm.full[c],
                      pol);
      }
    }
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const uint32_t buf = smem_addr(og_buf);
  if (g.shift > 0) og_passes<TIn, true>(p, g, sm, buf, piece);
  else og_passes<TIn, false>(p, g, sm, buf, piece);
}

}  // namespace specv
