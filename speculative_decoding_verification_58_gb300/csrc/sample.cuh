// Sampling under temperature, top-k, top-p and min-p, and the truncation alone.
//
//   order of a row's entries: z descending, index ascending; as one 64-bit number
//   ("rank") (order-preserving bits of z) << 32 | ~index, descending
//   K = a prefix of that order: the entries whose rank is at least `limit`
//   token = first index whose cumulative mass over K exceeds u * mass(K)
//
// Which entries are kept, and which one is drawn, are discrete: a sum off by one part
// in 2^24 moves a border between two entries of a flat row every few rows.
// So every entry's mass exp((z - max) / T) is a whole number of units of 2^-42 of the
// largest (2^-45 for V up to 2^18), formed to about 2^-38 of itself, and sums of
// masses are 64-bit integers: exact, and the same in any order of additions.
#pragma once

#include "common.cuh"

namespace specv {

struct SampleParams {
  const void* logits;
  const float* temperature;
  const int32_t* top_k;   // or null
  const float* top_p;     // or null
  const float* min_p;     // or null
  const float* uniforms;  // with tokens
  int32_t* tokens;        // or null
  void* kept;             // or null
  int rows, V, group;
  int unit_bits;  // the largest entry's mass is 2^unit_bits
};

// Units such that V masses fit 64 bits, none finer than 2^-45.
inline int sample_unit_bits(int V) {
  int bits = 1;
  while ((1ll << bits) < V) ++bits;
  return std::min(45, 63 - bits);
}

// Bits of z whose unsigned order is z's (-0 counts as 0).
__device__ __forceinline__ uint32_t order_bits(float z) {
  const uint32_t b = __float_as_uint(__fadd_rn(z, 0.0f));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t b) {
  return __uint_as_float(b & 0x80000000u ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ unsigned long long entry_rank(float z, int v) {
  return ((unsigned long long)order_bits(z) << 32) | (uint32_t)~v;
}

// 2^(j / 256) in units of 2^-39, j = 0 .. 255: formed by each CTA in double precision.
struct MassTable {
  unsigned long long e[256];
};
__device__ __forceinline__ void mass_table_fill(MassTable& t) {
  for (int j = threadIdx.x; j < 256; j += blockDim.x)
    t.e[j] = (unsigned long long)__double2ll_rn(exp2((double)j * (1.0 / 256.0)) * 549755813888.0);
}

// exp((z - max) / T) in units of 2^-unit_bits, rounded.  x = (z - max) log2(e) / T is formed
// in float-float and split as n + j / 256 + g, g < 2^-8 in units of 2^-40;
// 2^g = 1 + r by three terms of its series in integers.
struct MassScale {
  float max;
  FF inv;  // log2(e) / T
  int unit_bits;
};
__device__ __forceinline__ unsigned long long entry_mass(const MassScale& s, const MassTable& t,
                                                         float z) {
  const FF d = two_sum(z, -s.max);
  FF x = two_prod(d.hi, s.inv.hi);
  if (!(x.hi > -62.0f)) return 0;  // less than half a unit (or z = -inf)
  x.lo = __fmaf_rn(d.hi, s.inv.lo, __fmaf_rn(d.lo, s.inv.hi, x.lo));
  const float nf = __fadd_rn(x.hi, 12582912.0f);  // 1.5 * 2^23: rounds to a whole number
  const int n = __float_as_int(nf) - 0x4b400000;
  const float f = __fsub_rn(x.hi, __fsub_rn(nf, 12582912.0f));  // exact, |f| <= 1/2
  const float y1 = __fadd_rn(f, 12.0f);                         // to units of 2^-20
  const int i1 = __float_as_int(y1) - 0x41400000;
  const float rest = __fadd_rn(__fsub_rn(f, __fsub_rn(y1, 12.0f)), x.lo);
  const float magic = 1.5f / 131072.0f;  // to units of 2^-40
  const int i2 = __float_as_int(__fadd_rn(rest, magic)) - __float_as_int(magic);
  const long long F = ((long long)i1 << 20) + i2;
  const uint32_t g = (uint32_t)F;
  const int hi = (int)(F >> 32) + n * 256;
  const unsigned long long e = t.e[hi & 255];
  const uint32_t u = __umulhi(g, 2977044472u);  // ln 2 in units of 2^-32
  const uint32_t u2 = __umulhi(u, u);           // units of 2^-48
  const uint32_t u3 = __umulhi(u2, u);          // units of 2^-56
  const uint32_t r = u + (u2 >> 9) + (__umulhi(u3, 715827883u) >> 16);
  const unsigned long long m = e + __umulhi((uint32_t)(e >> 8), r);  // 2^-39
  // (hi >> 8 <= 0; with rounding it may be 0 where x is slightly above 0: z = max only.)
  const int shift = 39 - s.unit_bits - (hi >> 8);
  if (shift <= 0) return m << -shift;
  if (shift > 41) return 0;
  return (m + (1ull << (shift - 1))) >> shift;
}

// ceil(p * m) and floor(p * m) for a float 0 <= p <= 1.
__device__ __forceinline__ unsigned long long mass_part(float p, unsigned long long m, bool up) {
  if (!(p > 0.0f)) return 0;
  const uint32_t b = __float_as_uint(p);
  const int e = max((int)(b >> 23), 1);
  const uint32_t sig = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0);
  const int shift = 150 - e;  // p = sig * 2^-shift, shift >= 23
  const unsigned __int128 prod = (unsigned __int128)m * sig;  // below 2^88
  if (shift >= 100) return up && m > 0 ? 1 : 0;
  const unsigned __int128 add = up ? (((unsigned __int128)1 << shift) - 1) : 0;
  return (unsigned long long)((prod + add) >> shift);
}

struct CountMass {
  unsigned long long count, mass;
};

constexpr int kSampleThreads = 512;

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(0xffffffffu, x, o);
    x = y > x ? y : x;
  }
  return x;
}

// Settings of a row, checked.
struct RowSettings {
  float T, top_p, min_p;
  int top_k;
  bool ok;
};
__device__ __forceinline__ RowSettings row_settings(const SampleParams& p, int r) {
  const int q = r / p.group;
  RowSettings s;
  s.T = p.temperature[q];
  s.top_k = p.top_k != nullptr ? p.top_k[q] : 0;
  s.top_p = p.top_p != nullptr ? p.top_p[q] : 1.0f;
  s.min_p = p.min_p != nullptr ? p.min_p[q] : 0.0f;
  s.ok = temperature_ok(s.T) &&
         (s.T == 0.0f || (s.top_k >= 0 && s.top_p > 0.0f && s.top_p <= 1.0f && s.min_p >= 0.0f &&
                          s.min_p <= 1.0f));
  return s;
}

// One CTA per row; every sum is a pass over the row.
template <typename TIn>
__global__ void __launch_bounds__(kSampleThreads) sample_kernel(SampleParams p) {
  using Tr = ElemTraits<TIn>;
  __shared__ MassTable table;
  __shared__ unsigned long long red[2][kSampleThreads / 32];
  __shared__ unsigned long long best;
  __shared__ float sh_min;
  __shared__ FF sh_inv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  mass_table_fill(table);
  const int V = p.V;
  const int row = blockIdx.x;
  const TIn* in = static_cast<const TIn*>(p.logits) + (size_t)row * V;
  const RowSettings st = row_settings(p, row);
  const bool greedy = st.T == 0.0f;
  // The largest entry's rank; whether the row holds what it may not.
  unsigned long long top = 0;
  bool bad = !st.ok;
  for (int v = threadIdx.x; v < V; v += kSampleThreads) {
    const float z = Tr::to_float(in[SPEC_CHECKED(v, V, kSiteSample)]);
    if (z != z) {
      bad |= !greedy;
      continue;
    }
    bad |= !greedy && z > FLT_MAX;
    const unsigned long long rk = z < -FLT_MAX ? 0 : entry_rank(z, v);
    top = rk > top ? rk : top;
  }
  if (threadIdx.x == 0) {
    best = 0;
    const double inv = greedy ? 0.0 : 1.4426950408889634074 / (double)st.T;
    sh_inv.hi = (float)inv;
    sh_inv.lo = (float)(inv - (double)sh_inv.hi);
  }
  bad = __syncthreads_or(bad);
  top = warp_max_u64(top);
  if (lane == 0) atomicMax(&best, top);
  __syncthreads();
  top = best;
  bad = bad || top == 0;
  int token = bad ? -1 : (int)~(uint32_t)top;
  unsigned long long limit = top;
  if (!greedy && !bad) {
    MassScale s;
    s.max = Tr::to_float(in[token]);
    s.inv = sh_inv;
    s.unit_bits = p.unit_bits;
    auto sums = [&](unsigned long long from, int last) -> CountMass {  // ranks >= from, indices <= last
      unsigned long long c = 0, m = 0;
      for (int v = threadIdx.x; v <= last; v += kSampleThreads) {
        const float z = Tr::to_float(in[v]);
        if (entry_rank(z, v) >= from) {
          ++c;
          m += entry_mass(s, table, z);
        }
      }
      c = warp_sum_u64(c);
      m = warp_sum_u64(m);
      __syncthreads();
      if (lane == 0) {
        red[0][warp] = c;
        red[1][warp] = m;
      }
      __syncthreads();
      CountMass r = {0, 0};
      for (int w = 0; w < kSampleThreads / 32; ++w) {
        r.count += red[0][w];
        r.mass += red[1][w];
      }
      return r;
    };
    limit = 0;
    if (st.top_k > 0 && st.top_k < V) {
      for (int b = 63; b >= 0; --b) {
        const unsigned long long c = limit | (1ull << b);
        if (sums(c, V - 1).count >= (unsigned long long)st.top_k) limit = c;
      }
    }
    if (st.top_p < 1.0f) {
      const unsigned long long want = mass_part(st.top_p, sums(limit, V - 1).mass, true);
      unsigned long long at = 0;
      for (int b = 63; b >= 0; --b) {
        const unsigned long long c = at | (1ull << b);
        if (c <= limit || sums(c, V - 1).mass >= want) at = c;
      }
      limit = at > limit ? at : limit;
    }
    if (st.min_p > 0.0f) {
      if (threadIdx.x == 0)
        sh_min = __double2float_ru((double)s.max + (double)st.T * log((double)st.min_p));
      __syncthreads();
      const unsigned long long c = (unsigned long long)order_bits(sh_min) << 32;
      limit = c > limit ? c : limit;
    }
    if (p.tokens != nullptr) {
      const float u = p.uniforms[row];
      const unsigned long long level = mass_part(u, sums(limit, V - 1).mass, false);
      int lo = 0, hi = V - 1;  // the token is in lo .. hi
      while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (sums(limit, mid).mass > level) hi = mid;
        else lo = mid + 1;
      }
      token = u >= 0.0f && u < 1.0f ? lo : -1;
    }
  }
  if (p.tokens != nullptr && threadIdx.x == 0) p.tokens[row] = token;
  if (p.kept == nullptr) return;
  TIn* out = static_cast<TIn*>(p.kept) + (size_t)row * V;
  TIn nan, off;
  if constexpr (sizeof(TIn) == 4) {
    nan = __int_as_float(0x7fc00000);
    off = -INFINITY;
  } else {
    nan = 0x7fc0;
    off = 0xff80;
  }
  for (int v = threadIdx.x; v < V; v += kSampleThreads) {
    const TIn x = in[v];
    const float z = Tr::to_float(x);
    out[v] = bad ? nan : z == z && entry_rank(z, v) >= limit ? x : off;
  }
}

}  // namespace specv
