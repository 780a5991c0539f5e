// Sampling under temperature, top-k, top-p and min-p, and the truncation alone.
//
//   order of a row's entries: z descending, index ascending; as one 64-bit number
//   ("rank") (order-preserving bits of z) << 32 | ~index, descending
//   K = a prefix of that order: the entries whose rank is at least `limit`
//   token = first index whose cumulative mass over K exceeds u * mass(K)
//
// Which entries are kept, and which one is drawn, are discrete: a sum off by one part
// in 2^24 moves a border between two entries of a flat row every few rows.
// So where a border is decided every entry's mass exp((z - max) / T) is a whole number of
// units of 2^-42 of the largest (2^-45 for V up to 2^18), formed to about 2^-37 of itself,
// and sums of masses are 64-bit integers: exact, and the same in any order of additions.
// Masses that are less exact, but quicker to form, stand in for them only where the border is
// further away than their sums may be off by (quick_mass, 2^-28 of themselves; near_mass, 2^-16,
// of what is far below it).  A draw is a border too, and weighs its entries alike.  (Weights from
// the exponential unit alone, 10^-7 off, draw another token in one of some hundred rows: every
// border between two of 10^5 entries may be on the wrong side of the level.  And errors of that
// size do not average out where thousands of entries are equal, as plateaus of bfloat16 rows.)
//
// Measured on rows of 151936 (2048 of them, us; reading them once takes 92 in bfloat16 and
// 184 in float): greedy 119 and 215, top_k = 50 227 and 294, top_k = 400 353 and 394, no
// truncation 590 to 670 and 735 (a draw by exact masses alone: 1000 and 1040), top_p = 0.95 alone
// on rows with Zipf's tail 1760 and 1660; one row, top_k = 50: 17.  Greedy and top-k rows are
// bound by memory and by the latencies of the list's steps (two CTAs an SM; four of 256
// threads: 200, but the rows no longer stay in L2, and those that take several passes
// take longer), the others by instruction issue.
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

// 2^(j / 256) in units of 2^-39, j = 0 .. 255, from the exponential's series.
struct MassTable {
  unsigned long long e[256];
};
constexpr MassTable mass_table() {
  MassTable t = {};
  for (int j = 0; j < 256; ++j) {
    const double x = j * 0.69314718055994530942 / 256;
    double sum = 1.0, term = 1.0;
    for (int n = 1; n < 24; ++n) {
      term *= x / n;
      sum += term;
    }
    t.e[j] = (unsigned long long)(sum * 549755813888.0 + 0.5);
  }
  return t;
}
__device__ const MassTable g_mass_table = mass_table();

// exp((z - max) / T) in units of 2^-unit_bits, rounded.  x = (z - max) log2(e) / T is formed
// in float-float and split as n + j / 256 + g, g < 2^-8 in units of 2^-40;
// 2^g = 1 + r by three terms of its series in integers.
struct MassScale {
  float max;
  FF inv;  // log2(e) / T
  int unit_bits;
  float floor;  // of near_mass
  // For quick_mass: x = max log2(e) / T is start / 32 (less the bits of its rounding constant)
  // and `rest`; entries below `low` have less than half a unit.
  float rest, low;
  int start;
  bool quick;
};
__device__ __forceinline__ unsigned long long entry_mass(const MassScale& s, const MassTable& t,
                                                         float z) {
  const FF d = two_sum(z, -s.max);
  FF x = two_prod(d.hi, s.inv.hi);
  x.lo = __fmaf_rn(d.hi, s.inv.lo, __fmaf_rn(d.lo, s.inv.hi, x.lo));
  x.hi = fmaxf(x.hi, -63.0f);  // less than half a unit (or z = -inf, and x.lo anything)
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
  // (hi >> 8 <= 0, so that the shift is 17 at least.)
  const int shift = 62 - s.unit_bits - (hi >> 8);
  return shift > 63 ? 0 : ((m << 23) + (1ull << ((shift - 1) & 63))) >> (shift & 63);
}

// exp((z - max) / T) in single precision for z <= max, to 2^-16 of itself: |x| <= 64 has three
// roundings of 2^-24 of itself, times ln 2, and the exponential is right to 2^-22.  (What is
// below `floor` counts as 2^-64.)
__device__ __forceinline__ float near_mass(const MassScale& s, float z) {
  return ex2(__fmul_rn(__fsub_rn(fmaxf(z, s.floor), s.max), s.inv.hi));
}
// The same mass as entry_mass, but for 2^-28 of itself and two units, in a third of its
// instructions: sums of it tell on which side of a border they are unless they are next to it
// (`quick_doubt`).  x = (z - max) log2(e) / T is k / 32 + r, |r| < 2^-5; 2^r = 1 + q by four
// terms of its series.  Roundings of r: 2^-31 each of z's part and the maximum's, of their
// product with inv.lo and of `rest`, 2^-30 of their sum, times ln 2; q: 2^-30 of its sum, 2^-31
// of ln 2; 2^(k / 32) in units of 2^-30 and its product with 1 + q: half a unit each; what the
// series leaves out 2^-34: 4.4 2^-30 in all.  (Measured: 2^-28.3 at most.)
constexpr float kQuickRound = 393216.0f;  // 1.5 2^18: rounds to 1 / 32
struct QuickTable {
  int e[32];
};
constexpr QuickTable quick_table() {
  QuickTable t = {};
  for (int j = 0; j < 32; ++j)
    t.e[j] = (int)((mass_table().e[8 * j] + 256) >> 9);
  return t;
}
__device__ const QuickTable g_quick_table = quick_table();

__device__ __forceinline__ unsigned long long quick_mass(const MassScale& s, const int* table, float z) {
  constexpr float kOne = 4294967296.0f;  // (q in units of 2^-32)
  const float x = fmaxf(z, s.low);
  const float t = __fmaf_rn(x, s.inv.hi, kQuickRound);
  const float r = __fadd_rn(__fmaf_rn(x, s.inv.hi, -__fsub_rn(t, kQuickRound)),
                            __fmaf_rn(x, s.inv.lo, -s.rest));
  const int k = __float_as_int(t) - s.start;
  const int e = table[k & 31];
  const float h = __fmaf_rn(r, __fmaf_rn(r, 0.00961812910762847716f * kOne, 0.0555041086648215800f * kOne),
                            0.240226506959100712f * kOne);
  const int q = __float2int_rn(__fmaf_rn(r, kLn2f * kOne, __fmul_rn(__fmul_rn(r, r), h)));
  const long long m = (long long)e * q + (((long long)e << 32) | 0x80000000u);
  // (k is 1 at most, -57 * 32 at least.)
  return ((m >> 32) << 15) >> (45 - s.unit_bits - (k >> 5));
}
// How far a sum of quick masses may be from the exact ones': of n entries, `total` in all.
__device__ __forceinline__ unsigned long long quick_doubt(unsigned long long total, int n) {
  return (total >> 27) + 2ull * n;
}

// Masses next to the largest entry's; false where the temperature is too high for `floor` to
// leave out entries of -inf.
__device__ __forceinline__ bool mass_scale(MassScale& s, float max, FF inv, int unit_bits) {
  s.max = max;
  s.inv = inv;
  s.unit_bits = unit_bits;
  s.floor = __fsub_rn(max, __fdiv_rn(64.0f, inv.hi));
  FF x = two_prod(max, inv.hi);
  x.lo = __fmaf_rn(max, inv.lo, x.lo);
  const float k = rintf(__fmul_rn(x.hi, 32.0f));
  s.rest = __fadd_rn(__fsub_rn(x.hi, __fmul_rn(k, 0.03125f)), x.lo);  // (the difference is exact)
  s.low = __fsub_rn(max, __fdiv_rn(56.0f, inv.hi));
  s.quick = fabsf(x.hi) <= 16384.0f && inv.hi >= 0x1p-80f && s.low >= -FLT_MAX;
  s.start = __float_as_int(kQuickRound) + (s.quick ? (int)k : 0);
  return s.floor >= -FLT_MAX;
}

// NaN in either half of the result once an entry of the vectors so far is: maxima that keep it.
__device__ __forceinline__ uint32_t nan_of(const uint4& v, uint32_t before) {
  uint32_t d;
  asm("{\n\t.reg .b32 t, u;\n\tmax.NaN.bf16x2 t, %1, %2;\n\tmax.NaN.bf16x2 u, %3, %4;\n\t"
      "max.NaN.bf16x2 t, t, u;\n\tmax.NaN.bf16x2 %0, t, %5;\n\t}"
      : "=r"(d)
      : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(before));
  return d;
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

// ---------------------------------------------------------------------------
// One CTA per row, or a cluster of them where there are few rows, each with a run of the
// row's 16-byte vectors (the entries before the first go with the first run, those
// behind the last with the last).
//
//   top_k up to kSampleFew: one pass.  A sample of the run bounds the top_k-th largest entry from
//     below, as a rule; what is not below the bound goes to a list in shared memory.  The
//     list, sorted, has all of K: no mass of any other entry is needed.  (If it has less than
//     top_k, or does not fit, the entries are counted as for a larger top_k.)
//   top_p alone: the same pass, which lists about the largest thousand and sums the others'
//     masses in single precision.  The list's exact masses decide where the border is in it,
//     whatever the others' may be within the error of their sum.  If it is not, a histogram
//     of the distances from the maximum shows where about it is, a third pass sums quick
//     masses, of all entries and of those above that place, and counts or lists the entries
//     there; where that leaves a doubt, exact masses above the place and in fine bins of
//     the entries' bits decide.
//   Larger top_k: fine bins of the bits over all entries, counted, finer and finer until a bin's
//     entries fit the list or are all equal.
// Passes after the first find the row in L2.  (Histograms of every row's whole range by bits,
// and bisecting the rank, one pass a bit, took 5 to 30 times as long.)
// ---------------------------------------------------------------------------
constexpr int kSampleMaxCluster = 8;
constexpr int kSampleFew = 512;
constexpr int kSampleList = 2048;    // entries of the list
constexpr int kSampleTop = 1024;     // of top_p, about what is listed
constexpr int kSampleLong = 256;     // what is not cut before it is sorted
constexpr int kSampleBins = 4096;    // of the first histogram
constexpr int kSampleFine = 1024;    // of the others
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kSampleBatch = 4;      // vectors a thread has on their way
constexpr int kSamplePerSm = 2;      // CTAs

struct SamplePeer {  // what a CTA tells the others
  unsigned long long a, b;
  float x, y;
  int i, j;
};
struct SampleShared {
  union {
    unsigned long long list[kSampleList];
    uint32_t hist[kSampleBins];
  };
  union {
    unsigned long long mass[kSampleList];  // sums up to and with an entry of the sorted list
    unsigned long long fine[kSampleFine];
  };
  MassTable table;
  QuickTable quick;
  unsigned long long sums[256];  // of a draw from the list
  SamplePeer peer[2][kSampleMaxCluster];
  unsigned long long red[2][kSampleWarps];
  SamplePeer mine[kSampleWarps];
  uint32_t digit[kSampleWarps];
  int counts[17];
  FF inv;          // log2(e) / T
  double min_off;  // T log(min_p)
  int count, rest, border;
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void dsmem_st_u64(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t dsmem_ld_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long dsmem_ld_u64(uint32_t a) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// A 64-bit sum in shared memory by its halves: the hardware adds 32 bits there, and thousands of
// equal entries add to one place (as one 64-bit addition: rows of 2 ms).
__device__ __forceinline__ void add_u64(unsigned long long* sum, unsigned long long x) {
  uint32_t* half = reinterpret_cast<uint32_t*>(sum);
  const uint32_t lo = (uint32_t)x, old = atomicAdd(half, lo);
  const uint32_t hi = (uint32_t)(x >> 32) + (old + lo < old ? 1 : 0);
  if (hi != 0) atomicAdd(half + 1, hi);
}

// The first of n ascending sums that is at least `want`, n if none.
__device__ __forceinline__ int first_reaching(const unsigned long long* sums, int n,
                                              unsigned long long want) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] >= want) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// What a border is looked for by: a number of entries, or a share of their mass.
struct SampleGoal {
  bool by_count;
  unsigned long long want;  // 0: the share of the mass, found in the first pass
  float share;
};

// A CTA's part in one row.
template <typename TIn>
struct SampleJob {
  using Tr = ElemTraits<TIn>;
  static constexpr int kPer = 16 / (int)sizeof(TIn);
  SampleShared& sh;
  const SampleParams& p;
  const TIn* row;       // the whole row
  const uint4* run;     // this CTA's vectors
  int nvec, first;      // how many, index of their first entry
  int head, tail;       // entries before and behind them that are this CTA's
  int rank, ctas, round;
  MassScale s;

  // f(values, index of the first, how many) for all of the run, threads in turn, but for
  // vectors whose entries are all below `least`.
  template <typename F>
  __device__ __forceinline__ void each(float least, F&& f) const {
    for (int i0 = threadIdx.x; i0 < nvec; i0 += kSampleBatch * kSampleThreads) {
      uint4 v[kSampleBatch];
#pragma unroll
      for (int j = 0; j < kSampleBatch; ++j) {
        const int i = i0 + j * kSampleThreads;
        if (i < nvec) v[j] = run[i];
      }
#pragma unroll
      for (int j = 0; j < kSampleBatch; ++j) {
        const int i = i0 + j * kSampleThreads;
        if (i >= nvec) break;
        float x[kPer];
        Tr::unpack(v[j], x);
        if (reaches(x, least)) f(x, first + i * kPer, kPer);
      }
    }
    if ((int)threadIdx.x < head + tail) {
      float x[kPer];
      const int v = edge(threadIdx.x);
      x[0] = Tr::to_float(row[SPEC_CHECKED(v, p.V, kSiteSample)]);
      f(x, v, 1);
    }
  }
  static __device__ __forceinline__ bool reaches(const float* x, float least) {
    float most = x[0];
#pragma unroll
    for (int e = 1; e < kPer; ++e) most = fmaxf(most, x[e]);
    return most >= least;
  }
  // The sum of all CTAs' words at the same place of shared memory; their loads go together.
  __device__ __forceinline__ uint32_t sum_of(const uint32_t* x) const {
    if (ctas == 1) return *x;
    uint32_t v[kSampleMaxCluster], sum = 0;
#pragma unroll
    for (int i = 0; i < kSampleMaxCluster; ++i) v[i] = dsmem_ld_u32(dsmem_map(x, ::min(i, ctas - 1)));
#pragma unroll
    for (int i = 0; i < kSampleMaxCluster; ++i) sum += i < ctas ? v[i] : 0;
    return sum;
  }
  __device__ __forceinline__ unsigned long long sum_of(const unsigned long long* x) const {
    if (ctas == 1) return *x;
    unsigned long long v[kSampleMaxCluster], sum = 0;
#pragma unroll
    for (int i = 0; i < kSampleMaxCluster; ++i) v[i] = dsmem_ld_u64(dsmem_map(x, ::min(i, ctas - 1)));
#pragma unroll
    for (int i = 0; i < kSampleMaxCluster; ++i) sum += i < ctas ? v[i] : 0;
    return sum;
  }
  // The t-th entry outside the vectors.
  __device__ __forceinline__ int edge(int t) const {
    return t < head ? first - head + t : first + nvec * kPer + t - head;
  }

  // Every CTA's word for all of them, in rank order; thread 0's argument counts.
  __device__ __forceinline__ const SamplePeer* exchange(const SamplePeer& word) {
    SamplePeer* slot = sh.peer[round++ & 1];
    __syncthreads();
    if (ctas == 1) {
      if (threadIdx.x == 0) slot[0] = word;
      __syncthreads();
      return slot;
    }
    if (threadIdx.x == 0) sh.mine[0] = word;
    __syncthreads();
    if ((int)threadIdx.x < ctas) {
      const uint32_t to = dsmem_map(&slot[rank], threadIdx.x);
      const SamplePeer m = sh.mine[0];
      dsmem_st_u64(to, m.a);
      dsmem_st_u64(to + 8, m.b);
      dsmem_st_u64(to + 16, ((unsigned long long)__float_as_uint(m.y) << 32) | __float_as_uint(m.x));
      dsmem_st_u64(to + 24, ((unsigned long long)(uint32_t)m.j << 32) | (uint32_t)m.i);
    }
    cluster_arrive();
    cluster_wait();
    return slot;
  }
  __device__ __forceinline__ void sync_all() {
    if (ctas == 1) {
      __syncthreads();
    } else {
      cluster_arrive();
      cluster_wait();
    }
  }
  // Sums over the CTA's threads, for all of them.
  __device__ __forceinline__ CountMass block_sums(unsigned long long c, unsigned long long m) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    c = warp_sum_u64(c);
    m = warp_sum_u64(m);
    __syncthreads();
    if (lane == 0) {
      sh.red[0][warp] = c;
      sh.red[1][warp] = m;
    }
    __syncthreads();
    CountMass r = {0, 0};
#pragma unroll
    for (int w = 0; w < kSampleWarps; ++w) {
      r.count += sh.red[0][w];
      r.mass += sh.red[1][w];
    }
    return r;
  }
  __device__ __forceinline__ CountMass cluster_sums(unsigned long long c, unsigned long long m) {
    const CountMass r = block_sums(c, m);
    SamplePeer w = {};
    w.a = r.count;
    w.b = r.mass;
    const SamplePeer* all = exchange(w);
    CountMass t = {0, 0};
    for (int i = 0; i < ctas; ++i) {
      t.count += all[i].a;
      t.mass += all[i].b;
    }
    return t;
  }

  // The largest 16-bit number that at least k of the threads' kN numbers reach, 0 if there are
  // fewer (but for zeros).  Each warp finds the one that its share of the k reach among its
  // own; the result is between the least and the largest of those, and the CTA's counts
  // are needed only for the bits in which they differ.
  template <int kN>
  __device__ __forceinline__ uint32_t kth(const uint32_t (&g)[kN], int k) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = (k + kSampleWarps - 1) / kSampleWarps;
    auto count = [&](uint32_t c) -> int {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) n += g[i] >= c ? 1 : 0;
      return __reduce_add_sync(0xffffffffu, n);
    };
    uint32_t mine = 0;
#pragma unroll 1
    for (int b = 15; b >= 0; --b)
      if (count(mine | (1u << b)) >= share) mine |= 1u << b;
    __syncthreads();
    if (lane == 0) sh.digit[warp] = mine;
    if (threadIdx.x < 17) sh.counts[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t least = __reduce_min_sync(0xffffffffu, sh.digit[lane % kSampleWarps]);
    // (At least k reach `least`: every warp has its share.)
    uint32_t at = least, over = __reduce_max_sync(0xffffffffu, sh.digit[lane % kSampleWarps]) + 1;
    for (int round = 0; over - at > 1; ++round) {
      const uint32_t mid = (at + over) >> 1;
      const int n = count(mid);
      if (lane == 0 && n) atomicAdd(&sh.counts[round], n);
      __syncthreads();
      if (sh.counts[round] >= k) at = mid;
      else over = mid;
    }
    return at;
  }

  __device__ __forceinline__ void append(float z, int v) {
    const int k = atomicAdd(&sh.count, 1);
    if (k < kSampleList) sh.list[k] = entry_rank(z, v);
  }
  // What of the list is at least `least` (an order's upper 16 bits).
  __device__ __forceinline__ void cut_list(uint32_t least) {
    constexpr int kEach = kSampleList / kSampleThreads;
    unsigned long long x[kEach];
    __syncthreads();
    const int n = min(sh.count, kSampleList);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + e * kSampleThreads;
      x[e] = i < n ? sh.list[i] : 0;
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (x[e] != 0 && (uint32_t)(x[e] >> 48) >= least) sh.list[atomicAdd(&sh.count, 1)] = x[e];
    __syncthreads();
  }
  __device__ __forceinline__ uint32_t list_kth(int k) {
    constexpr int kEach = kSampleList / kSampleThreads;
    uint32_t g[kEach];
    __syncthreads();
    const int n = min(sh.count, kSampleList);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + e * kSampleThreads;
      g[e] = i < n ? (uint32_t)(sh.list[i] >> 48) : 0;
    }
    return kth(g, k);
  }
  // The CTAs' lists one behind the other in the first one's.  Returns their length, -1 if they
  // do not fit.
  __device__ __forceinline__ int gather() {
    __syncthreads();
    if (ctas == 1) return sh.count <= kSampleList ? sh.count : -1;
    SamplePeer w = {};
    w.i = sh.count;
    const SamplePeer* all = exchange(w);
    int before = 0, total = 0;
    bool fits = true;
    for (int i = 0; i < ctas; ++i) {
      fits = fits && all[i].i <= kSampleList;
      if (i < rank) before += all[i].i;
      total += fits ? all[i].i : 0;
    }
    if (!fits || total > kSampleList) return -1;
    if (rank > 0)
      for (int i = threadIdx.x; i < sh.count; i += kSampleThreads)
        dsmem_st_u64(dsmem_map(&sh.list[before + i], 0), sh.list[i]);
    sync_all();
    return total;
  }
  // Sorts the list (descending); the first CTA alone.  A short one by counting for each entry
  // those before it, several threads to an entry (138 entries 0.6 us, by exchanges 3).
  __device__ __forceinline__ void sort(int n) {
    int size = 32;
    while (size < n) size *= 2;
    if (size <= 256) {
      const int i = threadIdx.x & (size - 1), part = threadIdx.x / size;
      const int parts = kSampleThreads / size, each = (n + parts - 1) / parts;
      const unsigned long long x = i < n ? sh.list[i] : 0;
      int* place = reinterpret_cast<int*>(sh.mass);
      __syncthreads();
      if ((int)threadIdx.x < n) place[threadIdx.x] = 0;
      __syncthreads();
      int before = 0;
      if (i < n)
        for (int j = part * each; j < min(n, (part + 1) * each); ++j) before += sh.list[j] > x ? 1 : 0;
      if (before > 0) atomicAdd(&place[i], before);
      __syncthreads();
      if ((int)threadIdx.x < n) {
        const int to = place[threadIdx.x];
        before = to;
      }
      __syncthreads();
      if ((int)threadIdx.x < n) sh.list[before] = x;
      __syncthreads();
      return;
    }
    if (size <= kSampleThreads) sort_exchange<1>(n);
    else if (size <= 2 * kSampleThreads) sort_exchange<2>(n);
    else sort_exchange<4>(n);
  }
  // A longer one by exchanges (bitonic), kE neighbours in a thread's registers: those that stay
  // within a warp by shuffles (930 entries through shared memory alone: 15 us).
  template <int kE>
  __device__ __forceinline__ void sort_exchange(int n) {
    const int at = threadIdx.x * kE;
    unsigned long long x[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) x[e] = at + e < n ? sh.list[at + e] : 0;
#pragma unroll 1
    for (int k = 2; k <= kE * kSampleThreads; k *= 2) {
#pragma unroll 1
      for (int j = k / 2; j >= kE; j /= 2) {
        unsigned long long y[kE];
        if (j < 32 * kE) {
#pragma unroll
          for (int e = 0; e < kE; ++e) y[e] = __shfl_xor_sync(0xffffffffu, x[e], j / kE);
        } else {
          __syncthreads();
#pragma unroll
          for (int e = 0; e < kE; ++e) sh.list[at + e] = x[e];
          __syncthreads();
#pragma unroll
          for (int e = 0; e < kE; ++e) y[e] = sh.list[(at + e) ^ j];
        }
        // (Runs whose bit k is 0 descend; of a pair there the lower place has the larger.)
        const bool larger = ((at & k) == 0) == ((at & j) == 0);
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = (x[e] > y[e]) == larger ? x[e] : y[e];
      }
#pragma unroll
      for (int j = kE / 2; j > 0; j /= 2) {
        if (j >= k) continue;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          if (e & j) continue;
          const bool descends = ((at + e) & k) == 0;
          const unsigned long long a = x[e], b = x[e | j];
          if ((a < b) == descends) {
            x[e] = b;
            x[e | j] = a;
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kE; ++e) sh.list[at + e] = x[e];
    __syncthreads();
  }
  // In sh.mass the masses of the sorted list's entries, summed up.
  __device__ __forceinline__ void list_masses(int n) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kEach = kSampleList / kSampleThreads;
    unsigned long long m[kEach], mine = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x * kEach + e;
      const float z = i < n ? from_order_bits((uint32_t)(sh.list[i] >> 32)) : -INFINITY;
      m[e] = entry_mass(s, sh.table, z);
      mine += m[e];
    }
    unsigned long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) sh.red[0][warp] = upto;
    __syncthreads();
    unsigned long long before = upto - mine;
    for (int w = 0; w < warp; ++w) before += sh.red[0][w];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      before += m[e];
      const int i = threadIdx.x * kEach + e;
      if (i < n) sh.mass[i] = before;
    }
    __syncthreads();
  }

  // The lowest index among the list's first n entries whose mass with those of all lower ones
  // exceeds the level; the first CTA alone.
  __device__ __forceinline__ int draw_listed(int n, unsigned long long level) {
    const int tid = threadIdx.x;
    if (tid == 0) sh.border = p.V;
    __syncthreads();
    int size = 32;
    while (size < n) size *= 2;
    if (size <= 256) {
      // Each entry's sum, several threads to an entry.
      const int i = tid & (size - 1), part = tid / size;
      const int parts = kSampleThreads / size, each = (n + parts - 1) / parts;
      if (tid < n) sh.sums[tid] = 0;
      __syncthreads();
      const uint32_t mine = i < n ? (uint32_t)sh.list[i] : 0xffffffffu;  // (~index)
      unsigned long long m = 0;
      if (i < n) {
        const int j0 = part * each, j1 = min(n, j0 + each);
        unsigned long long last = j0 > 0 && j0 < j1 ? sh.mass[j0 - 1] : 0;
        for (int j = j0; j < j1; ++j) {
          const unsigned long long upto = sh.mass[j];
          if ((uint32_t)sh.list[j] >= mine) m += upto - last;
          last = upto;
        }
      }
      if (m != 0) atomicAdd(&sh.sums[i], m);
      __syncthreads();
      if (tid < n && sh.sums[tid] > level) atomicMin(&sh.border, (int)~(uint32_t)sh.list[tid]);
      __syncthreads();
      return sh.border;
    }
    // By halving the range of the index, but into as many parts as there are warps, each of
    // which sums up to one of the ends.
    const int warp = tid >> 5, lane = tid & 31;
    int lo = 0, hi = p.V - 1;
    while (lo < hi) {
      auto end = [&](int w) -> int { return lo + (int)((long long)(hi - lo) * (w + 1) / (kSampleWarps + 1)); };
      const int mine = end(warp);
      unsigned long long m = 0;
      for (int i = lane; i < n; i += 32)
        if ((int)~(uint32_t)sh.list[i] <= mine) m += sh.mass[i] - (i > 0 ? sh.mass[i - 1] : 0);
      m = warp_sum_u64(m);
      __syncthreads();
      if (lane == 0) sh.red[0][warp] = m;
      __syncthreads();
      int w = 0;
      while (w < kSampleWarps && sh.red[0][w] <= level) ++w;
      const int below = w > 0 ? end(w - 1) + 1 : lo;
      if (w < kSampleWarps) hi = end(w);
      lo = below;
    }
    return lo;
  }

  // The first index, ascending, whose weight with all lower ones' exceeds `level(total)`; -1
  // if none does, or if the level is not further than `doubt(total)` from both that sum and
  // the one before.  Weights of the warps' runs first; the warp in whose run the level is passed
  // goes through it again.
  // Then the CTA in whose run the level is passed goes through that warp's run again, shared
  // out among its warps, and one of these through its share (one warp through all of the
  // run, a load after the other, took 17 us of a row of 151936).
  template <typename W, typename L, typename D>
  __device__ __forceinline__ int locate(float least, W&& weight, L&& level_of, D&& doubt_of) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tail0 = first + nvec * kPer;
    auto single = [&](int v, bool here) -> unsigned long long {
      return here ? weight(Tr::to_float(row[v]), v) : 0;
    };
    auto vector_weight = [&](int i) -> unsigned long long {
      float x[kPer];
      Tr::unpack(run[i], x);
      unsigned long long m = 0;
      if (reaches(x, least)) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) m += weight(x[e], first + i * kPer + e);
      }
      return m;
    };
    // Vectors from .. to - 1, the entries before all and behind all: of this warp.
    int from = (int)((long long)nvec * warp / kSampleWarps);
    int to = (int)((long long)nvec * (warp + 1) / kSampleWarps);
    int heads = warp == 0 ? head : 0, tails = warp == kSampleWarps - 1 ? tail : 0;
    // The warps' sums, and for all threads what is before each.
    auto sums = [&]() -> unsigned long long {
      unsigned long long m =
          single(first - head + lane, lane < heads) + single(tail0 + lane, lane < tails);
#pragma unroll 4
      for (int i = from + lane; i < to; i += 32) m += vector_weight(i);
      m = warp_sum_u64(m);
      __syncthreads();
      if (lane == 0) sh.red[0][warp] = m;
      if (threadIdx.x == 0) sh.border = -1;
      __syncthreads();
      unsigned long long all = 0;
      for (int i = 0; i < kSampleWarps; ++i) all += sh.red[0][i];
      return all;
    };
    SamplePeer w = {};
    w.a = sums();
    const SamplePeer* all = exchange(w);
    unsigned long long total = 0, upto = 0;
    for (int i = 0; i < ctas; ++i) {
      if (i < rank) upto += all[i].a;
      total += all[i].a;
    }
    const unsigned long long level = level_of(total), doubt = doubt_of(total);
    if (upto <= level && level < upto + w.a) {
      auto pick = [&]() -> int {  // the warp in whose part the level is passed
        int q = 0;
        while (q < kSampleWarps - 1 && upto + sh.red[0][q] <= level) upto += sh.red[0][q++];
        return q;
      };
      const int q = pick();
      const int a = (int)((long long)nvec * q / kSampleWarps);
      const int n = (int)((long long)nvec * (q + 1) / kSampleWarps) - a;
      from = a + n * warp / kSampleWarps;
      to = a + n * (warp + 1) / kSampleWarps;
      heads = q == 0 && warp == 0 ? head : 0;
      tails = q == kSampleWarps - 1 && warp == kSampleWarps - 1 ? tail : 0;
      sums();
      if (pick() == warp) {
        int found = -1;
        auto look = [&](unsigned long long x, auto&& finish) {  // the lanes' weights, in order
          unsigned long long sum = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
          }
          const uint32_t over = __ballot_sync(0xffffffffu, upto + sum > level);
          if (over != 0) {
            const int l = __ffs(over) - 1;
            if (lane == l) found = finish(upto + sum - x, upto + sum);
            found = __shfl_sync(0xffffffffu, found, l);
          }
          upto += __shfl_sync(0xffffffffu, sum, 31);
        };
        // (The sums before an entry and with it.)
        auto sure = [&](int v, unsigned long long less, unsigned long long sum) {
          return level - less >= doubt && sum - level > doubt ? v : -2;
        };
        if (heads > 0) {
          const int v = first - head + lane;
          look(single(v, lane < heads),
               [&](unsigned long long less, unsigned long long sum) { return sure(v, less, sum); });
        }
        for (int i0 = from; i0 < to && found == -1; i0 += 32) {
          const int i = i0 + lane;
          look(i < to ? vector_weight(i) : 0, [&](unsigned long long less, unsigned long long) {
            float x[kPer];
            Tr::unpack(run[i], x);
            int v = first + i * kPer;
            unsigned long long sum = less;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              if (sum > level) break;
              less = sum;
              sum += weight(x[e], first + i * kPer + e);
              v = first + i * kPer + e;
            }
            return sure(v, less, sum);
          });
        }
        if (tails > 0 && found == -1) {
          const int v = tail0 + lane;
          look(single(v, lane < tails),
               [&](unsigned long long less, unsigned long long sum) { return sure(v, less, sum); });
        }
        if (lane == 0) sh.border = found;
      }
    }
    __syncthreads();
    SamplePeer w2 = {};
    w2.i = sh.border;
    all = exchange(w2);
    int found = -1;
    for (int i = 0; i < ctas; ++i) found = ::max(found, all[i].i);
    return found;
  }

  // The value of a key.  (The bits that bfloat16 does not have are ones in a negative number's
  // order.)
  static __device__ __forceinline__ float key_value(uint32_t k) {
    return from_order_bits(sizeof(TIn) == 4 ? k : (k << 16) | (k & 0x8000u ? 0u : 0xffffu));
  }

  // The largest rank from which on the entries of rank `from` and more reach the goal (all of
  // them together do).  lo .. hi: order bits between which it is thought to be; taken to be
  // anywhere if it is not.
  __device__ __forceinline__ unsigned long long border_rank(SampleGoal goal, unsigned long long from,
                                                            uint32_t lo, uint32_t hi) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // bfloat16: the lower 16 bits say nothing.
    constexpr int kDrop = sizeof(TIn) == 2 ? 16 : 0;
    bool widened = false;
    for (;;) {
      const uint32_t k0 = lo >> kDrop, k1 = hi >> kDrop;
      int shift = 0;
      while (((k1 - k0) >> shift) >= (uint32_t)kSampleFine) ++shift;
      __syncthreads();
      for (int i = tid; i < kSampleFine; i += kSampleThreads) {
        sh.hist[i] = 0;
        sh.fine[i] = 0;
      }
      __syncthreads();
      unsigned long long count = 0, mass = 0;  // above hi
      float low = from_order_bits(k0 << kDrop);
      if (!(low == low)) low = -INFINITY;  // (no bound)
      const bool all_mass = !goal.by_count && goal.want == 0;  // `count` is the mass of all
      const bool equal = kDrop && shift == 0;  // a bin's entries are
      each(all_mass ? -INFINITY : low, [&](const float* x, int v, int n) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const uint32_t k = order_bits(x[e]) >> kDrop;
          const bool counts = (e < n) & (entry_rank(x[e], v + e) >= from);
          if (goal.by_count) {
            count += counts & (k > k1) ? 1 : 0;
          } else if (all_mass || k >= k0) {
            const unsigned long long m = counts ? entry_mass(s, sh.table, x[e]) : 0;
            if (all_mass) count += m;
            mass += k > k1 ? m : 0;
            if (!equal && (m != 0) & (k >= k0) & (k <= k1)) add_u64(&sh.fine[(k - k0) >> shift], m);
          }
          if (counts & (k >= k0) & (k <= k1)) atomicAdd(&sh.hist[(k - k0) >> shift], 1u);
        }
      });
      const CountMass above = cluster_sums(count, mass);
      if (all_mass) goal.want = mass_part(goal.share, above.count, true);
      // From the top bin down: thread t has two bins, and what is above them.
      const unsigned long long start = goal.by_count ? above.count : above.mass;
      SamplePeer w = {};
      w.i = -1;
      if (rank == 0) {
        constexpr int kEach = kSampleFine / kSampleThreads;
        unsigned long long n[kEach], mine = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int b = kSampleFine - 1 - (tid * kEach + e);
          if (goal.by_count || equal) {
            n[e] = sum_of(&sh.hist[b]);
            if (!goal.by_count && n[e] != 0) n[e] *= entry_mass(s, sh.table, key_value(k0 + b));
          } else {
            n[e] = sum_of(&sh.fine[b]);
          }
          mine += n[e];
        }
        unsigned long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        if (lane == 31) sh.red[0][warp] = upto;
        if (tid == 0) sh.border = -1;
        __syncthreads();
        unsigned long long before = start + upto - mine;
        for (int q = 0; q < warp; ++q) before += sh.red[0][q];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          if (before < goal.want && before + n[e] >= goal.want) {
            sh.border = kSampleFine - 1 - (tid * kEach + e);
            sh.red[1][0] = before;
          }
          before += n[e];
        }
        __syncthreads();
        if (tid == 0 && sh.border >= 0) {
          w.i = sh.border;
          w.a = sh.red[1][0];
          w.j = (int)sum_of(&sh.hist[sh.border]);
        }
      }
      const SamplePeer* all = exchange(w);
      const int bin = all[0].i, entries = all[0].j;
      const unsigned long long before = all[0].a;
      if (bin < 0) {
        if (widened) return from;  // (does not happen: all entries together reach the goal)
        widened = true;
        lo = 0;
        hi = 0xffffffffu;
        continue;
      }
      const uint32_t b0 = k0 + ((uint32_t)bin << shift);
      const uint32_t b1 = ::min(k1, b0 + ((1u << shift) - 1));
      if (entries <= kSampleList) {
        __syncthreads();
        if (tid == 0) sh.count = 0;
        __syncthreads();
        each(low, [&](const float* x, int v, int n) {
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            if (e >= n) continue;
            const uint32_t k = order_bits(x[e]) >> kDrop;
            if (k >= b0 && k <= b1 && entry_rank(x[e], v + e) >= from) append(x[e], v + e);
          }
        });
        const int n = gather();
        SamplePeer w2 = {};
        if (rank == 0) {
          sort(n);
          int i;
          if (goal.by_count) {
            i = (int)(goal.want - before) - 1;
          } else {
            list_masses(n);
            i = first_reaching(sh.mass, n, goal.want - before);
          }
          w2.a = sh.list[::min(i, n - 1)];
        }
        return exchange(w2)[0].a;
      }
      if (shift == 0) {
        // All equal: the lowest indices, as many as are wanted.
        const float z = key_value(b0);
        unsigned long long nth = goal.want - before;
        if (!goal.by_count) {
          const unsigned long long m = entry_mass(s, sh.table, z);
          nth = (nth + m - 1) / m;
        }
        const int v = locate(
            z, [&](float y, int at) -> unsigned long long {
              return order_bits(y) >> kDrop == b0 && entry_rank(y, at) >= from ? 1 : 0;
            },
            [&](unsigned long long) { return nth - 1; }, [](unsigned long long) { return 0ull; });
        return entry_rank(z, v);
      }
      lo = b0 << kDrop;
      hi = (b1 << kDrop) | (kDrop ? 0xffffu : 0u);
    }
  }
};

// The draw by exact masses, for all threads.  A function of its own, with a copy of the job: its
// code within the kernel costs the other paths registers (2048 rows, top_k = 50: 240 us, 227 so).
template <typename TIn>
__device__ __noinline__ int exact_draw(SampleJob<TIn> job, float least, uint32_t last, float u) {
  return job.locate(
      least,
      [&](float z, int v) -> unsigned long long {
        return (z > least) | ((z == least) & ((uint32_t)v <= last)) ? entry_mass(job.s, job.sh.table, z)
                                                                    : 0;
      },
      [&](unsigned long long total) { return mass_part(u, total, false); },
      [](unsigned long long) { return 0ull; });
}

template <typename TIn>
__global__ void __launch_bounds__(kSampleThreads, kSamplePerSm)
    sample_kernel(const __grid_constant__ SampleParams p) {
  using Tr = ElemTraits<TIn>;
  constexpr int kPer = SampleJob<TIn>::kPer;
  __shared__ __align__(16) SampleShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), ctas = (int)cluster_size();
  const int V = p.V, r = blockIdx.x / ctas;
  if (ctas > 1) cluster_arrive();  // (waited for before the first word to another CTA)
  if (tid == 0) sh.count = 0;
  for (int i = tid; i < 256; i += kSampleThreads) sh.table.e[i] = g_mass_table.e[i];
  if (tid < 32) sh.quick.e[tid] = g_quick_table.e[tid];
  pdl_wait();
  pdl_launch_dependents();
  SampleJob<TIn> job = {sh, p};
  job.rank = rank;
  job.ctas = ctas;
  job.round = 0;
  job.row = static_cast<const TIn*>(p.logits) + (size_t)r * V;
  const uintptr_t at = reinterpret_cast<uintptr_t>(job.row);
  const int before = min((int)((16 - at % 16) % 16 / sizeof(TIn)), V);
  const int nv = (V - before) / kPer;
  const int v0 = (int)((long long)nv * rank / ctas), v1 = (int)((long long)nv * (rank + 1) / ctas);
  job.nvec = v1 - v0;
  job.first = before + v0 * kPer;
  job.head = rank == 0 ? before : 0;
  job.tail = rank == ctas - 1 ? V - before - nv * kPer : 0;
  job.run = reinterpret_cast<const uint4*>(job.row + job.first);
  const int nvec = job.nvec, edges = job.head + job.tail;

  // The sample, 512 bytes here and there of the whole run, and the first vectors are on
  // their way while the settings are read.
  uint4 next[kSampleBatch];
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kSampleBatch; ++j) {
      const int i = i0 + j * kSampleThreads + tid;
      if (i < nvec) next[j] = job.run[i];
    }
  };
  // (A run shorter than the sample is all of it.)
  constexpr int kPieces = kSampleBatch * kSampleWarps;
  auto sample_at = [&](int j) -> int {
    const int piece = j * kSampleWarps + warp;
    const int at = nvec <= kPieces * 32 ? piece * 32
                                        : (int)((long long)(nvec - 32) * piece / (kPieces - 1));
    return at + lane;
  };
  const RowSettings st = row_settings(p, r);
  const bool greedy = st.T == 0.0f;
  const bool cut_k = !greedy && st.top_k > 0 && st.top_k < V, cut_p = !greedy && st.top_p < 1.0f;
  const bool few = cut_k && st.top_k <= kSampleFew;
  const bool share = cut_p && !cut_k;  // a share of the whole row's mass
  const bool listing = st.ok && (few || share);
  // How many of the sample's entries the list's bound is to leave: with `share` any bound will
  // do, and one that leaves about kSampleTop entries of all CTAs is taken; top_k's has to
  // leave top_k, so that what the sample should have of them is taken five standard
  // deviations and some more (if that does not do, all entries are counted).
  constexpr int kStep = kSampleBatch * kSampleThreads;
  const float part_of = fminf(1.0f, (float)kStep / (float)::max(nvec, 1));
  const float mean = (float)(few ? st.top_k : kSampleTop) * part_of / (float)ctas;
  const int target = part_of == 1.0f && ctas == 1 ? (few ? st.top_k : kSampleTop)
                                                   : (int)(mean + (few ? 5.0f * sqrtf(mean) + 8.0f : 1.0f));
  if (st.ok && !greedy) {
    if (tid == 32) {  // (in double precision, which is slow: beside the loads)
      const double inv = 1.4426950408889634074 / (double)st.T;
      sh.inv.hi = (float)inv;
      sh.inv.lo = (float)(inv - (double)sh.inv.hi);
    }
    if (tid == 64 && st.min_p > 0.0f) sh.min_off = (double)st.T * log((double)st.min_p);
  }

  // First pass: the list, the largest, and with `share` the mass of what is not listed in single
  // precision, next to the largest of the sample (which none of it is above).
  bool bad = !st.ok, overflow = false;
  float top = -INFINITY;  // the largest entry of the vectors
  const float edge = tid < edges ? Tr::to_float(job.row[SPEC_CHECKED(job.edge(tid), V, kSiteSample)])
                                 : -INFINITY;
  bad |= edge != edge && !greedy;
  int top_vec = -1;  // greedy: the vector it is in, the first
  float nan = 0.0f;  // NaN once an entry is
  uint32_t least_bits = 0;
  MassScale s0 = {};
  bool scaled = true;
  if (!listing) load(0);
  FF sum = {0.0f, 0.0f};
  float listed_sum = 0.0f;  // about
  if (listing) {
    float half[2 * kSampleBatch], most = -INFINITY;
#pragma unroll
    for (int j = 0; j < kSampleBatch; ++j) {
      const int i = sample_at(j);
      if (i < nvec) next[j] = job.run[i];
    }
#pragma unroll
    for (int j = 0; j < kSampleBatch; ++j) {
      half[2 * j] = half[2 * j + 1] = -INFINITY;
      if (sample_at(j) < nvec) {
        float x[kPer];
        Tr::unpack(next[j], x);
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          half[2 * j + (e >= kPer / 2)] = fmaxf(half[2 * j + (e >= kPer / 2)], x[e]);
      }
      most = fmaxf(most, fmaxf(half[2 * j], half[2 * j + 1]));
    }
    load(0);
    uint32_t g[2 * kSampleBatch];
#pragma unroll
    for (int j = 0; j < 2 * kSampleBatch; ++j)
      g[j] = half[j] < -FLT_MAX ? 0 : order_bits(half[j]) >> 16;
    least_bits = job.kth(g, target);
    if (share) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      if (lane == 0) sh.mine[warp].x = most;
      __syncthreads();
      for (int w = 0; w < kSampleWarps; ++w) most = fmaxf(most, sh.mine[w].x);
      scaled = mass_scale(s0, most >= -FLT_MAX && most <= FLT_MAX ? most : 0.0f, sh.inv, p.unit_bits);
    }
  }
  // (An entry of -inf has no mass, and is -inf in the result too.)
  float least = fmaxf(from_order_bits(least_bits << 16), -FLT_MAX);
  if (listing && tid < edges) {
    if (edge >= least) job.append(edge, job.edge(tid));
    if (share) (edge >= least ? listed_sum : sum.hi) = near_mass(s0, edge);
  }
  for (int i0 = 0; i0 < nvec; i0 += kStep) {
    uint4 v[kSampleBatch];
#pragma unroll
    for (int j = 0; j < kSampleBatch; ++j) v[j] = next[j];
    if (i0 + kStep < nvec) load(i0 + kStep);
#pragma unroll
    for (int j = 0; j < kSampleBatch; ++j) {
      const int i = i0 + j * kSampleThreads + tid;
      if (i >= nvec) break;
      float x[kPer];
      Tr::unpack(v[j], x);
      float most = x[0];
#pragma unroll
      for (int e = 1; e < kPer; ++e) most = fmaxf(most, x[e]);
      if constexpr (sizeof(TIn) == 2) {
        nan = __uint_as_float(nan_of(v[j], __float_as_uint(nan)));
      } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e) nan = x[e] != x[e] ? x[e] : nan;
      }
      if (most > top) {
        top = most;
        top_vec = i;
      }
      if (listing && most >= least) {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (x[e] >= least) {
            job.append(x[e], job.first + i * kPer + e);
            if (share) listed_sum = __fadd_rn(listed_sum, near_mass(s0, x[e]));
          }
      }
      if (share) {
        float part[2] = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          part[e & 1] = __fadd_rn(part[e & 1], near_mass(s0, x[e] >= least ? -INFINITY : x[e]));
        sum = ff_add_f(sum, __fadd_rn(part[0], part[1]));
      }
    }
  }
  if constexpr (sizeof(TIn) == 2) {
    const float other = __uint_as_float(__float_as_uint(nan) << 16);
    nan = other != other ? other : nan;
  }
  const float vec_top = top;
  top = fmaxf(top, edge);
  bad |= !greedy && (nan != nan || top > FLT_MAX);
  bad = __syncthreads_or(bad);
  if (listing && !bad) {
    // A long list is cut before it is sorted.
    overflow = sh.count > kSampleList;
    if (few && !overflow && sh.count > kSampleLong) least_bits = ::max(least_bits, job.list_kth(st.top_k));
  }

  // What the CTAs have found.
  SamplePeer word = {};
  {
    unsigned long long best = 0;
    if (greedy && top >= -FLT_MAX) {
      // The lowest index of the thread's largest.
      if (tid < edges && edge == top) best = entry_rank(edge, job.edge(tid));
      if (top_vec >= 0 && vec_top == top) {
        float x[kPer];
        Tr::unpack(job.run[top_vec], x);
#pragma unroll
        for (int e = kPer - 1; e >= 0; --e)
          if (x[e] == top) {
            const unsigned long long rk = entry_rank(top, job.first + top_vec * kPer + e);
            best = rk > best ? rk : best;
          }
      }
    }
    if (greedy) best = warp_max_u64(best);
    float m = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (share) {
      sum = warp_sum_ff(sum);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) listed_sum += __shfl_xor_sync(0xffffffffu, listed_sum, o);
    }
    __syncthreads();
    if (lane == 0) {
      sh.mine[warp].x = m;
      sh.mine[warp].y = listed_sum;
      sh.mine[warp].a = best;
      sh.mine[warp].b = ((unsigned long long)__float_as_uint(sum.lo) << 32) | __float_as_uint(sum.hi);
    }
    __syncthreads();
    if (tid == 0) {
      word.x = -INFINITY;
      FF all = {0.0f, 0.0f};
      for (int w = 0; w < kSampleWarps; ++w) {
        const SamplePeer q = sh.mine[w];
        word.x = fmaxf(word.x, q.x);
        word.a = q.a > word.a ? q.a : word.a;
        if (share) {
          if (w > 0) listed_sum += q.y;
          all = ff_add(all, {__uint_as_float((uint32_t)q.b), __uint_as_float((uint32_t)(q.b >> 32))});
        }
      }
      sum = all;
      word.b = least_bits;
      word.i = bad;
      word.j = overflow;
    }
  }
  if (ctas > 1) cluster_wait();
  const SamplePeer* all = job.exchange(word);
  float most = -INFINITY;
  unsigned long long limit = 0;
  overflow = false;
  for (int i = 0; i < ctas; ++i) {
    most = fmaxf(most, all[i].x);
    bad |= all[i].i != 0;
    overflow |= all[i].j != 0;
    least_bits = ::max(least_bits, (uint32_t)all[i].b);
    if (greedy) limit = all[i].a > limit ? all[i].a : limit;
  }
  bad |= !(most >= -FLT_MAX);
  scaled &= mass_scale(job.s, most, sh.inv, p.unit_bits);
  // The mass of what is not listed, between `rest_lo` and `rest_hi` units; about that of the
  // row, next to the largest entry's (0: not known).
  unsigned long long rest_lo = 0, rest_hi = 0;
  float about = 0.0f;
  bool known = false;
  if (share && !bad) {
    SamplePeer w = {};
    if (tid == 0) {
      const double shift = exp2(((double)s0.max - (double)most) *
                                    ((double)sh.inv.hi + (double)sh.inv.lo) + (double)p.unit_bits);
      const double rest = ((double)sum.hi + (double)sum.lo) * shift;
      const bool fits = rest < 9.2e18 && scaled;
      w.a = fits ? (unsigned long long)rest : 0;
      w.i = fits;
      w.x = (float)((rest + (double)listed_sum * shift) * exp2(-(double)p.unit_bits));
    }
    all = job.exchange(w);
    known = true;
    unsigned long long rest = 0;
    for (int i = 0; i < ctas; ++i) {
      rest += all[i].a;
      about += all[i].x;
      known = known && all[i].i != 0;
    }
    // (near_mass is off by 2^-16 of itself; V: whole units, what is below `floor`, and sums.)
    rest_lo = rest - min(rest, (rest >> 15) + V);
    rest_hi = rest + (rest >> 15) + V;
    if (!known || !(about <= FLT_MAX)) about = 0.0f;
  }

  int token = -1;
  int listed = -1;  // entries of K in the first CTA's list, if it has all of K
  const bool want_kept = p.kept != nullptr, want_token = p.tokens != nullptr;
  float u = want_token ? p.uniforms[r] : 0.0f;
  const bool u_ok = u >= 0.0f && u < 1.0f;
  if (!u_ok) u = 0.0f;
  if (bad) {
  } else if (greedy) {
    token = (int)~(uint32_t)limit;
    if (tid == 0) sh.list[0] = limit;
    listed = 1;
  } else {
    unsigned long long min_rank = 0;
    if (st.min_p > 0.0f)
      min_rank = (unsigned long long)order_bits(__double2float_ru((double)most + sh.min_off)) << 32;
    bool done = false;
    if (listing && !overflow && (few || known)) {
      if (few && (sh.count > kSampleLong || ctas > 1)) job.cut_list(least_bits);
      const int n = job.gather();
      bool enough = true;  // of a share's mass, to hold the border
      unsigned long long want_lo = 0, want_hi = 0;
      if (n >= 0 && rank == 0 && share) {
        unsigned long long m = 0;
        for (int i = tid; i < n; i += kSampleThreads)
          m += entry_mass(job.s, sh.table, from_order_bits((uint32_t)(sh.list[i] >> 32)));
        m = job.block_sums(0, m).mass;
        want_lo = mass_part(st.top_p, m + rest_lo, true);
        want_hi = mass_part(st.top_p, m + rest_hi, true);
        enough = m >= want_hi;
      }
      if (few && n < min(st.top_k, V) && !(n >= 0 && least_bits == 0)) enough = false;
      if (n >= 0 && rank == 0 && enough) {
        job.sort(n);
        job.list_masses(n);
        int kept = min(n, st.top_k);
        if (share) {
          // (The CTAs' lists have all entries from the largest of their bounds on.)
          const int i = first_reaching(sh.mass, n, want_lo);
          kept = i < n && sh.mass[i] >= want_hi && (uint32_t)(sh.list[i] >> 48) >= least_bits ? i + 1 : 0;
        }
        if (few && cut_p) {
          const unsigned long long part = mass_part(st.top_p, sh.mass[kept - 1], true);
          kept = min(first_reaching(sh.mass, kept, part) + 1, kept);
        }
        if (kept > 0) {
          if (min_rank > 0) {
            int lo = 0, hi = kept;  // entries of min_rank and more
            while (lo < hi) {
              const int mid = (lo + hi) >> 1;
              if (sh.list[mid] >= min_rank) lo = mid + 1;
              else hi = mid;
            }
            kept = lo;
          }
          done = true;
          listed = kept;
          limit = sh.list[kept - 1];
        }
        if (done && want_token && u_ok) {
          const unsigned long long level = mass_part(u, sh.mass[kept - 1], false);
          token = job.draw_listed(kept, level);
        }
      }
      if (n >= 0 && ctas > 1 && (share || want_kept)) {
        SamplePeer w = {};
        w.a = limit;
        w.i = done;
        all = job.exchange(w);
        limit = all[0].a;
        done = all[0].i != 0;
      } else if (few) {
        done = n >= 0 && enough;
      }
    }
    if (!done) {
      const uint32_t top_bits = order_bits(most);
      if (cut_k) limit = job.border_rank({true, (unsigned long long)st.top_k, 0.0f}, 0, 0, top_bits);
      if (cut_p) {
        // The border is among the entries whose mass is at least their share of what may be
        // left out; where about, a histogram of the distances from the maximum shows.
        uint32_t lo = (uint32_t)(limit >> 32), hi = top_bits;
        unsigned long long found = 0;
        const float range = logf((float)V / ((1.0f - st.top_p) * about)) + 0.001f;
        const float per = __fmul_rn(__fmul_rn(job.s.inv.hi, kLn2f), (float)kSampleBins / range);
        if (about > 0.0f && range > 0.0f && per > 0.0f && per <= FLT_MAX) {
          __syncthreads();
          for (int i = tid; i < kSampleBins; i += kSampleThreads) sh.hist[i] = 0;
          __syncthreads();
          job.each(most - (float)kSampleBins / per * 1.0001f, [&](const float* x, int v, int k) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const float f = __fmul_rn(__fsub_rn(most, x[e]), per);
              if ((e < k) & (f >= 0.0f) & (f < (float)kSampleBins)) atomicAdd(&sh.hist[(int)f], 1u);
            }
          });
          job.sync_all();
          SamplePeer w = {};
          if (rank == 0) {
            // The masses of the bins, taken at their middles, up to what is wanted.
            constexpr int kEach = kSampleBins / kSampleThreads;
            // (Lanes next to each other for the loads from other CTAs: 32 bytes apart they took
            // 16 us.)
            if (ctas > 1) {
#pragma unroll
              for (int e = 0; e < kEach; ++e) {
                const int b = e * kSampleThreads + tid;
                sh.hist[b] = job.sum_of(&sh.hist[b]);
              }
              __syncthreads();
            }
            const float width = range / (float)kSampleBins;
            float mine = 0.0f, squares = 0.0f, bin[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
              const int b = tid * kEach + e;
              const uint32_t c = sh.hist[b];
              bin[e] = (float)c * ex2(__fmul_rn(-((float)b + 0.5f) * width, kLog2e));
              mine += bin[e];
              squares = fmaf(bin[e], bin[e], squares);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) squares += __shfl_xor_sync(0xffffffffu, squares, o);
            float upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const float x = __shfl_up_sync(0xffffffffu, upto, o);
              if (lane >= o) upto += x;
            }
            if (tid == 0) sh.border = sh.rest = kSampleBins - 1;
            if (lane == 31) {
              sh.mine[warp].x = upto;
              sh.mine[warp].y = squares;
            }
            __syncthreads();
            float below = upto - mine;
            squares = 0.0f;
            for (int q = 0; q < kSampleWarps; ++q) {
              if (q < warp) below += sh.mine[q].x;
              squares += sh.mine[q].y;
            }
            // A bin's entries are off its middle by up to half a width, all alike at worst: four
            // standard deviations of that.
            const float slack = 1.2f * width * sqrtf(squares);
            const float goal = st.top_p * about;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
              const float upper = below + bin[e];
              if (below < goal - slack && upper >= goal - slack)
                atomicMin(&sh.border, tid * kEach + e);
              if (below < goal + slack && upper >= goal + slack)
                atomicMin(&sh.rest, tid * kEach + e);
              below = upper;
            }
            if (tid == 0 && goal - slack <= 0.0f) sh.border = 0;
            __syncthreads();
            w.i = ::max(sh.border - 1, 0);
            w.j = sh.rest + 2;
          }
          const SamplePeer* bins = job.exchange(w);
          // (Where exactly the places of the bins' ends lie does not matter.)
          const float z_lo = fmaxf(most - (float)bins[0].j / per, -FLT_MAX);
          const float z_hi = bins[0].i == 0 ? INFINITY : most - (float)bins[0].i / per;
          // bfloat16: the entries between are counted by their bits, of which there are few (a
          // flat row may have thousands of the same).
          const uint32_t k0 = order_bits(z_lo) >> 16, k1 = order_bits(fminf(z_hi, most)) >> 16;
          if (!job.s.quick) {
          } else if (sizeof(TIn) == 2 && k1 - k0 < (uint32_t)kSampleFine) {
            __syncthreads();
            for (int i = tid; i < kSampleFine; i += kSampleThreads) sh.hist[i] = 0;
            __syncthreads();
            unsigned long long all_mass = 0, mass = 0;  // (above the keys)
            job.each(-INFINITY, [&](const float* x, int v, int k) {
#pragma unroll
              for (int e = 0; e < kPer; ++e) {
                const uint32_t key = order_bits(x[e]) >> 16;
                const unsigned long long m = quick_mass(job.s, sh.quick.e, x[e]);
                all_mass += e < k ? m : 0;
                mass += (e < k) & (key > k1) ? m : 0;
                if ((e < k) & (key >= k0) & (key <= k1)) atomicAdd(&sh.hist[key - k0], 1u);
              }
            });
            const CountMass sums = job.cluster_sums(all_mass, mass);
            const unsigned long long above = sums.mass, doubt = quick_doubt(sums.count, V);
            const unsigned long long want = mass_part(st.top_p, sums.count, true);
            // Thread t has two keys, from the top down.
            SamplePeer w2 = {};
            if (rank == 0) {
              constexpr int kEach = kSampleFine / kSampleThreads;
              unsigned long long m[kEach], mine = 0;
              uint32_t c[kEach];
#pragma unroll
              for (int e = 0; e < kEach; ++e) {
                const int b = (int)(k1 - k0) - (tid * kEach + e);
                c[e] = 0;
                m[e] = 0;
                if (b >= 0) {
                  c[e] = job.sum_of(&sh.hist[b]);
                  const uint32_t key = k0 + b;
                  m[e] = entry_mass(job.s, sh.table, job.key_value(key));
                }
                mine += c[e] * m[e];
              }
              unsigned long long upto = mine;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
              }
              if (lane == 31) sh.red[0][warp] = upto;
              if (tid == 0) sh.border = -1;
              __syncthreads();
              unsigned long long less = above + upto - mine;
              for (int q = 0; q < warp; ++q) less += sh.red[0][q];
#pragma unroll
              for (int e = 0; e < kEach; ++e) {
                if (less < want && less + c[e] * m[e] >= want) {
                  const unsigned long long nth = (want - less + m[e] - 1) / m[e];
                  const unsigned long long over = less + nth * m[e];
                  if (over - want > doubt && want - (over - m[e]) > doubt) {
                    sh.border = (int)(k1 - k0) - (tid * kEach + e);
                    sh.red[1][0] = nth;
                    sh.rest = nth == c[e];
                  }
                }
                less += c[e] * m[e];
              }
              __syncthreads();
              w2.i = sh.border;
              w2.a = sh.border >= 0 ? sh.red[1][0] : 0;
              w2.j = sh.border >= 0 ? sh.rest : 0;
            }
            const SamplePeer* got = job.exchange(w2);
            const int bin = got[0].i, whole = got[0].j;
            const unsigned long long nth = got[0].a;
            if (bin >= 0) {
              const uint32_t key = k0 + bin;
              const float z = job.key_value(key);
              // The lowest indices of those equal to the last.
              found = whole ? (unsigned long long)order_bits(z) << 32
                            : entry_rank(z, job.locate(
                                                z,
                                                [&](float y, int) -> unsigned long long {
                                                  return order_bits(y) >> 16 == key ? 1 : 0;
                                                },
                                                [&](unsigned long long) { return nth - 1; },
                                                [](unsigned long long) { return 0ull; }));
            }
          } else {
          // What is above those bins, and their entries one by one.
          __syncthreads();
          if (tid == 0) sh.count = 0;
          __syncthreads();
          unsigned long long all_mass = 0, mass = 0;  // (above the bins)
          job.each(-INFINITY, [&](const float* x, int v, int k) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
              const unsigned long long m = quick_mass(job.s, sh.quick.e, x[e]);
              all_mass += e < k ? m : 0;
              mass += (e < k) & (x[e] > z_hi) ? m : 0;
              if ((e < k) & (x[e] >= z_lo) & (x[e] <= z_hi)) job.append(x[e], v + e);
            }
          });
          const CountMass sums = job.cluster_sums(all_mass, mass);
          const unsigned long long above = sums.mass, doubt = quick_doubt(sums.count, V);
          const unsigned long long want = mass_part(st.top_p, sums.count, true);
          const int n = job.gather();
          SamplePeer w2 = {};
          if (rank == 0 && n > 0) {
            job.sort(n);
            job.list_masses(n);
            const int i = want > above ? first_reaching(sh.mass, n, want - above) : n;
            if (i < n) {
              const unsigned long long less = above + (i > 0 ? sh.mass[i - 1] : 0);
              if (above + sh.mass[i] - want > doubt && want - less > doubt) w2.a = sh.list[i];
            }
          }
          found = job.exchange(w2)[0].a;
          }
          lo = order_bits(z_lo);
          hi = order_bits(fminf(z_hi, most));
        }
        if (found == 0) found = job.border_rank({false, 0, st.top_p}, limit, lo, hi);
        limit = found > limit ? found : limit;
      }
      limit = min_rank > limit ? min_rank : limit;
      if (want_token) {
        // (z itself decides but for the entries equal to the last one kept.)
        const float z_least = limit > 0 ? from_order_bits((uint32_t)(limit >> 32)) : -INFINITY;
        const uint32_t last = ~(uint32_t)limit;
        auto drawn = [&](float z, int v) -> bool {
          return (z > z_least) | ((z == z_least) & ((uint32_t)v <= last));
        };
        auto level = [&](unsigned long long total) { return mass_part(u, total, false); };
        // Quick masses tell the token, but for one draw in some hundred over a flat row.
        if (job.s.quick)
          token = job.locate(
              z_least,
              [&](float z, int v) -> unsigned long long {
                const unsigned long long m = quick_mass(job.s, sh.quick.e, z);
                return drawn(z, v) ? m : 0;
              },
              level, [&](unsigned long long total) { return quick_doubt(total, V); });
        if (token < 0) token = exact_draw<TIn>(job, z_least, last, u);  // (the last exchange)
      }
    }
    if (!u_ok) token = -1;
  }
  if (want_token && rank == 0 && tid == 0) p.tokens[r] = token;
  if (!want_kept) return;
  TIn* out = static_cast<TIn*>(p.kept) + (size_t)r * V;
  TIn none, off;
  if constexpr (sizeof(TIn) == 4) {
    none = __int_as_float(0x7fc00000);
    off = -INFINITY;
  } else {
    none = 0x7fc0;
    off = 0xff80;
  }
  __syncthreads();  // (in place: nobody reads the row any more)
  const bool lines = reinterpret_cast<uintptr_t>(out + job.first) % 16 == 0;
  if (lines && (bad || (listed >= 0 && (ctas == 1 || greedy)))) {
    // All of K is in the list: the row is not read again, but for those entries.
    const TIn all_over = bad ? none : off;
    uint32_t two;
    if constexpr (sizeof(TIn) == 4) two = __float_as_uint(all_over);
    else two = (uint32_t)all_over * 0x10001u;
    constexpr int kEach = kSampleList / kSampleThreads;
    TIn keep[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = tid + e * kSampleThreads;
      if (i < listed) keep[e] = job.row[(int)~(uint32_t)sh.list[i]];
    }
    if (ctas > 1) job.sync_all();  // (in place: the one entry is read by all)
    else __syncthreads();
    uint4* dst = reinterpret_cast<uint4*>(out + job.first);
    for (int i = tid; i < nvec; i += kSampleThreads) dst[i] = make_uint4(two, two, two, two);
    if (tid < edges) out[job.edge(tid)] = all_over;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = tid + e * kSampleThreads;
      if (i >= listed) break;
      const int v = (int)~(uint32_t)sh.list[i];
      const bool mine = v >= job.first - job.head && v < job.first + nvec * kPer + job.tail;
      if (mine) out[SPEC_CHECKED(v, V, kSiteSample)] = keep[e];
    }
    return;
  }
  auto result = [&](TIn x, int v) -> TIn {
    const float z = Tr::to_float(x);
    return bad ? none : z == z && entry_rank(z, v) >= limit ? x : off;
  };
  for (int i = tid; i < nvec; i += kSampleThreads) {
    const uint4 v = job.run[i];
    TIn x[kPer];
    *reinterpret_cast<uint4*>(x) = v;
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = result(x[e], job.first + i * kPer + e);
    if (lines) {
      *reinterpret_cast<uint4*>(out + job.first + i * kPer) = *reinterpret_cast<uint4*>(x);
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) out[job.first + i * kPer + e] = x[e];
    }
  }
  if (tid < edges) {
    const int v = job.edge(tid);
    out[v] = result(job.row[v], v);
  }
}

}  // namespace specv
