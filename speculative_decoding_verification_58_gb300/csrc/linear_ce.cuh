// Softmax cross entropy of a linear vocabulary head, and its gradients, without
// keeping the logits.
//
//   z_iv  = h_i . w_v          lse_i = log sum_v exp z_iv
//   nll_i = lse_i - z_{i,y_i}
//   dZ_iv = g_i (exp(z_iv - lse_i) - [v = y_i]),  dH = dZ W,  dW = dZ^T H
//
// The loss forms the logits tile by tile and keeps of each tile one (max, sum)
// pair per row.  The gradients form them again, a piece of the vocabulary at a
// time: the piece's dZ is written in bfloat16 to the workspace, and both products read
// it from there.  dZ is rounded to bfloat16 (relative
// 2^-8) because the matrix units take both operands in one type, and the
// gradients come out in bfloat16 anyway; every sum is in single precision.  The
// label's entry, which is the largest of most rows and would pass its own rounding
// on to a whole row of dW and dH, is made good: what the rounding took from it is
// kept per token and added to both in single precision.  The other entries' roundings
// stay: at most 2^-8 of their share of a row.
//
// Measured (V = 151936): loss of 2048 tokens, D = 2048, 727 to 746 us on several boxes
// (1.71 to 1.75 PFLOP/s); loss and gradients of 2048 tokens, D = 4096, 5.9 to 6.1 ms and of
// 512 tokens, D = 2048, 0.91 to 0.95 ms (1.7 and 1.37 PFLOP/s, the logits formed twice).
// Bound by the tensor cores (88 to 94 % of their cycles) where there are many tokens, by
// dW's epilogue and stores at 512, by reading W at a few (loss of one token, D = 1024:
// 60 us, 5.2 TB/s).
#pragma once

#include "grad_norm.cuh"
#include "opd_grad.cuh"
#include "tcgen05.cuh"

namespace specv {

constexpr int kCeTileV = 256;      // vocabulary entries per tile of the products
constexpr int kCePartV = 128;      // and per (max, sum) pair
constexpr int kCePieceBytes = 160 << 20;  // most bytes of a piece's dZ
constexpr int kCeMaxTokens = SPEC_MAX_TOKENS;
constexpr int kCeMaxWidth = SPEC_MAX_WIDTH;
constexpr int kCeFixes = 4;  // tokens of a label that a tile of dW adds one by one

struct CeLayout {
  size_t partials, resid, in_rows, dz, dh_acc, label_sums, total;
  int tiles;   // vocabulary tiles
  int parts;   // (max, sum) pairs of a token
  int piece;   // vocabulary entries per piece (a multiple of kCeTileV)
  int splits;  // slices of a piece whose parts of dH are summed apart
  bool direct;  // dH comes out of one tile whole: no sums to keep
};

constexpr int kCePairs = 76;  // CTA pairs the sizes below are chosen for (152 SMs)

inline long long ce_waves(long long tiles) { return (tiles + kCePairs - 1) / kCePairs; }

// Vocabulary tiles per piece of the gradients: of those whose dZ fits, the number
// that needs the fewest rounds of 76 tiles in all, a round's tenth counted for each
// piece's launches.  Few large pieces: every piece ends with a round that is not full
// (512 tokens, V = 151936, D = 2048: gradients in 694 us as one piece, in 766 us as
// four of 48 MB whose dZ stays in L2; 2048 tokens, D = 4096: 4.60 ms as four pieces,
// 4.90 ms as sixteen).
inline int ce_piece_tiles(int N, int tiles) {
  const long long mb = (N + 255) / 256;
  const int most = (int)std::max<long long>(
      1, std::min<long long>(tiles, kCePieceBytes / 2 / N / kCeTileV));
  int best = most;
  long long cost = -1;
  for (int n = most; n >= std::max({1, most / 2, most - 256}); --n) {
    const int pieces = (tiles + n - 1) / n, last = tiles - (pieces - 1) * n;
    const long long c =
        10 * ((pieces - 1) * ce_waves(mb * n) + ce_waves(mb * last)) + pieces;
    if (cost < 0 || c < cost) {
      cost = c;
      best = n;
    }
  }
  return best;
}

// Slices of the piece's entries that dH = dZ W is summed over: the fewest that
// fill nine tenths of the pairs' rounds with 256 x 256 tiles of dH, or else those
// that fill them best; none shorter than 16 steps of 64 entries.  The same whether
// dW is wanted too (its units would even out less), so that dH is.
inline int ce_splits(int N, int D, int piece) {
  const long long tiles = (long long)((N + 255) / 256) * ((D + 255) / 256);
  const int most = (int)std::max<long long>(
      1, std::min<long long>((4 * kCePairs + tiles - 1) / tiles, piece / (16 * 64)));
  int best = 1;
  double fill = 0.0;
  for (int n = 1; n <= most && fill < 0.9; ++n) {
    const double f = (double)(tiles * n) / (double)(ce_waves(tiles * n) * kCePairs);
    if (f > fill + 0.02) {
      fill = f;
      best = n;
    }
  }
  return best;
}

inline CeLayout ce_layout(int N, int V, int D, bool grad) {
  CeLayout l = {};
  l.tiles = (V + kCeTileV - 1) / kCeTileV;
  l.parts = (V + kCePartV - 1) / kCePartV;
  l.piece = grad ? ce_piece_tiles(N, l.tiles) * kCeTileV : 0;
  size_t o = align256(sizeof(WsHeader));
  if (!grad) {
    l.partials = o;
    o = align256(o + (size_t)N * l.parts * sizeof(float2));
  } else {
    l.resid = o;
    o = align256(o + (size_t)N * sizeof(float));
    l.in_rows = o;
    o = align256(o + (size_t)(l.piece / 32) * ((N + 31) / 32) * sizeof(uint32_t));
    l.dz = o;
    o = align256(o + (size_t)N * l.piece * 2);
    l.splits = ce_splits(N, D, l.piece);
    l.direct = l.splits == 1 && l.piece >= V;
    l.dh_acc = o;
    if (!l.direct) o = align256(o + (size_t)l.splits * N * D * sizeof(float));
    l.label_sums = o;
    if (N > kCeFixes) o = align256(o + (size_t)N * D * sizeof(float));
  }
  l.total = o;
  return l;
}

// Units of dH and dW over the pairs.  A unit of dH costs split_iters steps, one of
// dW as many as the tokens need, each some more for its epilogue.  The units of dH
// go round, so that the first `more` pairs have one more of them; dW's are dealt to
// bring every pair up to the same level (w1 to each of the first `more` pairs, w0 to
// each of the others), and those that are left go round.  Worked out on the host.
struct CeDeal {
  int h, more;  // dH units of every pair, pairs with one more
  int w0, w1;   // dW units under the level
};
constexpr int kCeEpilogueSteps = 6;  // an epilogue's time, in steps
inline CeDeal ce_deal(int dh_units, int dw_units, int dh_iters, int dw_iters, int G) {
  CeDeal d;
  d.h = dh_units / G;
  d.more = dh_units % G;
  const int less = G - d.more;
  const long long ch = dh_iters + kCeEpilogueSteps, cw = dw_iters + kCeEpilogueSteps;
  const long long level = ((long long)dh_units * ch + (long long)dw_units * cw) / G;
  const long long w0 = level > d.h * ch ? (level - d.h * ch) / cw : 0;
  d.w0 = (int)std::min<long long>(w0, dw_units / less);
  const long long w1 = d.more > 0 && level > (d.h + 1) * ch ? (level - (d.h + 1) * ch) / cw : 0;
  d.w1 = d.more > 0
             ? (int)std::min<long long>(w1, (dw_units - (long long)d.w0 * less) / d.more)
             : 0;
  return d;
}
// Pair c's i-th unit, dH's first, then dh_units + dW's; -1: no more.
__host__ __device__ inline int ce_unit(const CeDeal& d, int dh_units, int dw_units, int G, int c,
                                       int i) {
  const bool first = c < d.more;
  const int mine = d.h + (first ? 1 : 0), less = G - d.more;
  if (i < mine) return i * G + c;
  int j = i - mine;
  const int w = first ? d.w1 : d.w0;
  if (j < w) return dh_units + (first ? d.w0 * less + j * d.more + c : j * less + (c - d.more));
  j -= w;
  const long long idx = (long long)d.w0 * less + (long long)d.w1 * d.more + (long long)j * G +
                        (G - 1 - c);
  return idx < dw_units ? dh_units + (int)idx : -1;
}

struct CeParams {
  const int32_t* labels;   // [N]
  const float* nll;        // [N] (gradients)
  const float* lse;        // [N] (gradients)
  const float* g;          // [N] (gradients)
  int N, V, D, parts;
  float2* partials;        // [parts, N]: (max log2 e, sum 2^(z log2 e - max log2 e))
  int piece, v0, nv;       // piece: buffer width, first entry, entries
  const uint16_t* h;       // [N, D]
  const uint16_t* w;       // [V, D]
  float* resid;            // [N]: the label's entry of dZ less its bf16 rounding
  uint32_t* in_rows;       // [piece / 32, N / 32]: tokens whose label is one of 32 entries
  float* dh_acc;           // [splits, N, D]
  float* label_sums;       // [N, D]: row i for the label whose (kCeFixes + 1)-th token is i
  int dh_direct;           // dH comes out of one tile whole
  int first;               // first piece: dh_acc is set, not added to
  int splits, split_iters;  // slices of the piece in dH, 64-entry steps of a slice
  int z_tiles, m_blocks;   // tiles of z, of which so many are one vocabulary tile's
  int dh_units, dw_units;  // units of the two products (0: not wanted)
  CeDeal deal;             // and how the pairs share them
  int group;               // loss: rows of the product that the tokens take (32: one each)
  int a_rows;              // rows of A in a box (fewer than 128 where there are fewer tokens)
  int check;               // CTA 0 checks labels and lse and writes the header (one kernel a call)
  WsHeader* header;
};

// ---------------------------------------------------------------------------
// The products.  A persistent kernel of CTA pairs, one CTA per SM, on tiles of
// 256 x 256 (rows 0..127 of a tile are the first CTA's): in each CTA a warp that
// issues the TMA loads into a ring of six 64-deep stages and eight warps that take
// finished tiles out of tensor memory (half a row each thread), in the first a warp
// that issues the tcgen05.mma for both.  Two accumulators of 256 columns alternate, so that one
// tile's epilogue runs under the next one's products.  A pair's CTAs each load one
// half of either operand, 32 KB for the products of a stage; single CTAs on
// 128 x 256 tiles need 48 KB for as many, which the L2 did not deliver where
// operands are MN-major (dW of 2048 tokens at 58 % of the tensor cores' cycles;
// without the loads of one operand they ran at full rate).
//   loss   z  = H W^T          both operands K-major
//   dz     z  = H W^T          the piece's columns
//   grads  dH = dZ W           A K-major, B MN-major  (K: the piece's entries)
//          dW = dZ^T H         A and B MN-major       (K: the tokens)
// ---------------------------------------------------------------------------
enum CeMode { kCeLoss, kCeDz, kCeGrads };

constexpr int kMmM = 256, kMmN = 256, kMmK = 64, kMmStages = 6;
// The loss sums a logit in chunks of kMmChunk steps, each from zero in an accumulator of
// its own, and adds the chunks in registers, rounded to nearest: the tensor cores'
// sums are cut off towards zero at every step, which over a long row is a bias (loss
// of 2048 tokens, D = 2048: off by 1.1e-6 of itself in one chunk, 5e-7 in chunks of 16
// steps; of 8 or 4 half and a fourth of that, but 772 and 881 us instead of 739).
constexpr int kMmChunk = 16;
// Up to kCeFewTokens tokens leave rows of the product unused.  `group` of them (a power of
// two) take one part of the sum over D, the next `group` rows the next part, and so on
// over 32 rows: the hidden states are loaded that many rows lower, with zeros around
// them, and a zero is added without a cut.  One token's logits so are sums of 32 parts,
// joined in the epilogue (D = 1024, V = 151936: worst error of the loss of one token in
// 24 4e-6 of itself, 8e-7 in parts; 60.9 us, 58.7 without; chunks of four steps
// instead: 72).
constexpr int kCeFewTokens = 16;
// dW sums over the tokens and dH over a slice of the vocabulary; so long a sum of one sign
// that the cuts would show beside the result's own rounding (up to 2^-8) is summed in
// chunks as well (262144 tokens in one: short by 4.8e-4 of itself; 65536: 7e-5).
constexpr int kMmGradChunk = 1024;
constexpr int kMmHalf = 128;  // rows of A, of B and of the result in each CTA
constexpr int kMmABytes = kMmHalf * kMmK * 2, kMmBBytes = kMmHalf * kMmK * 2;
constexpr int kMmStageBytes = kMmABytes + kMmBBytes;  // each CTA's
constexpr int kMmThreads = 320;
constexpr int kMmProducer = 0, kMmIssuer = 1, kMmEpilogue = 2;  // first warps of the roles
// Results leave through kMmBoxes boxes of 32 rows x 128 bytes for each epilogue warp.
constexpr int kMmBoxes = 1;
constexpr int kMmBoxBytes = 32 * 128, kMmOutBytes = 8 * kMmBoxes * kMmBoxBytes;
constexpr int kMmSmem = kMmStages * kMmStageBytes + kMmOutBytes + 1024;  // + alignment

struct CeMaps {
  CUtensorMap h_k, w_k, dz_k;      // boxes of 64 x 128: rows of hidden, weight, dZ
  CUtensorMap h_mn, w_mn, dz_mn;   // 64 x 64
  CUtensorMap dz_out, dh_out, dw_out;  // 64 x 32: stores of bf16 results
  CUtensorMap acc;                     // 32 x 32 x 1: sums of dH, [splits, N, D] floats
};

struct CeBars {
  uint64_t full[kMmStages], empty[kMmStages], tfull[2], tempty[2];
  uint32_t tmem;
  int abort_flag;
  int bad;   // labels outside the vocabulary
  int lost;  // tokens whose loss timed out (gradients)
};

struct CeTile {
  int kind;  // 0: z, 1: dH, 2: dW
  int m0, n0;
  int k0, iters;  // first entry of the sum, steps of kMmK
  int slice;      // dH: which of the sums kept apart
};

// This pair's tiles: which is the i-th (kind -1: no more).
template <CeMode M>
__device__ __forceinline__ CeTile ce_tile(const CeParams& p, int i) {
  CeTile t;
  t.kind = -1;
  t.k0 = t.slice = 0;
  const int G = gridDim.x >> 1, c = blockIdx.x >> 1;
  if (M != kCeGrads) {
    // Token blocks fastest: a vocabulary tile is read once from memory, and by
    // the other token blocks from L2.
    const long long at = (long long)i * G + c;
    if (at >= p.z_tiles) return t;
    const uint32_t idx = (uint32_t)at, mb = (uint32_t)p.m_blocks;
    t.kind = 0;
    t.m0 = (int)(idx % mb) * kMmM;
    t.n0 = (int)(idx / mb) * kMmN;
    t.iters = (p.D + kMmK - 1) / kMmK;
  } else {
    const int idx = ce_unit(p.deal, p.dh_units, p.dw_units, G, c, i);
    if (idx < 0) return t;
    const uint32_t nb = (uint32_t)(p.D + kMmN - 1) / kMmN;
    uint32_t j = (uint32_t)idx;
    if (idx < p.dh_units) {
      // Token blocks fastest: those that share a part of W run together, and find it
      // in L2 (one after the other they read it from memory twice: 512 tokens).
      const uint32_t mb = (uint32_t)p.m_blocks;
      t.kind = 1;
      t.m0 = (int)(j % mb) * kMmM;
      j /= mb;
      t.n0 = (int)(j % nb) * kMmN;
      t.slice = (int)(j / nb);
      t.k0 = t.slice * p.split_iters * kMmK;
      t.iters = min(p.split_iters, max((p.nv - t.k0 + kMmK - 1) / kMmK, 0));
    } else {
      t.kind = 2;
      j -= (uint32_t)p.dh_units;
      t.iters = (p.N + kMmK - 1) / kMmK;
      t.m0 = (int)(j / nb) * kMmM;
      t.n0 = (int)(j % nb) * kMmN;
    }
  }
  return t;
}

// Epilogue of one thread: row `m` of the tile, one half of its columns in tensor memory.
// The label's logit is left out of the sums (ce_finish_kernel forms it itself).
__device__ __forceinline__ void ce_loss_row(const CeParams& p, const CeTile& t, uint32_t addr,
                                            int m, int half, const float (&sum)[kCePartV]) {
  const bool live = m < p.N;
  const int y = max(live ? p.labels[m] : -1, -1);
  const int from = half * kCePartV, cols = min(from + kCePartV, p.V - t.n0);
  // Below every logit: a tile of -inf keeps a finite maximum and a sum of 0.
  float ms = -FLT_MAX / 2, s = 0.0f;
#pragma unroll
  for (int q = 0; q < kCePartV; q += 32) {
    const int c0 = from + q;
    if (c0 >= cols) break;
    float x[32];
    tmem_load32(addr + c0, x);
#pragma unroll
    for (int c = 0; c < 32; ++c) x[c] = __fadd_rn(x[c], sum[q + c]);
    if (c0 + 32 > cols) {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c0 + c >= cols) x[c] = -INFINITY;
    }
    const int rel = y - t.n0 - c0;
    if (__any_sync(0xffffffffu, rel >= 0 && rel < 32)) {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        if (c == rel) x[c] = -INFINITY;
    }
    float mx = x[0];
#pragma unroll
    for (int c = 1; c < 32; ++c) mx = fmaxf(mx, x[c]);
    const float nms = fmaxf(ms, __fmul_rn(mx, kLog2e));
    float2 a[2] = {make_float2(__fmul_rn(s, ex2(__fsub_rn(ms, nms))), 0.0f),
                   make_float2(0.0f, 0.0f)};
    const float2 l2 = make_float2(kLog2e, kLog2e), mm = make_float2(-nms, -nms);
#pragma unroll
    for (int c = 0; c < 32; c += 2)
      a[(c >> 1) & 1] =
          f32x2_add(a[(c >> 1) & 1], ex2x2(f32x2_fma(make_float2(x[c], x[c + 1]), l2, mm)));
    const float2 r = f32x2_add(a[0], a[1]);
    s = __fadd_rn(r.x, r.y);
    ms = nms;
  }
  if (live && from < cols)
    p.partials[(size_t)(t.n0 / kCePartV + half) * p.N + m] = make_float2(ms, s);
}

// The same for a few tokens, whose logits' parts lie in the 32 rows of a warp: lane l
// has a part of token l mod group.  Each exchange adds the parts of two lanes and leaves
// either with half of the columns, so that in the end a lane has `group` of 32
// columns, whole.
__device__ __forceinline__ void ce_loss_few(const CeParams& p, const CeTile& t, uint32_t addr,
                                            int half, const float (&sum)[kCePartV]) {
  const int lane = threadIdx.x & 31, group = p.group;
  const int m = lane & (group - 1), first = lane & ~(group - 1);
  const int y = m < p.N ? p.labels[m] : -1;
  const int from = half * kCePartV, cols = min(from + kCePartV, p.V - t.n0);
  float ms = -FLT_MAX / 2, s = 0.0f;
#pragma unroll
  for (int q = 0; q < kCePartV; q += 32) {
    const int c0 = from + q;
    if (c0 >= cols) break;
    float x[32];
    tmem_load32(addr + c0, x);
#pragma unroll
    for (int c = 0; c < 32; ++c) x[c] = __fadd_rn(x[c], sum[q + c]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o < group) break;
      const bool up = lane & o;
#pragma unroll
      for (int c = 0; c < o; ++c) {
        const float mine = up ? x[c + o] : x[c], theirs = up ? x[c] : x[c + o];
        x[c] = __fadd_rn(mine, __shfl_xor_sync(0xffffffffu, theirs, o));
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int c = 0; c < kCeFewTokens; ++c) {
      const int col = c0 + first + c;
      if (c >= group || col >= cols || col == y - t.n0) x[c] = -INFINITY;
      mx = fmaxf(mx, x[c]);
    }
    const float nms = fmaxf(ms, __fmul_rn(mx, kLog2e));
    s = __fmul_rn(s, ex2(__fsub_rn(ms, nms)));
#pragma unroll
    for (int c = 0; c < kCeFewTokens; ++c)
      if (c < group) s = __fadd_rn(s, ex2(fmaf(x[c], kLog2e, -nms)));
    ms = nms;
  }
  for (int o = 16; o >= group; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, ms, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const float n = fmaxf(ms, m2);
    s = __fadd_rn(__fmul_rn(s, ex2(__fsub_rn(ms, n))), __fmul_rn(s2, ex2(__fsub_rn(m2, n))));
    ms = n;
  }
  if (lane < p.N && lane < group && from < cols)
    p.partials[(size_t)(t.n0 / kCePartV + half) * p.N + lane] = make_float2(ms, s);
}

// A warp's results go through shared memory: a box of 32 rows x 128 bytes, its
// 16-byte pieces swizzled as the tensor map has them (no two lanes of a store meet in a
// bank), then one TMA store.  Rows written by the lanes themselves, 16 bytes at a
// time, were half sectors each and took as long as the products (2 x 230 us of
// 1236 for 512 tokens, V = 151936, D = 2048).
struct CeOut {
  uint32_t base;  // the warp's boxes
  int n;          // boxes stored so far
};

__device__ __forceinline__ uint32_t ce_box_begin(CeOut& o) {
  if ((threadIdx.x & 31) == 0) bulk_wait_read<kMmBoxes - 1>();
  __syncwarp();
  return o.base + (o.n++ % kMmBoxes) * kMmBoxBytes;
}

// The lane's 16-byte piece `q` of its row.
__device__ __forceinline__ void ce_box_put(uint32_t box, int q, uint4 v) {
  const uint32_t lane = threadIdx.x & 31;
  st_shared16(box + lane * 128 + ((q ^ (lane & 7)) << 4), v);
}

__device__ __forceinline__ void ce_box_ready() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// The label's entry of dZ is g (exp(-nll) - 1): from the loss itself, because for a token
// that is well predicted the difference of its logit and lse has few bits left.
__device__ __forceinline__ float ce_label_entry(float nll, float g) {
  return __fmul_rn(expm1f(-nll), g);
}
// What rounding to bf16 takes from it.
__device__ __forceinline__ float ce_rounded_off(float x) {
  return __fsub_rn(x, __uint_as_float(pack_bf16(x, 0.0f) << 16));
}

// `sum`: what earlier chunks of the sums over D gave (kChunks).
template <bool kChunks>
__device__ __forceinline__ void ce_dz_tile(const CeParams& p, const CeMaps& maps, const CeTile& t,
                                           uint32_t addr, int row0, int half, CeOut& o,
                                           const float (&sum)[kCePartV]) {
  const int lane = threadIdx.x & 31, m = t.m0 + row0 + lane;
  int y = m < p.N ? p.labels[m] : -1;
  const bool has = y >= 0 && y < p.V;
  const float g = has ? p.g[m] : 0.0f;
  const float l2 = has ? __fmul_rn(p.lse[m], kLog2e) : 0.0f;
  y = has ? y - p.v0 - t.n0 : -1;
  const int from = half * 128, cols = min(from + 128, p.nv - t.n0);
  const float at_label = has && y >= 0 && y < kMmN ? ce_label_entry(p.nll[m], g) : 0.0f;
  // Which tokens have a label among each 32 entries of this warp's half.
  const int words = (p.N + 31) / 32;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t tokens = __ballot_sync(0xffffffffu, has && y >> 5 == from / 32 + k);
    if (lane == k && t.m0 + row0 < p.N)
      p.in_rows[(size_t)(t.n0 / 32 + from / 32 + k) * words + (t.m0 + row0) / 32] = tokens;
  }
  if (has && y >= from && y < from + 128)
    p.resid[m] = ce_rounded_off(at_label);
#pragma unroll
  for (int q0 = 0; q0 < kCePartV; q0 += 64) {
    const int c0 = from + q0;
    if (c0 >= cols) break;
    const uint32_t box = ce_box_begin(o);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[32];
      tmem_load32(addr + c0 + h * 32, x);
      const int rel = y - c0 - h * 32;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        if (kChunks) x[c] = __fadd_rn(x[c], sum[q0 + h * 32 + c]);
        const float d = has ? __fmul_rn(ex2(fmaf(x[c], kLog2e, -l2)), g) : 0.0f;
        x[c] = c == rel && has ? at_label : d;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) ce_box_put(box, h * 4 + q, pack_vec<uint16_t>(x + q * 8));
    }
    ce_box_ready();
    if (lane == 0 && t.m0 + row0 < p.N) {
      tma_store(&maps.dz_out, box, t.n0 + c0, t.m0 + row0);
      bulk_commit();
    }
  }
}

// 32 entries of a row of hidden or weight, of which `n` (a multiple of 8) exist.
struct CeRow {
  uint4 v[4];
};
__device__ __forceinline__ CeRow ce_row(const uint16_t* src, int n) {
  CeRow r;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    r.v[q] = q * 8 < n ? reinterpret_cast<const uint4*>(src)[q] : make_uint4(0, 0, 0, 0);
  return r;
}
__device__ __forceinline__ void ce_add_row(float (&x)[32], const CeRow& row, float r) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float a[8];
    ElemTraits<uint16_t>::unpack(row.v[q], a);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[q * 8 + e] = fmaf(r, a[e], x[q * 8 + e]);
  }
}

// Whose rounding residual a lane's row takes: of dH the row's own token's, of dW those
// of all tokens with this label.  Their roundings are not independent: under a mean loss
// every badly predicted token has -g there, rounded alike, and a frequent label's row
// would be off as a whole by up to 2^-8.  Up to kCeFixes tokens are kept here, in
// order (`src`: where the row to add starts); for a row with more, ce_label_kernel has
// summed all of them (`sum`).
struct CeFix {
  int toks;
  const uint16_t* src[kCeFixes];
  float r[kCeFixes];
  const float* sum;  // or null
};
// The first 32 words of the map of labels for a warp's 32 entries of dW, one per lane
// (read a tile ahead).
__device__ __forceinline__ uint32_t ce_fix_word(const CeParams& p, const CeTile& t, int row0) {
  const int lane = threadIdx.x & 31, words = (p.N + 31) / 32, r0 = t.m0 + row0;
  return t.kind == 2 && r0 < p.nv && lane < words ? p.in_rows[(size_t)(r0 / 32) * words + lane]
                                                  : 0;
}

__device__ __forceinline__ CeFix ce_fix(const CeParams& p, const CeTile& t, int row0,
                                        uint32_t word0) {
  const int lane = threadIdx.x & 31, r0 = t.m0 + row0;
  CeFix f;
  f.toks = 0;
  f.sum = nullptr;
  if (t.kind == 1) {
    // (Sums of several slices or pieces get theirs at the end.)
    const int y = p.dh_direct && r0 + lane < p.N ? p.labels[r0 + lane] : -1;
    if (y >= 0 && y < p.V) {
      f.toks = 1;
      f.src[0] = p.w + (size_t)y * p.D;
      f.r[0] = p.resid[r0 + lane];
    }
    return f;
  }
  if (r0 >= p.nv) return f;
  int tok[kCeFixes + 1];
#pragma unroll
  for (int k = 0; k <= kCeFixes; ++k) tok[k] = 0;
  const int words = (p.N + 31) / 32;
  const uint32_t* in_rows = p.in_rows + (size_t)(r0 / 32) * words;
  for (int base = 0; base < words; base += 32) {
    const uint32_t mine = base == 0               ? word0
                          : base + lane < words ? in_rows[base + lane]
                                                : 0;
    uint32_t some = __ballot_sync(0xffffffffu, mine != 0);
    while (some != 0) {
      // Up to four words with tokens at a time: their labels' loads go together.
      int first[4], rel[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        first[k] = some != 0 ? __ffs(some) - 1 : -1;
        some &= some - 1;
        const uint32_t word = __shfl_sync(0xffffffffu, mine, first[k] < 0 ? 0 : first[k]);
        const bool bit = first[k] >= 0 && ((word >> lane) & 1);
        rel[k] = bit ? p.labels[(base + first[k]) * 32 + lane] - p.v0 - r0 : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t m = __ballot_sync(0xffffffffu, rel[k] >= 0);
        for (; m != 0; m &= m - 1) {
          const int j = __ffs(m) - 1;
          if (__shfl_sync(0xffffffffu, rel[k], j) == lane) {
#pragma unroll
            for (int q = 0; q <= kCeFixes; ++q)
              if (f.toks == q) tok[q] = (base + first[k]) * 32 + j;
            ++f.toks;
          }
        }
      }
    }
  }
  if (f.toks > kCeFixes) {
    f.sum = p.label_sums + (size_t)SPEC_CHECKED(tok[kCeFixes], p.N, kSiteLinearCe) * p.D;
    f.toks = 0;
  }
#pragma unroll
  for (int q = 0; q < kCeFixes; ++q)
    if (q < f.toks) {
      f.src[q] = p.h + (size_t)SPEC_CHECKED(tok[q], p.N, kSiteLinearCe) * p.D;
      f.r[q] = p.resid[tok[q]];
    }
  return f;
}

// dH and dW: bf16 where the tile is the whole sum, else dH's sums in single
// precision, set by the first piece and added to by the others.  `dead`: a wait ran
// out, here or before, and the result is NaN.  `sum`: what earlier chunks gave (kChunks).
template <bool kChunks>
__device__ __forceinline__ void ce_grad_tile(const CeParams& p, const CeMaps& maps,
                                             const CeTile& t, uint32_t addr, int row0, int half,
                                             CeOut& o, const CeFix& fix, bool dead,
                                             const float* sum) {
  const int lane = threadIdx.x & 31;
  const bool dh = t.kind == 1;
  const int rows = dh ? p.N : p.nv, r0 = t.m0 + row0;
  const int from = half * 128, cols = min(from + 128, p.D - t.n0);
  const bool sums = dh && !p.dh_direct;
  const int step = sums ? 32 : 64;
  for (int c0 = from; c0 < cols; c0 += step) {
    const uint32_t box = ce_box_begin(o);
    for (int h = 0; h < step; h += 32) {
      const int at = t.n0 + c0 + h;
      CeRow row;
      if (fix.toks > 0) row = ce_row(fix.src[0] + at, p.D - at);
      float x[32];
      tmem_load32(addr + c0 + h, x);
      if (kChunks) {
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = __fadd_rn(x[c], sum[c0 - from + h + c]);
      }
      if (t.iters == 0) {  // a slice past the end of a short last piece
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = 0.0f;
      }
      if (dead) {
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = __int_as_float(0x7fc00000);
      }
      if (fix.toks > 0) ce_add_row(x, row, fix.r[0]);
#pragma unroll
      for (int q = 1; q < kCeFixes; ++q)
        if (q < fix.toks) ce_add_row(x, ce_row(fix.src[q] + at, p.D - at), fix.r[q]);
      if (fix.sum != nullptr) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q * 4 < p.D - at) {
            const float4 a = reinterpret_cast<const float4*>(fix.sum + at)[q];
            x[q * 4] = __fadd_rn(x[q * 4], a.x);
            x[q * 4 + 1] = __fadd_rn(x[q * 4 + 1], a.y);
            x[q * 4 + 2] = __fadd_rn(x[q * 4 + 2], a.z);
            x[q * 4 + 3] = __fadd_rn(x[q * 4 + 3], a.w);
          }
      }
      if (sums) {
#pragma unroll
        for (int q = 0; q < 8; ++q) ce_box_put(box, q, pack_vec<float>(x + q * 4));
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) ce_box_put(box, h / 8 + q, pack_vec<uint16_t>(x + q * 8));
      }
    }
    ce_box_ready();
    if (lane == 0 && r0 < rows) {
      if (!sums) tma_store(dh ? &maps.dh_out : &maps.dw_out, box, t.n0 + c0, (dh ? 0 : p.v0) + r0);
      else if (p.first) tma_store3(&maps.acc, box, t.n0 + c0, r0, t.slice);
      else tma_add3(&maps.acc, box, t.n0 + c0, r0, t.slice);
      bulk_commit();
    }
  }
}

// Header of the workspace: labels outside the vocabulary, and for the gradients a loss
// that timed out, which lse tells (the loss's own status may have stood in this header).
// Done by the epilogue warps of one CTA (its other warps go on).
template <CeMode M>
__device__ __forceinline__ void ce_check(const CeParams& p, CeBars& bars) {
  const int th = threadIdx.x - kMmEpilogue * 32, n = kMmThreads - kMmEpilogue * 32;
  int bad = 0, lost = 0;
#pragma unroll 4
  for (int i = th; i < p.N; i += n) {
    bad += p.labels[i] >= p.V ? 1 : 0;
    if (M == kCeDz) lost |= __float_as_uint(p.lse[i]) == SPEC_TIMEOUT_NAN ? 1 : 0;
  }
  if (bad) atomicAdd(&bars.bad, bad);
  if (lost) atomicOr(&bars.lost, 1);
  asm volatile("bar.sync 1, %0;" ::"r"(n) : "memory");
  if (th == 0) {
    const int found = *(volatile int*)&bars.bad;
    int status = found ? SPEC_ERR_BAD_INPUT : SPEC_OK;
    if (*(volatile int*)&bars.lost) status = SPEC_ERR_TIMEOUT;
#ifdef SPEC_DEBUG
    if (g_debug_inject != SPEC_OK) status = g_debug_inject;
#endif
    p.header->status = status;
    p.header->bad_requests = found;
    p.header->first_bad = INT32_MAX;
  }
}

// kChunks: sums are taken in chunks (the loss; dZ and the gradients where some sum has more
// than one: the code for it costs dZ's short form 1 us of a call of 15 us, 64 tokens,
// V = 1024, D = 128).  With the 128 sums of a thread the compiler spills a few registers
// around the chunks' loop (60 to 92 bytes of 168 registers, the share of ten warps
// on an SM), the gradients' form all of the sums: their loop turns once in 300 us.
template <CeMode M, bool kChunks>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmThreads, 1)
    ce_mma_kernel(const __grid_constant__ CeMaps maps, const __grid_constant__ CeParams p) {
  constexpr int kChunk = M == kCeGrads ? kMmGradChunk : kMmChunk;
  extern __shared__ unsigned char smem_raw[];
  __shared__ CeBars bars;
  const uint32_t ring = (smem_addr(smem_raw) + 1023) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMmStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bars.tfull[a], 1);
      mbar_init(&bars.tempty[a], 16);  // the epilogue warps of both CTAs
    }
    bars.abort_flag = 0;
    bars.bad = bars.lost = 0;
    fence_mbar_init();
  }
  if (warp == kMmIssuer) tmem_alloc(&bars.tmem, 512);
  if (warp == kMmProducer && lane < 6) {  // the maps this kernel loads from
    const CUtensorMap* m = lane == 0   ? &maps.h_k
                           : lane == 1 ? &maps.w_k
                           : lane == 2 ? &maps.dz_k
                           : lane == 3 ? &maps.h_mn
                           : lane == 4 ? &maps.w_mn
                                       : &maps.dz_mn;
    if (M == kCeGrads ? lane >= 2 : lane < 2) tma_prefetch_map(m);
  }
  tmem_fence_before();
  cluster_sync();  // both CTAs' barriers are there
  tmem_fence_after();
  const uint32_t tmem = bars.tmem;
  pdl_wait();
  pdl_launch_dependents();
  bool ok = true;
  int loads = 0;  // stages the producer has filled

  if (warp == kMmProducer) {
    if (lane == 0) {
      // The previous kernel's stores (dZ) before this one's asynchronous reads.
      asm volatile("fence.proxy.async;" ::: "memory");
      for (int i = 0; ok; ++i) {
        const CeTile t = ce_tile<M>(p, i);
        if (t.kind < 0) break;
        const int am = t.m0 + rank * kMmHalf, bn = t.n0 + rank * kMmHalf;
        const int parts_len = M == kCeLoss ? (t.iters * p.group + 31) / 32 : 1;
        for (int k = 0; k < t.iters; ++k, ++loads) {
          const int s = loads % kMmStages, round = loads / kMmStages;
          if (round > 0 && !mbar_sleep(&bars.empty[s], (round - 1) & 1, &bars.abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t a = ring + s * kMmStageBytes, b = a + kMmABytes;
          // Both CTAs' loads complete on the first one's barrier.
          const uint32_t bar = dsmem_map(&bars.full[s], 0);
          // Rows of A past the last token are not loaded where the tile is the only
          // one: what is left there reaches rows of the result that nobody reads.
          const bool a_mn = t.kind == 2, all_a = a_mn || p.a_rows == kMmHalf;
          if (rank == 0)
            mbar_arrive_expect_tx(&bars.full[s], 2 * kMmBBytes + (all_a ? 2 * kMmABytes
                                                                        : p.a_rows * kMmK * 2));
          const int k0 = t.k0 + k * kMmK;
          if (M != kCeGrads) {
            // (Rows before the first and past the last token read as 0.)
            const int part = M == kCeLoss && p.group < 32 ? k / parts_len * p.group : 0;
            if (all_a || rank == 0) tma_load(a, &maps.h_k, k0, am - part, bar);
            tma_load(b, &maps.w_k, k0, (M == kCeDz ? p.v0 : 0) + bn, bar);
          } else {
            if (!a_mn) {
              if (all_a || rank == 0) tma_load(a, &maps.dz_k, k0, am, bar);
            } else {
              for (int c = 0; c < kMmHalf; c += 64)
                tma_load(a + c * 128, &maps.dz_mn, am + c, k0, bar);
            }
            for (int c = 0; c < kMmHalf; c += 64)
              tma_load(b + c * 128, t.kind == 1 ? &maps.w_mn : &maps.h_mn, bn + c,
                       (t.kind == 1 ? p.v0 : 0) + k0, bar);
          }
        }
      }
      // The products' last arrivals on `empty` come before the CTA ends.
      for (int l = max(0, loads - kMmStages); ok && l < loads; ++l)
        ok = mbar_sleep(&bars.empty[l % kMmStages], (l / kMmStages) & 1, &bars.abort_flag);
    }
  } else if (warp == kMmIssuer) {
    if (lane == 0 && rank == 0) {
      int it = 0, sub = 0;  // stages used, accumulators filled
      for (int i = 0; ok; ++i) {
        const CeTile t = ce_tile<M>(p, i);
        if (t.kind < 0) break;
        const bool a_mn = t.kind == 2, b_mn = t.kind != 0;
        const uint32_t idesc = mma_idesc(kMmM, kMmN, a_mn, b_mn);
        const uint32_t a_step = a_mn ? 2048 : 32, b_step = b_mn ? 2048 : 32;
        int k = 0;
        do {  // (once where there is nothing to sum)
          const int acc = sub & 1, end = kChunks ? min(t.iters, k + kChunk) : t.iters;
          if (sub >= 2 &&
              !mbar_sleep(&bars.tempty[acc], ((sub >> 1) - 1) & 1, &bars.abort_flag)) {
            ok = false;
            break;
          }
          tmem_fence_after();
          for (const int first = k; k < end; ++k, ++it) {
            const int s = it % kMmStages;
            if (!mbar_sleep(&bars.full[s], (it / kMmStages) & 1, &bars.abort_flag)) {
              ok = false;
              break;
            }
            tmem_fence_after();
            const uint32_t a = ring + s * kMmStageBytes, b = a + kMmABytes;
#pragma unroll
            for (int j = 0; j < kMmK / 16; ++j)
              mma_f16(tmem + acc * kMmN, mma_desc(a + j * a_step, 8192, 1024),
                      mma_desc(b + j * b_step, 8192, 1024), idesc, k > first || j > 0);
            mma_commit(&bars.empty[s]);
          }
          if (!ok) break;
          mma_commit(&bars.tfull[acc]);
          ++sub;
        } while (k < t.iters);
      }
    }
  } else {
    if (p.check && blockIdx.x == 0) ce_check<M>(p, bars);
    const int quarter = warp & 3;  // the lanes of tensor memory this warp may read
    const int half = (warp - kMmEpilogue) >> 2;
    CeOut out = {ring + kMmStages * kMmStageBytes + (warp - kMmEpilogue) * kMmBoxes * kMmBoxBytes, 0};
    CeTile next = ce_tile<M>(p, 0);
    next.m0 += rank * kMmHalf;
    uint32_t word = M == kCeGrads ? ce_fix_word(p, next, quarter * 32) : 0;
    // After a timeout (the loss's, dZ's) nothing here is this call's: not the map of
    // labels either, which then is not looked at.
    bool dead = M == kCeGrads && p.header->status == SPEC_ERR_TIMEOUT;
    int sub = 0;
    auto filled = [&]() -> uint32_t {  // the next accumulator, once filled
      const int acc = sub & 1;
      if (!mbar_sleep(&bars.tfull[acc], (sub >> 1) & 1, &bars.abort_flag)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      tmem_fence_after();
      return tmem + acc * kMmN + ((uint32_t)(quarter * 32) << 16);
    };
    auto drained = [&]() {
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(dsmem_map(&bars.tempty[sub & 1], 0));
      ++sub;
    };
    for (int i = 0;; ++i) {
      const CeTile t = next;
      if (t.kind < 0) break;
      next = ce_tile<M>(p, i + 1);
      next.m0 += rank * kMmHalf;
      CeFix fix;
      if (M == kCeGrads) {
        fix.toks = 0;
        fix.sum = nullptr;
        if (!dead) fix = ce_fix(p, t, quarter * 32, word);
        word = ce_fix_word(p, next, quarter * 32);
      }
      float sum[kCePartV];
      if (kChunks) {
#pragma unroll
        for (int c = 0; c < kCePartV; ++c) sum[c] = 0.0f;
        for (int k = kChunk; k < t.iters && ok; k += kChunk) {
          const uint32_t addr = filled() + half * kCePartV;
          if (!ok) break;
#pragma unroll
          for (int q = 0; q < kCePartV; q += 32) {
            float x[32];
            tmem_load32(addr + q, x);
#pragma unroll
            for (int c = 0; c < 32; ++c) sum[q + c] = __fadd_rn(sum[q + c], x[c]);
          }
          drained();
        }
      }
      if constexpr (M != kCeGrads) {
        const uint32_t addr = ok ? filled() : 0;
        if (!ok) break;
        if (M == kCeLoss && p.group < 32) {
          if (t.m0 + quarter == 0) ce_loss_few(p, t, addr, half, sum);
        } else if constexpr (M == kCeLoss)
          ce_loss_row(p, t, addr, t.m0 + quarter * 32 + lane, half, sum);
        else
          ce_dz_tile<kChunks>(p, maps, t, addr, quarter * 32, half, out, sum);
      } else {
        const uint32_t addr = ok ? filled() : tmem;
        dead |= !ok;  // the tiles that are left become NaN
        ce_grad_tile<kChunks>(p, maps, t, addr, quarter * 32, half, out, fix, dead, sum);
      }
      if (ok) drained();
    }
    if (M != kCeLoss && lane == 0) bulk_wait_read<0>();
  }
  if (!ok) {
    *(volatile int*)&bars.abort_flag = 1;
    if (lane == 0) atomicMax(&p.header->status, SPEC_ERR_TIMEOUT);  // over bad labels
    // Loads still on their way have to land before the CTAs end.
    if (warp == kMmProducer && lane == 0 && rank == 0) {
      int never = 0;
      for (int l = max(0, loads - kMmStages); l < loads; ++l)
        mbar_sleep(&bars.full[l % kMmStages], (l / kMmStages) & 1, &never);
    }
  }
  __syncwarp();
  tmem_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still reach its barriers
  tmem_fence_after();
  if (warp == kMmIssuer) tmem_free(tmem, 512);
}

// Labels with more than kCeFixes tokens: what rounding took from their entries of dZ,
// times the tokens' hidden states, summed into the row of label_sums that belongs to the
// label's (kCeFixes + 1)-th token.  Each of a CTA's eight warps looks whether its
// token is such a one; the whole CTA then goes through the labels 4096 at a time, lists the
// tokens in order and sums 512 columns, each 8 of them by one thread of each
// quarter.  The additions' order depends on the sizes and labels alone.
//
// The kernel runs beside the first piece's dZ, on SMs that has none of or is done with: it
// reads only what was there before that kernel, which lets its successor start after its
// own wait for its predecessors.  It ends with a wait for that kernel, so that whoever
// waits for this one has waited for both.
// (Summing in dW's epilogue instead, the warp listing a row's tokens again for each 32
// columns, took 1907 us where this takes 510, loss and gradients: 2048 tokens, V = 32000,
// D = 1024, labels with p(v) ~ 1/v, whose many frequent labels share a few tiles.  Labels
// that hardly repeat take 370 us there.  65536 tokens, V = 1000, D = 512, gradients: 854 us,
// 653 without this kernel; with lists of 1024 labels 1020.)
constexpr int kCeLabelThreads = 256, kCeLabelCols = 512, kCeLabelChunk = 4096;
__global__ void __launch_bounds__(kCeLabelThreads)
    ce_label_kernel(const __grid_constant__ CeParams p) {
  constexpr int kWarps = kCeLabelThreads / 32, kGroups = kCeLabelCols / 8;
  constexpr int kSubs = kCeLabelThreads / kGroups;
  constexpr int kWords = kCeLabelChunk / kCeLabelThreads;  // 32 labels each, of a warp
  __shared__ int owner[kWarps];
  __shared__ int found[kWarps];
  __shared__ int list[kCeLabelChunk];
  __shared__ float weight[kCeLabelChunk];
  __shared__ float part[kSubs][kGroups][9];
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  {
    const int i = blockIdx.x * kWarps + warp;
    const int y = i < p.N ? p.labels[i] : -1;
    int before = 0;  // tokens with this label before i
    if (y >= 0 && y < p.V) {
      for (int j0 = 0; j0 < i && before <= kCeFixes; j0 += 256) {
        int l[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int j = j0 + k * 32 + lane;
          l[k] = j < i ? p.labels[j] : -1;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) before += __popc(__ballot_sync(0xffffffffu, l[k] == y));
      }
    }
    if (lane == 0) owner[warp] = before == kCeFixes ? y : -1;
  }
  __syncthreads();
  const int group = tid % kGroups, sub = tid / kGroups;
  const int col = blockIdx.y * kCeLabelCols + group * 8;
  for (int w = 0; w < kWarps; ++w) {
    const int y = owner[w];
    if (y < 0) continue;
    float s[8] = {};
    for (int c = 0; c < p.N; c += kCeLabelChunk) {
      // Each warp takes 512 labels in a row.
      const int c0 = c + warp * (kWords * 32) + lane;
      uint32_t hits = 0;  // the lane's own labels, one bit a word
#pragma unroll
      for (int k = 0; k < kWords; ++k)
        hits |= (uint32_t)(c0 + k * 32 < p.N && p.labels[c0 + k * 32] == y) << k;
      int mine = 0;  // the warp's tokens
#pragma unroll
      for (int k = 0; k < kWords; ++k)
        mine += __popc(__ballot_sync(0xffffffffu, (hits >> k) & 1));
      if (lane == 0) found[warp] = mine;
      __syncthreads();
      int at = 0, n = 0;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        at += k < warp ? found[k] : 0;
        n += found[k];
      }
      if (mine > 0) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          const uint32_t m = __ballot_sync(0xffffffffu, (hits >> k) & 1);
          if ((hits >> k) & 1) {
            const int slot = at + __popc(m & ((1u << lane) - 1)), i = c0 + k * 32;
            list[slot] = i;
            weight[slot] = ce_rounded_off(ce_label_entry(p.nll[i], p.g[i]));
          }
          at += __popc(m);
        }
      }
      __syncthreads();
      if (col < p.D) {
        for (int k = sub; k < n; k += 4 * kSubs) {
          uint4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            v[u] = k + u * kSubs < n
                       ? *reinterpret_cast<const uint4*>(
                             p.h + (size_t)SPEC_CHECKED(list[k + u * kSubs], p.N, kSiteLinearCe) *
                                       p.D + col)
                       : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float r = k + u * kSubs < n ? weight[k + u * kSubs] : 0.0f;
            float a[8];
            ElemTraits<uint16_t>::unpack(v[u], a);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = fmaf(r, a[e], s[e]);
          }
        }
      }
      __syncthreads();  // before the lists are written again
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[sub][group][e] = s[e];
    __syncthreads();
    if (sub == 0 && col < p.D) {
#pragma unroll
      for (int k = 1; k < kSubs; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = __fadd_rn(s[e], part[k][group][e]);
      float4* out = reinterpret_cast<float4*>(
          p.label_sums +
          (size_t)SPEC_CHECKED(blockIdx.x * kWarps + w, p.N, kSiteLinearCe) * p.D + col);
      out[0] = make_float4(s[0], s[1], s[2], s[3]);
      out[1] = make_float4(s[4], s[5], s[6], s[7]);
    }
    __syncthreads();
  }
  pdl_wait();
}

// h . w over D entries, by a warp, the sum in every lane.
__device__ __forceinline__ float ce_dot(const uint16_t* h, const uint16_t* w, int D) {
  const int lane = threadIdx.x & 31;
  float2 a[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll 4
  for (int d = lane * 8; d < D; d += 256) {
    float x[8], y[8];
    ElemTraits<uint16_t>::unpack(*reinterpret_cast<const uint4*>(h + d), x);
    ElemTraits<uint16_t>::unpack(*reinterpret_cast<const uint4*>(w + d), y);
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      a[(e >> 1) & 1] = f32x2_fma(make_float2(x[e], x[e + 1]), make_float2(y[e], y[e + 1]),
                                  a[(e >> 1) & 1]);
  }
  const float2 t = f32x2_add(a[0], a[1]);
  return warp_sum(__fadd_rn(t.x, t.y));
}

// Tokens' pairs into lse and nll: `tokens` (a power of two up to 32) a CTA, the
// other threads over each one's pairs, eight loads at a time.  The labels' logits are
// formed here, a warp each, rounded to nearest: the tensor cores' sums are cut off
// towards zero, which for the largest logit of a row, a long sum of one sign, is a
// bias of 3e-7 of itself, and a small loss has all of it.  That comes before the wait for
// the products, which start this kernel after their own wait: what the caller gave is
// there.
constexpr int kCeFinishThreads = 1024;
__global__ void __launch_bounds__(kCeFinishThreads)
    ce_finish_kernel(const __grid_constant__ CeParams p, int tokens, float* nll, float* lse) {
  __shared__ float sm[2][kCeFinishThreads / 32][32];
  __shared__ float z_label[32];
  const int tid = threadIdx.x, tok = tid & (tokens - 1), groups = kCeFinishThreads / tokens;
  const int warp = tid >> 5;
  if (warp < tokens && blockIdx.x * tokens + warp < p.N) {
    const int at = blockIdx.x * tokens + warp, y = p.labels[at];
    if (y >= 0 && y < p.V) {
      const float dot = ce_dot(p.h + (size_t)at * p.D, p.w + (size_t)y * p.D, p.D);
      if ((tid & 31) == 0) z_label[warp] = dot;
    }
  }
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x * tokens + tok;
  const bool lost = p.header->status == SPEC_ERR_TIMEOUT;
  const float2* part = p.partials + i;
  const float none = -FLT_MAX / 2;
  float m = none, s = 0.0f;
  if (i < p.N) {
    for (int t = tid / tokens; t < p.parts; t += 8 * groups) {
      float2 q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        q[j] = t + j * groups < p.parts ? part[(size_t)(t + j * groups) * p.N]
                                        : make_float2(none, 0.0f);
      float n = m;
#pragma unroll
      for (int j = 0; j < 8; ++j) n = fmaxf(n, q[j].x);
      s = __fmul_rn(s, ex2(__fsub_rn(m, n)));
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(q[j].y, ex2(__fsub_rn(q[j].x, n)), s);
      m = n;
    }
  }
  // Each token's maximum and sum: over its lanes in a warp, then over the warps.
  for (int o = 16; o >= tokens; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const float n = fmaxf(m, m2);
    s = __fadd_rn(__fmul_rn(s, ex2(__fsub_rn(m, n))), __fmul_rn(s2, ex2(__fsub_rn(m2, n))));
    m = n;
  }
  if ((tid & 31) < tokens) {
    sm[0][warp][tok] = m;
    sm[1][warp][tok] = s;
  }
  __syncthreads();
  if (tid >= tokens || i >= p.N) return;
  if (lost) {  // a wait ran out: some pairs are not this call's
    nll[i] = lse[i] = __uint_as_float(SPEC_TIMEOUT_NAN);
    return;
  }
  float top = sm[0][0][tok];
#pragma unroll
  for (int w = 1; w < kCeFinishThreads / 32; ++w) top = fmaxf(top, sm[0][w][tok]);
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < kCeFinishThreads / 32; ++w)
    s = fmaf(sm[1][w][tok], ex2(__fsub_rn(sm[0][w][tok], top)), s);
  const float nan = __int_as_float(0x7fc00000);
  const int y = p.labels[i];
  const bool has = y >= 0 && y < p.V;
  const float z = has ? z_label[tok] : -INFINITY;
  // s = sum over the others of 2^(z_v log2 e - top); the label's own term is apart.
  // `gap` is how far the others' maximum lies above the label, in base 2:
  //   nll = log(1 + s 2^gap),  lse = log(s 2^top + 2^(z log2 e)).
  // A token that is well predicted so keeps the relative precision of its small
  // loss, which the difference of lse and z does not have.
  const float zl = __fmul_rn(z, kLog2e), gap = fmaf(z, -kLog2e, top), T = fmaxf(top, zl);
  const float all = __fadd_rn(__fmul_rn(s, ex2(__fsub_rn(top, T))), ex2(__fsub_rn(zl, T)));
  // A sum that is not positive and finite (an infinity or NaN among the inputs)
  // gives NaN.
  const float l = all > 0.0f && all <= FLT_MAX && s >= 0.0f
                      ? __fmul_rn(__fadd_rn(T, log2f(all)), kLn2f)
                      : nan;
  lse[i] = l;
  if (y < 0) nll[i] = 0.0f;
  else if (!has || !(l == l)) nll[i] = nan;
  else if (gap <= 0.0f) nll[i] = log1pf(__fmul_rn(s, ex2(gap)));
  else nll[i] = __fmul_rn(__fadd_rn(gap, log2f(__fadd_rn(s, ex2(-gap)))), kLn2f);
}

// dH from its parts: the slices are added in a fixed order, then what rounding took
// from the label's entry, and rounded once.  A CTA does 32 groups of eight entries, eight
// threads over the slices of each.
__global__ void __launch_bounds__(256)
    ce_round_kernel(const __grid_constant__ CeParams p, uint16_t* out) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float part[8][32][9];
  const long long n = (long long)p.N * p.D;
  const int g = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const long long i = (blockIdx.x * 32LL + g) * 8;
  float x[8] = {};
  if (i < n) {
#pragma unroll 4
    for (int s = sl; s < p.splits; s += 8) {
      const float4* a = reinterpret_cast<const float4*>(p.dh_acc + s * n + i);
      const float4 u = a[0], v = a[1];
      x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
      x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) part[sl][g][e] = x[e];
  __syncthreads();
  if (sl != 0 || i >= n) return;
  for (int k = 1; k < min(8, p.splits); ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += part[k][g][e];
  if (p.header->status == SPEC_ERR_TIMEOUT) {  // some of the sums are not this call's
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __int_as_float(0x7fc00000);
  }
  const int row = (int)(i / p.D), col = (int)(i - (long long)row * p.D);
  const int y = p.labels[row];
  if (y >= 0 && y < p.V) {
    float a[8];
    ElemTraits<uint16_t>::unpack(
        *(reinterpret_cast<const uint4*>(p.w + (size_t)y * p.D + col)), a);
    const float r = p.resid[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(r, a[e], x[e]);
  }
  *reinterpret_cast<uint4*>(out + i) = pack_vec<uint16_t>(x);
}

}  // namespace specv
