// Softmax cross entropy of a linear vocabulary head, and its gradients, without
// keeping the logits.
//
//   z_iv  = h_i . w_v          lse_i = log sum_v exp z_iv
//   nll_i = lse_i - z_{i,y_i}
//   dZ_iv = g_i (exp(z_iv - lse_i) - [v = y_i]),  dH = dZ W,  dW = dZ^T H
//
// The loss forms the logits tile by tile and keeps of each tile one (max, sum)
// pair per row.  The gradients form them again, a piece of the vocabulary at a
// time: the piece's dZ is written in bfloat16 to a scratch buffer that stays in
// L2, and both products read it from there.  dZ is rounded to bfloat16 (relative
// 2^-9) because the matrix units take both operands in one type, and the
// gradients come out in bfloat16 anyway; every sum is in single precision.
#pragma once

#include "grad_norm.cuh"

namespace specv {

constexpr int kCeTileV = 64;       // vocabulary entries per (max, sum) pair
constexpr int kCePiece = 8192;     // vocabulary entries per piece of the gradients
constexpr int kCeMaxTokens = 1 << 18;
constexpr int kCeMaxWidth = 1 << 15;

struct CeLayout {
  size_t header, partials, z_label, dz, dh_acc, total;
  int tiles;     // vocabulary tiles
  int piece;     // vocabulary entries per piece (a multiple of kCeTileV)
};

inline CeLayout ce_layout(int N, int V, int D, bool grad) {
  CeLayout l = {};
  l.tiles = (V + kCeTileV - 1) / kCeTileV;
  l.piece = (int)std::min<long long>(kCePiece, (long long)l.tiles * kCeTileV);
  size_t o = align256(sizeof(WsHeader));
  if (!grad) {
    l.partials = o;
    o = align256(o + (size_t)N * l.tiles * sizeof(float2));
    l.z_label = o;
    o = align256(o + (size_t)N * sizeof(float));
  } else {
    l.dz = o;
    o = align256(o + (size_t)N * l.piece * 2);
    l.dh_acc = o;
    o = align256(o + (size_t)N * D * sizeof(float));
  }
  l.total = o;
  return l;
}

struct CeParams {
  const uint16_t* h;       // [N, D]
  const uint16_t* w;       // [V, D]
  const int32_t* labels;   // [N]
  const float* lse;        // [N] (gradients)
  const float* g;          // [N] (gradients)
  int N, V, D, tiles;
  float2* partials;        // [N, tiles]
  float* z_label;          // [N]
  uint16_t* dz;            // [N, piece]
  int piece, v0, nv;       // piece: buffer width, first entry, entries
  float* dh_acc;           // [N, D]
  uint16_t* dw;            // [V, D]
  int first;               // first piece: dh_acc is set, not added to
};

enum CeMode { kCeLoss, kCeDz, kCeDh, kCeDw };

// C[m][n] = sum_k A[m][k] B[n][k] on 64 x 64 tiles, one 4 x 4 block per thread.
template <CeMode M>
__global__ void __launch_bounds__(256) ce_gemm_kernel(CeParams p) {
  constexpr int BM = 64, BN = 64, BK = 16;
  __shared__ float sa[BK][BM + 4], sb[BK][BN + 4];
  const int rows = M == kCeDw ? p.nv : p.N;
  const int cols = M == kCeLoss ? p.V : M == kCeDz ? p.nv : p.D;
  const int K = M == kCeDh ? p.nv : M == kCeDw ? p.N : p.D;
  const int m0 = blockIdx.y * BM, n0 = blockIdx.x * BN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += BK) {
    for (int l = threadIdx.x; l < BM * BK; l += 256) {
      const int kk = (M == kCeDw) ? l / BM : l % BK, mm = (M == kCeDw) ? l % BM : l / BK;
      const int m = m0 + mm, k = k0 + kk;
      float x = 0.0f;
      if (m < rows && k < K) {
        if (M == kCeLoss || M == kCeDz) x = bf16_to_f32(p.h[(size_t)m * p.D + k]);
        if (M == kCeDh) x = bf16_to_f32(p.dz[(size_t)m * p.piece + k]);
        if (M == kCeDw) x = bf16_to_f32(p.dz[(size_t)k * p.piece + m]);
      }
      sa[kk][mm] = x;
    }
    for (int l = threadIdx.x; l < BN * BK; l += 256) {
      const bool kfast = M == kCeLoss || M == kCeDz;
      const int kk = kfast ? l % BK : l / BN, nn = kfast ? l / BK : l % BN;
      const int n = n0 + nn, k = k0 + kk;
      float x = 0.0f;
      if (n < cols && k < K) {
        if (kfast) x = bf16_to_f32(p.w[(size_t)(p.v0 + n) * p.D + k]);
        if (M == kCeDh) x = bf16_to_f32(p.w[(size_t)(p.v0 + k) * p.D + n]);
        if (M == kCeDw) x = bf16_to_f32(p.h[(size_t)k * p.D + n]);
      }
      sb[kk][nn] = x;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BK; ++kk) {
      float a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = sa[kk][ty * 4 + j];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = sb[kk][tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + ty * 4 + i;
    if (M == kCeLoss) {
      // The 16 threads of a row: one (max, sum) pair of the tile.
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + tx + 16 * j < cols) mx = fmaxf(mx, acc[i][j]);
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + tx + 16 * j < cols) s += ex2((acc[i][j] - mx) * kLog2e);
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (m < rows) {
        if (tx == 0) p.partials[(size_t)m * p.tiles + blockIdx.x] = make_float2(mx, s);
        const int y = p.labels[m];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + tx + 16 * j == y) p.z_label[m] = acc[i][j];
      }
    } else if (m < rows) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx + 16 * j;
        if (n >= cols) continue;
        if (M == kCeDz) {
          const int y = p.labels[m];
          float d = 0.0f;
          if (y >= 0 && y < p.V) {
            d = ex2((acc[i][j] - p.lse[m]) * kLog2e);
            if (p.v0 + n == y) d -= 1.0f;
            d *= p.g[m];
          }
          p.dz[(size_t)m * p.piece + n] = (uint16_t)pack_bf16(d, 0.0f);
        } else if (M == kCeDh) {
          float* at = p.dh_acc + (size_t)m * p.D + n;
          *at = p.first ? acc[i][j] : *at + acc[i][j];
        } else {
          p.dw[(size_t)(p.v0 + m) * p.D + n] = (uint16_t)pack_bf16(acc[i][j], 0.0f);
        }
      }
    }
  }
}

// Header of the workspace, and labels outside the vocabulary.
__global__ void ce_check_kernel(WsHeader* h, const int32_t* labels, int N, int V) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  int mine = 0;
  for (int i = threadIdx.x; i < N; i += blockDim.x) mine += labels[i] >= V ? 1 : 0;
  if (mine) atomicAdd(&bad, mine);
  __syncthreads();
  if (threadIdx.x == 0) {
    h->status = bad ? SPEC_ERR_BAD_INPUT : SPEC_OK;
    h->bad_requests = bad;
    h->first_bad = INT32_MAX;
  }
}

// One warp per token: its tiles' pairs into lse and nll.
__global__ void ce_finish_kernel(CeParams p, float* nll, float* lse) {
  const int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i >= p.N) return;
  const float2* part = p.partials + (size_t)i * p.tiles;
  float m = -INFINITY;
  bool nan = false;
  for (int t = lane; t < p.tiles; t += 32) m = fmaxf(m, part[t].x);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  FF s = {0.0f, 0.0f};
  for (int t = lane; t < p.tiles; t += 32) {
    const float e = __fmul_rn(part[t].y, ex2((part[t].x - m) * kLog2e));
    if (!(e <= FLT_MAX)) nan = true;
    else s = ff_add_f(s, e);
  }
  s = warp_sum_ff(s);
  nan = __any_sync(0xffffffffu, nan);
  if (lane == 0) {
    const float l = nan ? __int_as_float(0x7fc00000) : m + logf(ff_to_float(s));
    const int y = p.labels[i];
    lse[i] = l;
    nll[i] = y < 0 ? 0.0f : y < p.V ? l - p.z_label[i] : __int_as_float(0x7fc00000);
  }
}

__global__ void ce_round_kernel(const float* acc, uint16_t* out, long long n) {
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x)
    out[i] = (uint16_t)pack_bf16(acc[i], 0.0f);
}

}  // namespace specv
