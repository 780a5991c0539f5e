// A paged key-value cache: the append of new tokens' keys and values, and the attention of
// the new tokens over the pages.
//
//   s_tj = scale q_t . k_j     m_t = max_j s_tj     l_t = sum_j exp(s_tj - m_t)
//   out_t = sum_j exp(s_tj - m_t) v_j / l_t         lse_t = m_t + log l_t
#pragma once

#include "tcgen05.cuh"

namespace specv {

struct PagedParams {
  spec_paged_cache_t c;
  int rows;
  // Append.
  const uint16_t *k_new, *v_new;
  long long k_stride, v_stride;
  // Attention.
  const uint16_t* q;
  long long q_stride;
  int heads, causal, window;
  float scale;
  uint16_t* out;
  float* lse;
  WsHeader* header;
};

// The request a row belongs to: the last whose first row is at most `row` (new_start does
// not decrease), or -1.
__device__ __forceinline__ int request_of(const int32_t* new_start, int B, int row) {
  if (row < new_start[0] || row >= new_start[B]) return -1;
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (new_start[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  return row < new_start[lo + 1] ? lo : -1;
}

// What a request's rows and length have to be for its rows to be looked up.
__device__ __forceinline__ bool request_ok(const PagedParams& p, int first, int last, int len) {
  return first >= 0 && first <= last && last <= p.rows && len >= 0 &&
         (long long)len <= (long long)p.c.max_pages * p.c.page_size;
}

constexpr int kAppendThreads = 256;

// One thread per 16 bytes of a key and of a value.
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ PagedParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int vecs = p.c.width / 8, per_row = p.c.kv_heads * vecs;
  const long long at = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
  if (at >= (long long)p.rows * per_row) return;
  const int row = (int)(at / per_row), rest = (int)(at % per_row);
  const int h = rest / vecs, e = rest % vecs * 8;
  const int b = request_of(p.c.new_start, p.c.B, row);
  if (b < 0) return;
  const int first = p.c.new_start[b], last = p.c.new_start[b + 1], len = p.c.kv_len[b];
  if (!request_ok(p, first, last, len) || len < last - first) return;
  const int pos = len - (last - row);
  const int page = p.c.page_table[(size_t)b * p.c.max_pages + pos / p.c.page_size];
  if (page < 0 || page >= p.c.num_pages) return;
  const int slot = pos % p.c.page_size;
  const uint4 k = *reinterpret_cast<const uint4*>(p.k_new + row * p.k_stride + h * p.c.width + e);
  const uint4 v = *reinterpret_cast<const uint4*>(p.v_new + row * p.v_stride + h * p.c.width + e);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.c.k_cache) + page * p.c.k_page +
                            slot * p.c.k_slot + h * p.c.k_head + e) = k;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.c.v_cache) + page * p.c.v_page +
                            slot * p.c.v_slot + h * p.c.v_head + e) = v;
}

constexpr int kAttnWarps = 4;

// The workspace's header, and the requests whose rows or length are out of range.
__global__ void __launch_bounds__(1024) paged_header_kernel(const __grid_constant__ PagedParams p) {
  pdl_wait();
  pdl_launch_dependents();
  int bad = 0;
  for (int b = threadIdx.x; b < p.c.B; b += blockDim.x)
    bad |= !request_ok(p, p.c.new_start[b], p.c.new_start[b + 1], p.c.kv_len[b]);
  bad = __syncthreads_or(bad);
  if (threadIdx.x != 0) return;
  p.header->status = bad ? SPEC_ERR_BAD_INPUT : SPEC_OK;
  p.header->bad_requests = 0;
  p.header->first_bad = INT32_MAX;
}

// One warp per row and head: 32 entries at a time, one per lane for the scores, then the
// lanes share the width.
__global__ void __launch_bounds__(kAttnWarps * 32)
    paged_attention_kernel(const __grid_constant__ PagedParams p) {
  __shared__ float qs[kAttnWarps][128];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long at = (long long)blockIdx.x * kAttnWarps + warp;
  if (at >= (long long)p.rows * p.heads) return;
  const int row = (int)(at / p.heads), h = (int)(at % p.heads);
  const int hk = h / (p.heads / p.c.kv_heads), D = p.c.width;
  const int b = request_of(p.c.new_start, p.c.B, row);
  if (b < 0) return;
  const int first = p.c.new_start[b], last = p.c.new_start[b + 1], len = p.c.kv_len[b];
  bool bad = !request_ok(p, first, last, len);
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, m = -INFINITY, l = 0.0f;
  if (!bad) {
    for (int d = lane; d < D; d += 32)
      qs[warp][d] = bf16_to_f32(p.q[row * p.q_stride + h * D + d]) * p.scale;
    __syncwarp();
    const int pos = len - (last - row);
    const int to = p.causal ? pos + 1 : len;
    const int from = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    for (int j0 = from; j0 < to; j0 += 32) {
      const int j = j0 + lane;
      int page = -1, slot = 0;
      float s = -INFINITY;
      if (j < to) {
        page = p.c.page_table[(size_t)b * p.c.max_pages + j / p.c.page_size];
        slot = j % p.c.page_size;
        if (page < 0 || page >= p.c.num_pages) {
          bad = true;
          page = -1;
        } else {
          const uint16_t* k = static_cast<const uint16_t*>(p.c.k_cache) + page * p.c.k_page +
                              slot * p.c.k_slot + hk * p.c.k_head;
          s = 0.0f;
          for (int d = 0; d < D; ++d) s = fmaf(qs[warp][d], bf16_to_f32(k[d]), s);
        }
      }
      float mx = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float nm = fmaxf(m, mx);
      const float ref = nm == -INFINITY ? 0.0f : nm;
      const float fix = expf(m - ref), w = expf(s - ref);
      m = nm;
      l = l * fix + w;
      for (int i = 0; i < 4; ++i) acc[i] *= fix;
      for (int c = 0; c < 32; ++c) {
        const float wc = __shfl_sync(0xffffffffu, w, c);
        const int pc = __shfl_sync(0xffffffffu, page, c), sc = __shfl_sync(0xffffffffu, slot, c);
        if (pc < 0) continue;
        const uint16_t* v = static_cast<const uint16_t*>(p.c.v_cache) + pc * p.c.v_page +
                            sc * p.c.v_slot + hk * p.c.v_head;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i * 32 < D) acc[i] = fmaf(wc, bf16_to_f32(v[i * 32 + lane]), acc[i]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  }
  bad = __any_sync(0xffffffffu, bad);
  if (bad && lane == 0) atomicCAS(&p.header->status, SPEC_OK, SPEC_ERR_BAD_INPUT);
  const float nan = __int_as_float(0x7fc00000);
  for (int i = 0; i < 4; ++i)
    if (i * 32 < D) {
      const float o = bad ? nan : l > 0.0f || l != l ? acc[i] / l : 0.0f;
      p.out[((size_t)row * p.heads + h) * D + i * 32 + lane] =
          (uint16_t)(pack_bf16(o, 0.0f) & 0xffff);
    }
  if (p.lse != nullptr && lane == 0) p.lse[(size_t)row * p.heads + h] = bad ? nan : m + logf(l);
}

}  // namespace specv
