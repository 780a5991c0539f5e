// A paged key-value cache: what its calls share, and the append of new tokens' keys and
// values.
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

// One thread per 16 bytes of a key and of a value: bound by memory (32768 tokens of 8 heads of
// 128, 268 MB read and written, 44 us, 6.1 TB/s; 288 tokens 3 us, the launch).
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

}  // namespace specv
