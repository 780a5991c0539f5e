// Attention of a chunk of new tokens over a paged key-value cache.
//
//   s_tj = scale q_t . k_j     m_t = max_j s_tj     l_t = sum_j exp(s_tj - m_t)
//   out_t = sum_j exp(s_tj - m_t) v_j / l_t         lse_t = m_t + log l_t
//
// The query heads that share a key-value head are rows of one product: row r of a request
// and key-value head is token r / group, head r % group, so that a few tokens of many
// heads fill the 128 rows of a tensor-core tile that one token would leave empty.  A
// unit of work is up to 256 such rows against the tiles of 128 entries that some of
// them sees.  All units' tiles form one line, which the CTAs (one per SM) share out evenly:
// a unit that lies across a border is done in parts, each leaving unnormalised
// sums with its maximum, and a second kernel joins them (in the CTAs' order: the result's
// bits do not depend on timing).
//
// In a CTA: a warp that loads pages by TMA into a ring of tiles, one that issues the
// products, one that loads queries, one that works out the units, and two
// warpgroups of softmax.  Each warpgroup has a stream of its own, with scores and sums in
// tensor memory, so that one stream's softmax runs under the other's products.
//   more than 128 rows: each stream has 128 of them, a thread has a row.  The weights
//     exp(s - m) go back to tensor memory over the scores they come from, and are the
//     product's first operand there; a half of them is multiplied while the other is formed.
//   up to 128 rows: the tiles are transposed, S^T = K Q^T and O^T += V^T P^T: a thread
//     has an entry and all rows.  Up to 64 rows both streams have all of them and take
//     the tiles in turn, else each has a part of the rows and all tiles.
// The weights are rounded to bfloat16 (relative 2^-8: the products take both operands in one
// type).  The running maximum is only raised when a score passes it by more than 2^8,
// which leaves the sums' scaling out of almost every tile.
//
// Measured: 64 single tokens over up to 16384 entries (3.1 GB of keys and values) 475 to 496 us,
// 6.3 to 6.6 TB/s: memory.  32 requests of up to 17 tokens over up to 8192 entries, pages
// of 16: 189 us, 4.3 TB/s (pages of 64: 160 us; a page of 16 slots is 2 KB a copy, and the
// copies of a tile take the loading as long as memory does).  Two chunks of 4096 tokens
// behind 8192: 958 us, 1.13 PFLOP/s (half of the tensor cores' cycles): a
// stream's softmax takes 1.1 us of a tile, the other's products 0.65.  One token over 8000
// entries 24 us: 4.5 until the first page is on its way, 8 for three or four tiles and the
// part's store, 5 for the join, and their launches.
#pragma once

#include "paged.cuh"
#include "sample.cuh"
#include "tcgen05.cuh"

namespace specv {

constexpr int kAtThreads = 384;
// Roles by warp; the softmax's warpgroups are the second and third.
constexpr int kAtProducer = 0, kAtIssuer = 1, kAtQueries = 2, kAtPlanner = 3, kAtSoftmax = 4;
constexpr int kAtTile = 128;      // entries per tile, rows per stream
constexpr int kAtUnitRows = 256;  // rows per unit
constexpr int kAtFewRows = 64;    // rows per stream where the tiles are transposed
constexpr int kAtUnits = 4;       // units planned ahead
constexpr int kAtMaxCtas = 160;
constexpr int kAtReaders = 11;    // warps that read a planned unit
constexpr float kAtRaise = 8.0f;  // log2 of how far a score may pass the maximum in use

// A bounded wait that looks at the clock only when it has to wait long.
__device__ __forceinline__ bool at_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait_cluster(bar, parity) || mbar_sleep(bar, parity, abort);
}

// Shared memory: the ring of tiles, then the queries of a unit's streams (two buffers), and
// for units of few rows the weights of both streams.
template <int D>
struct AtSizes {
  static constexpr int kTileBytes = kAtTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kQ = kStages * kTileBytes;       // queries of up to 128 rows each
  static constexpr int kFewHalf = kAtFewRows * 128;     // few rows: 64 entries of each
  static constexpr int kFewQ = kAtFewRows * D * 2;
  static constexpr int kWeights = kQ + 2 * kFewQ;       // few rows: weights of a stream
  static constexpr int kFewWeights = kAtTile * 128;     // [entries, 64 rows]
  static constexpr int kTotal =
      kQ + (2 * kFewQ + 2 * kFewWeights > 2 * kTileBytes ? 2 * kFewQ + 2 * kFewWeights
                                                         : 2 * kTileBytes);
};

struct AtUnit {
  int b, h;        // request (-1: no more), key-value head
  int first, n;    // its first row in the batch, its new tokens
  int len;         // its entries
  int r0, rows;    // rows of the unit
  int lo, hi;      // entries that some row sees
  int tile0, nt;   // tiles done here
  int slot;        // where the part goes, -1: the result itself
  int bad;         // some row sees a page outside the cache
};

// The tiles of a unit, and which of their entries, that some of its rows see and others do not
// and whose values are not finite.  (The rows of a unit end, and under a window start, within
// 256 entries: in three tiles each.)
struct AtOdd {
  int tiles;
  int tile[6];
  uint32_t entries[6][kAtTile / 32];
};

struct AtControl {
  uint64_t full[10], empty[10];
  uint64_t s_full[2][2];  // of a stream; units of few rows have two sets of scores in turn
  uint64_t p_ready[2], p_half[2], pv_done[2], o_full[2], q_full[2], q_empty[2];
  uint64_t u_full[kAtUnits], u_empty[kAtUnits];
  uint64_t meet;  // of both warpgroups
  AtUnit unit[kAtUnits];
  AtOdd odd[kAtUnits];
  // Few rows, per stream and row: the maximum in use, negated (inf: none yet), and what scores
  // take for it; what the sums are multiplied by.
  __align__(16) float above[2][kAtFewRows];  // (read four at a time)
  __align__(16) float ref[2][kAtFewRows];
  float fix[2][kAtFewRows];
  int raise[2][2];
  uint64_t vote[2];
  uint64_t few_done[2];  // of units of few rows, in turn
  long long scan[kAtThreads / 32];
  long long start_off, start_left, start_line, start_cost, total;
  int start_b;
  int abort_flag, bad_page;
  uint32_t found_odd[kAtTile / 32];
  uint32_t tmem;
};

static_assert(offsetof(AtControl, above) % 16 == 0 && offsetof(AtControl, ref) % 16 == 0 &&
                  AtSizes<64>::kTotal % 16 == 0 && AtSizes<128>::kTotal % 16 == 0,
              "16-byte loads");

template <int D>
constexpr int at_smem() {
  return AtSizes<D>::kTotal + (int)sizeof(AtControl);
}
static_assert(at_smem<128>() <= 232448 && at_smem<64>() <= 232448, "shared memory of an SM");

// What a CTA leaves for the join: its two parts of units that lie across borders, the
// last of one (0) and the first of another (1).
struct AtPart {
  int used, end;  // end: the CTA with the unit's last part
  int b, h, first, r0, rows, pad;
};
struct AtCta {
  AtPart part[2];
};
constexpr int kAtLate = 1, kAtBadPage = 2;  // what a CTA has met: a timeout, a page outside the cache

struct AtParams {
  PagedParams p;
  int group;       // query heads per key-value head
  uint32_t magic;  // x / group = x magic >> shift for x < 2^31
  int shift;
  int page_bits;   // log2 of the page size
  int slot_rows;   // rows of a part
  float scale2;    // scale log2 e
  AtCta* ctas;     // [kAtMaxCtas]
  int* met;        // [kAtMaxCtas]
  float2* stats;   // [2 kAtMaxCtas, slot_rows]: (m, l)
  float* parts;    // [2 kAtMaxCtas, slot_rows, D]
  int main_ctas;
  int join_share;  // CTAs of the join per CTA of the first kernel
};
struct AtMaps {
  CUtensorMap k, v;
};

// Entries lo .. hi - 1 are those that tokens t0 .. t1 of a request see between them.
__device__ __forceinline__ void at_span(const PagedParams& p, int n, int len, int t0, int t1,
                                        int& lo, int& hi) {
  hi = p.causal ? min(max(len - n + t1 + 1, 0), len) : len;
  lo = p.window > 0 ? max(len - n + t0 - p.window + 1, 0) : 0;
}
__device__ __forceinline__ int at_token(const AtParams& a, int row) {
  return (int)(((unsigned long long)(uint32_t)row * a.magic) >> a.shift);
}
// Tiles of the unit of rows r0 .. and what one costs, in parts of the time of one that only its
// loads take (measured: 1.5 us with up to 64 rows, 1.9 with 68, 1.7 to 3 with 256).
struct AtSpan {
  int rows, lo, hi, tile0, tiles;
  int cost;  // of a tile
};
__device__ __forceinline__ AtSpan at_unit_span(const AtParams& a, int n, int len, int r0) {
  AtSpan s;
  s.rows = (int)min((long long)n * a.group - r0, (long long)kAtUnitRows);
  at_span(a.p, n, len, at_token(a, r0), at_token(a, r0 + s.rows - 1), s.lo, s.hi);
  s.tile0 = s.lo / kAtTile;
  s.tiles = s.hi > s.lo ? (s.hi + kAtTile - 1) / kAtTile - s.tile0 : 0;
  s.cost = s.rows <= kAtFewRows ? 4 : s.rows <= 2 * kAtFewRows ? 5 : 8;
  return s;
}
// How a unit is done.  Up to kAtFewRows rows: both streams have all rows and take the
// tiles in turn.  Else each stream has a part of the rows, the first at_first_rows of them.
__device__ __forceinline__ bool at_in_turn(const AtUnit& u) { return u.rows <= kAtFewRows; }
__device__ __forceinline__ bool at_few(const AtUnit& u) { return u.rows <= 2 * kAtFewRows; }
__device__ __forceinline__ int at_first_rows(const AtUnit& u) {
  return at_in_turn(u) ? u.rows : at_few(u) ? ((u.rows + 1) / 2 + 15) / 16 * 16 : kAtTile;
}

// How many tiles the values are behind the keys: as many scores are formed ahead.
__device__ __forceinline__ int at_lag(const AtUnit& u) {
  return at_in_turn(u) ? 4 : at_few(u) ? 2 : 0;
}

// The head of a unit's row among all rows' heads.
__device__ __forceinline__ long long at_head(const AtParams& a, int first, int h, int row) {
  const int t = at_token(a, row);
  return ((long long)first + t) * a.p.heads + h * a.group + (row - t * a.group);
}
// Cost of all units of a request and one key-value head (0: nothing to do, or out of range).
__device__ __forceinline__ long long at_head_cost(const AtParams& a, int b) {
  const int first = a.p.c.new_start[b], last = a.p.c.new_start[b + 1], len = a.p.c.kv_len[b];
  if (!request_ok(a.p, first, last, len)) return 0;
  const int n = last - first;
  long long cost = 0;
  for (int r0 = 0; r0 < n * a.group; r0 += kAtUnitRows) {
    const AtSpan s = at_unit_span(a, n, len, r0);
    cost += (long long)s.tiles * s.cost;
  }
  return cost;
}

// x * c / g, and the CTA whose share entry x of the line is in.
__device__ __forceinline__ long long at_border(long long x, int c, int g) {
  return x < (1 << 23) ? (int)x * c / g : x * c / g;
}
__device__ __forceinline__ int at_owner(long long x, long long total, int g) {
  return total < (1 << 23) ? (((int)x + 1) * g - 1) / (int)total
                           : (int)(((x + 1) * g - 1) / total);
}

// The share of the line that this CTA does: from start_off within request start_b on.
__device__ __forceinline__ void at_share(const AtParams& a, AtControl& ctl) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = a.p.c.B;
  const int each = (B + kAtThreads - 1) / kAtThreads;
  const int b0 = min(tid * each, B), b1 = min(b0 + each, B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += at_head_cost(a, b);
  const long long head = mine;
  mine *= a.p.c.kv_heads;
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) ctl.scan[warp] = upto;
  if (tid == 0) ctl.start_left = 0;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kAtThreads / 32; ++w) {
    if (w < warp) before += ctl.scan[w];
    total += ctl.scan[w];
  }
  before += upto - mine;
  const int c = blockIdx.x, G = gridDim.x;
  const long long start = at_border(total, c, G), end = at_border(total, c + 1, G);
  if (start < end && before <= start && start < before + mine) {
    for (int b = b0; b < b1; ++b) {
      const long long h = each == 1 ? head : at_head_cost(a, b), x = h * a.p.c.kv_heads;
      if (start < before + x) {
        ctl.start_b = b;
        ctl.start_off = start - before;
        ctl.start_left = end - start;
        ctl.start_line = start;
        ctl.start_cost = h;
        ctl.total = total;
        break;
      }
      before += x;
    }
  }
  __syncthreads();
}

// One thread hands the units of the CTA's share to the other warps, and notes the parts.
__device__ __forceinline__ bool at_plan(const AtParams& a, AtControl& ctl) {
  AtPart parts[2];
  parts[0].used = parts[1].used = 0;
  long long left = ctl.start_left, off = ctl.start_off, line = ctl.start_line;
  int slot = 0, round = 0;  // of the ring
  bool ok = true;
  auto publish = [&](const AtUnit& u) {
    if (round > 0 && !at_wait(&ctl.u_empty[slot], (round - 1) & 1, &ctl.abort_flag)) ok = false;
    if (!ok) return;
    ctl.unit[slot] = u;
    ctl.odd[slot].tiles = 0;
    mbar_arrive(&ctl.u_full[slot]);
    if (++slot == kAtUnits) {
      slot = 0;
      ++round;
    }
  };
  AtUnit u;
  u.bad = 0;
  for (int b = ctl.start_b; ok && left > 0 && b < a.p.c.B; ++b, off = 0) {
    const long long cost = b == ctl.start_b ? ctl.start_cost : at_head_cost(a, b);
    if (cost == 0) continue;
    u.b = b;
    u.first = a.p.c.new_start[b];
    u.n = a.p.c.new_start[b + 1] - u.first;
    u.len = a.p.c.kv_len[b];
    u.h = off == 0 ? 0 : off < INT32_MAX ? (int)off / (int)min(cost, (long long)INT32_MAX) : (int)(off / cost);
    off -= u.h * cost;
    for (; ok && left > 0 && u.h < a.p.c.kv_heads; ++u.h) {
      for (u.r0 = 0; ok && left > 0 && u.r0 < u.n * a.group; u.r0 += kAtUnitRows) {
        const AtSpan s = at_unit_span(a, u.n, u.len, u.r0);
        const long long c = (long long)s.tiles * s.cost;
        if (off >= c) {
          off -= c;
          continue;
        }
        const long long take = min(c - off, left);
        const int from = ((int)off + s.cost - 1) / s.cost;
        const int to = ((int)(off + take) + s.cost - 1) / s.cost;
        const long long unit_end = line + c - off;  // on the line
        left -= take;
        line += take;
        off = 0;
        if (to == from) continue;
        u.rows = s.rows;
        u.lo = s.lo;
        u.hi = s.hi;
        u.tile0 = s.tile0 + from;
        u.nt = to - from;
        u.slot = -1;
        if (from > 0 || to < s.tiles) {
          const int k = from > 0 ? 0 : 1;
          u.slot = 2 * blockIdx.x + k;
          parts[k] = {1, at_owner(unit_end - 1, ctl.total, gridDim.x), u.b, u.h, u.first, u.r0,
                      u.rows, 0};
        }
        publish(u);
      }
    }
  }
  u.b = -1;
  if (ok) publish(u);
  a.ctas[blockIdx.x].part[0] = parts[0];
  a.ctas[blockIdx.x].part[1] = parts[1];
  return ok;
}

// A warp's way through the planned units.
struct AtWalk {
  int slot = 0, round = 0;
  __device__ __forceinline__ bool next(AtControl& ctl, AtUnit& u, bool& ok) {
    if (!at_wait(&ctl.u_full[slot], round & 1, &ctl.abort_flag)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    u = ctl.unit[slot];
    return u.b >= 0;
  }
  __device__ __forceinline__ void done(AtControl& ctl) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl.u_empty[slot]);
    if (++slot == kAtUnits) {
      slot = 0;
      ++round;
    }
  }
};

// Stages of the ring in order.
template <int kStages>
struct AtRing {
  int stage = 0, round = 0;
  __device__ __forceinline__ void step() {
    if (++stage == kStages) {
      stage = 0;
      ++round;
    }
  }
};

// Keys and values of the tiles, in the order in which the products want them.
template <int D>
__device__ __forceinline__ bool at_produce(const AtParams& a, const AtMaps& maps, AtControl& ctl,
                                           uint32_t base) {
  using S = AtSizes<D>;
  const int lane = threadIdx.x & 31;
  const int P = a.p.c.page_size, box = min(P, kAtTile), per_tile = kAtTile / box;
  const int piece = lane % per_tile, half = lane / per_tile;
  const bool mine = half < D / 64;
  AtWalk walk;
  AtRing<S::kStages> ring;
  int loads = 0;
  bool ok = true;
  AtUnit u;
  // The previous kernel's stores (the append) before this one's asynchronous reads.
  asm volatile("fence.proxy.async;" ::: "memory");
  while (walk.next(ctl, u, ok)) {
    const int32_t* table = a.p.c.page_table + (size_t)u.b * a.p.c.max_pages;
    bool bad = false;
    // This lane's page of a tile: its number, -1 for one not to be loaded.  (In the place of one
    // outside the cache the first is: rows that do not see it go on as if it were any.)
    auto page_of = [&](int j) -> int {
      const int pos = (u.tile0 + j) * kAtTile + piece * box;
      if (j >= u.nt || !mine || pos >= u.hi || pos + box <= u.lo) return -1;
      const int id = table[pos >> a.page_bits];
      if (id >= 0 && id < a.p.c.num_pages) return id;
      bad = true;
      return 0;
    };
    auto load = [&](const CUtensorMap* map, int j, int id) {
      if (ring.round > 0 &&
          !at_wait(&ctl.empty[ring.stage], (ring.round - 1) & 1, &ctl.abort_flag))
        ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * box * 128;
      if (__any_sync(0xffffffffu, bad) && lane == 0) {  // known before the tile is
        *(volatile int*)&ctl.unit[walk.slot].bad = 1;
        ctl.bad_page = 1;
      }
      if (lane == 0) mbar_arrive_expect_tx(&ctl.full[ring.stage], bytes);
      __syncwarp();
      if (id >= 0)
        tma_load4(base + ring.stage * S::kTileBytes + half * (kAtTile * 128) +
                      piece * box * 128,
                  map, half * 64, ((u.tile0 + j) * kAtTile + piece * box) & (P - 1), u.h,
                  (int)SPEC_CHECKED(id, a.p.c.num_pages, kSitePage), &ctl.full[ring.stage]);
      ring.step();
      ++loads;
    };
    const int lag = at_lag(u);
    int id = page_of(0), old[4] = {-1, -1, -1, -1};  // of this tile and the last four
    for (int j = 0; ok && j < u.nt + lag; ++j) {
      const int next = page_of(j + 1);
      if (lag > 0 && j >= lag) load(&maps.v, j - lag, lag == 4 ? old[3] : old[1]);
      if (ok && j < u.nt) load(&maps.k, j, id);
      if (ok && lag == 0) load(&maps.v, j, id);
      old[3] = old[2];
      old[2] = old[1];
      old[1] = old[0];
      old[0] = id;
      id = next;
    }
    if (!ok) break;
    walk.done(ctl);
  }
  // The products' last arrivals come before the CTA ends; after a timeout, the loads that
  // are still on their way.
  int never = 0;
  for (int l = max(0, loads - S::kStages); l < loads; ++l) {
    if (ok) ok = at_wait(&ctl.empty[l % S::kStages], (l / S::kStages) & 1, &ctl.abort_flag);
    if (!ok) at_wait(&ctl.full[l % S::kStages], (l / S::kStages) & 1, &never);
  }
  return ok;
}

// Queries of a unit into shared memory, 128 rows to a buffer, swizzled as TMA would.
template <int D>
__device__ __forceinline__ bool at_load_queries(const AtParams& a, AtControl& ctl, uint32_t base) {
  using S = AtSizes<D>;
  const int lane = threadIdx.x & 31;
  AtWalk walk;
  int used = 0, few_units = 0;
  bool ok = true, was_few = false;
  AtUnit u;
  auto empty = [&](int l) {  // the buffer's l-th use is over
    if (l >= 0 && !at_wait(&ctl.q_empty[l & 1], (l >> 1) & 1, &ctl.abort_flag)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
  };
  // The f-th unit of few rows is over.  (A barrier each for odd and even ones: a phase is told from
  // the one before the last by nothing, and both of the last two units may end before either
  // is waited for, if the next one is planned late.  Unit f + 2 only starts behind this wait.)
  auto few_over = [&](int f) {
    if (ok && f >= 0 && !at_wait(&ctl.few_done[f & 1], (f >> 1) & 1, &ctl.abort_flag)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
  };
  while (walk.next(ctl, u, ok)) {
    // Buffers and weights of units of few rows lie over the others' buffers.
    const bool few = at_few(u);
    if (few) few_over(few_units++ - 2);
    if (few != was_few) {
      if (was_few) {
        few_over(few_units - 2);
        few_over(few_units - 1);
      }
      if (ok) empty(used - 1);
    }
    was_few = few;
    const int half = few ? S::kFewHalf : kAtTile * 128, size = few ? S::kFewQ : S::kTileBytes;
    const int first = at_first_rows(u);
    for (int r = 0; ok && r < u.rows; r += first, ++used) {
      empty(used - 2);
      if (!ok) break;
      const uint32_t dst = base + S::kQ + (used & 1) * size;
      const int rows = min(u.rows - r, first), chunks = rows * (D / 8);
      // (Columns of the product without a row are 0.)
      const int all = few ? (rows + 15) / 16 * 16 * (D / 8) : chunks;
      for (int i = chunks + lane; i < all; i += 32)
        st_shared16(dst + ((i % (D / 8)) >> 3) * half + i / (D / 8) * 128 + ((i & 7) << 4),
                    make_uint4(0, 0, 0, 0));
      for (int i = lane; i < chunks; i += 32) {
        const int row = i / (D / 8), e = i % (D / 8);
        const int at = u.r0 + r + row, t = at_token(a, at);
        const uint16_t* src = a.p.q + (u.first + t) * a.p.q_stride +
                              (u.h * a.group + at - t * a.group) * D + e * 8;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         dst + (e >> 3) * half + row * 128 + (((e ^ row) & 7) << 4)),
                     "l"(src)
                     : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.q_full[used & 1]);
    }
    if (!ok) break;
    walk.done(ctl);
  }
  if (ok) empty(used - 2);
  if (ok) empty(used - 1);
  return ok;
}

// Two bfloat16, those that are infinite or NaN as 0.
__device__ __forceinline__ uint32_t at_finite(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}

// 0 x + y of two bfloat16.
__device__ __forceinline__ uint32_t at_zero_times(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(y));
  return r;
}

// Values of a tile's entries from .. to - 1, which only some rows of the unit see: the others'
// weights for them are 0, and where one is not finite the product would be NaN.  Those are set
// to 0, and the rows that see them add them at the end.  A function of its own:
// two chunks of 4096 tokens take 1005 us with it inlined, 955 so, 912 if nothing is looked at.
template <int D>
__device__ __noinline__ void at_sift(AtControl& ctl, int slot, uint32_t v, int tile, int from,
                                     int to) {
  const int lane = threadIdx.x & 31;
  from = max(from - tile * kAtTile, 0);
  to = min(to - tile * kAtTile, kAtTile);
  if (from >= to) return;
  const int chunks = (to - from) * (D / 8);
  auto chunk = [&](int i) {
    const int row = from + i / (D / 8), e = i % (D / 8);
    return v + (e >> 3) * (kAtTile * 128) + row * 128 + (((e ^ row) & 7) << 4);
  };
  // (0 times them, added up, is NaN where one is.)
  uint32_t sum = 0;
  for (int first = lane; first < chunks; first += 32 * 8) {
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ld_shared16(chunk(min(first + 32 * i, chunks - 1)));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sum = at_zero_times(
          x[i].x, at_zero_times(x[i].y, at_zero_times(x[i].z, at_zero_times(x[i].w, sum))));
  }
  if (!__any_sync(0xffffffffu, (sum & 0x7fff7fffu) != 0)) return;
  for (int i = lane; i < chunks; i += 32) {
    const uint4 x = ld_shared16(chunk(i));
    const uint4 y = make_uint4(at_finite(x.x), at_finite(x.y), at_finite(x.z), at_finite(x.w));
    if (((x.x ^ y.x) | (x.y ^ y.y) | (x.z ^ y.z) | (x.w ^ y.w)) != 0) {
      const int row = from + i / (D / 8);
      st_shared16(chunk(i), y);
      atomicOr(&ctl.found_odd[row >> 5], 1u << (row & 31));
    }
  }
  __syncwarp();
  if (lane == 0) {
    AtOdd& odd = ctl.odd[slot];
    const int n = odd.tiles;
    odd.tile[n] = tile;
#pragma unroll
    for (int i = 0; i < kAtTile / 32; ++i) {
      odd.entries[n][i] = ctl.found_odd[i];
      ctl.found_odd[i] = 0;
    }
    odd.tiles = n + 1;
    __threadfence_block();
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// The products: S = Q K^T and O += P V, of the streams in turn.
template <int D>
__device__ __forceinline__ bool at_issue(const AtParams& a, AtControl& ctl, uint32_t base,
                                         uint32_t tmem) {
  using S = AtSizes<D>;
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kPv = mma_idesc(128, D, false, true);
  AtWalk walk;
  AtRing<S::kStages> ring;
  const uint32_t one = mma1_elect();
  int q_used = 0, p_count[2] = {0, 0}, half_count[2] = {0, 0};
  bool ok = true;
  AtUnit u = {};
  auto wait = [&](uint64_t* bar, int parity) {
    if (ok && !at_wait(bar, parity & 1, &ctl.abort_flag)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
    tmem_fence_after();
  };
  auto take = [&]() -> int {  // the next stage, filled
    const int s = ring.stage;
    wait(&ctl.full[s], ring.round);
    ring.step();
    return s;
  };
  // Whether every entry of a tile is seen; else the steps of 16 that are, in part.
  auto whole = [&](int j) {
    const int at = (u.tile0 + j) * kAtTile;
    return at >= u.lo && at + kAtTile <= u.hi;
  };
  auto first_step = [&](int j) { return max(u.lo - (u.tile0 + j) * kAtTile, 0) / 16; };
  auto last_step = [&](int j) {
    return (min(u.hi - (u.tile0 + j) * kAtTile, kAtTile) + 15) / 16;
  };
  // Few rows: S^T = K Q^T and O^T += V^T P^T, so that the product's 128 rows are entries and
  // the width, and its columns as many as the stream has rows.
  auto few_cols = [&](int s) {
    const int first = at_first_rows(u);
    return ((s == 0 || at_in_turn(u) ? first : u.rows - first) + 15) / 16 * 16;
  };
  auto scores_few = [&](int s, int buf, int stage, int set) {
    const uint32_t idesc = mma_idesc(128, few_cols(s), false, false);
    const uint32_t q = mma1_desc(base + S::kQ + buf * S::kFewQ, 0);
    const uint32_t k = mma1_desc(base + stage * S::kTileBytes, 0);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      mma1_f16(tmem + s * kAtTile + set * kAtFewRows,
               k + ((i >> 2) * (kAtTile * 128) + (i & 3) * 32) / 16,
               q + ((i >> 2) * S::kFewHalf + (i & 3) * 32) / 16, idesc, i > 0, one);
    mma1_commit(&ctl.s_full[s][set], one);
  };
  auto values_few = [&](int s, int stage, int j, bool first) {
    wait(&ctl.p_ready[s], p_count[s]++);
    if (!ok) return;
    const uint32_t idesc = mma_idesc(128, few_cols(s), true, true);
    // (Of a width of 64 the lower half of the product's rows is another tile's, and not used.)
    const uint32_t v = mma1_desc(base + stage * S::kTileBytes, kAtTile * 128);
    const uint32_t w = mma1_desc(base + S::kWeights + s * S::kFewWeights, 0);
    const uint32_t d = tmem + (2 + s) * kAtTile;
    if (whole(j)) {
#pragma unroll
      for (int i = 0; i < kAtTile / 16; ++i)
        mma1_f16(d, v + i * 128, w + i * 128, idesc, i > 0 || !first, one);
    } else {
      const int from = first_step(j), to = last_step(j);
      for (int i = from; i < to; ++i)
        mma1_f16(d, v + i * 128, w + i * 128, idesc, i > from || !first, one);
    }
    mma1_commit(&ctl.pv_done[s], one);
  };
  auto scores = [&](int s, int buf, int stage, int j) {
    const int cols = whole(j) ? kAtTile : last_step(j) * 16;
    const uint32_t idesc = mma_idesc(128, cols, false, false);
    const uint32_t q = mma1_desc(base + S::kQ + buf * S::kTileBytes, 0);
    const uint32_t k = mma1_desc(base + stage * S::kTileBytes, 0);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint32_t off = ((i >> 2) * (kAtTile * 128) + (i & 3) * 32) / 16;
      mma1_f16(tmem + s * kAtTile, q + off, k + off, idesc, i > 0, one);
    }
    mma1_commit(&ctl.s_full[s][0], one);
  };
  // Values of entries that nobody sees are set to 0 as far as the product reads them: their
  // weights are 0, but what lies there may not be finite.
  auto clear = [&](int stage, int j) {
    const int from = max(u.lo - (u.tile0 + j) * kAtTile, 0);
    const int to = min(u.hi - (u.tile0 + j) * kAtTile, kAtTile);
    if ((from | to) % 16 == 0) return;
    const uint32_t v = base + stage * S::kTileBytes;
    const int head = from % 16, tail = (16 - to % 16) % 16;
    for (int i = lane; i < (head + tail) * (D / 8); i += 32) {
      const int r = i / (D / 8), e = i % (D / 8);
      const int row = r < head ? from - head + r : to + r - head;
      st_shared16(v + (e >> 3) * (kAtTile * 128) + row * 128 + ((e & 7) << 4),
                  make_uint4(0, 0, 0, 0));
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  };
  // The first half of the weights is multiplied while the second is formed.
  auto values = [&](int s, int stage, int j, bool first) {
    const uint32_t v = mma1_desc(base + stage * S::kTileBytes, kAtTile * 128);
    const uint32_t p = tmem + s * kAtTile, d = tmem + (2 + s) * kAtTile;
    constexpr int kHalf = kAtTile / 32;
    const int from = first_step(j), to = last_step(j);
    wait(&ctl.p_half[s], half_count[s]++);
    if (!ok) return;
    if (whole(j)) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i)
        mma1_f16_ta(d, p + i * 8, v + i * 128, kPv, i > 0 || !first, one);
    } else {
      for (int i = from; i < min(to, kHalf); ++i)
        mma1_f16_ta(d, p + i * 8, v + i * 128, kPv, i > from || !first, one);
    }
    wait(&ctl.p_ready[s], p_count[s]++);
    if (!ok) return;
    if (whole(j)) {
#pragma unroll
      for (int i = kHalf; i < 2 * kHalf; ++i)
        mma1_f16_ta(d, p + i * 8, v + i * 128, kPv, 1, one);
    } else {
      for (int i = max(from, kHalf); i < to; ++i)
        mma1_f16_ta(d, p + i * 8, v + i * 128, kPv, i > from || !first, one);
    }
  };
  int lo_all = 0, hi_all = 0;  // entries that all rows of the unit see
  auto sift = [&](int stage, int j) {
    const int tile = u.tile0 + j;
    if (tile * kAtTile < lo_all)
      at_sift<D>(ctl, walk.slot, base + stage * S::kTileBytes, tile, u.lo, lo_all);
    if ((tile + 1) * kAtTile > hi_all)
      at_sift<D>(ctl, walk.slot, base + stage * S::kTileBytes, tile, hi_all, u.hi);
  };
  auto commit = [&](uint64_t* bar) { mma1_commit(bar, one); };
  while (ok && walk.next(ctl, u, ok)) {
    int unused;
    at_span(a.p, u.n, u.len, 0, at_token(a, u.r0), unused, hi_all);
    at_span(a.p, u.n, u.len, at_token(a, u.r0 + u.rows - 1), 0, lo_all, unused);
    const int buf = q_used & 1;
    wait(&ctl.q_full[buf], q_used >> 1);
    ++q_used;
    if (!at_few(u)) {
      wait(&ctl.q_full[buf ^ 1], q_used >> 1);
      ++q_used;
      int k = ok ? take() : 0;
      if (!ok) break;
      scores(0, buf, k, 0);
      scores(1, buf ^ 1, k, 0);
      commit(&ctl.empty[k]);
      for (int j = 0; ok && j < u.nt; ++j) {
        if (j + 1 == u.nt) {  // the last scores are under way
          commit(&ctl.q_empty[buf]);
          commit(&ctl.q_empty[buf ^ 1]);
        }
        const int v = take();
        if (!ok) break;
        clear(v, j);
        sift(v, j);
        values(0, v, j, j == 0);
        if (!ok) break;
        if (j + 1 < u.nt) {
          k = take();
          if (!ok) break;
          scores(0, buf, k, j + 1);
        } else {
          commit(&ctl.o_full[0]);
        }
        values(1, v, j, j == 0);
        if (!ok) break;
        commit(&ctl.empty[v]);
        if (j + 1 < u.nt) {
          scores(1, buf ^ 1, k, j + 1);
          commit(&ctl.empty[k]);
        } else {
          commit(&ctl.o_full[1]);
        }
      }
    } else {
      // Each stream's next scores are formed before its last ones are weights: the softmax
      // waits for neither product.
      const bool turn = at_in_turn(u);
      const int lag = at_lag(u);
      if (!turn) {
        wait(&ctl.q_full[buf ^ 1], q_used >> 1);
        ++q_used;
      }
      for (int j = 0; ok && j < u.nt + lag; ++j) {
        if (j >= lag) {
          const int v = take();
          if (!ok) break;
          clear(v, j - lag);
          sift(v, j - lag);
          if (turn) {
            values_few(j & 1, v, j - lag, j - lag < 2);
          } else {
            values_few(0, v, j - lag, j == lag);
            if (ok) values_few(1, v, j - lag, j == lag);
          }
          if (!ok) break;
          commit(&ctl.empty[v]);
        }
        if (j < u.nt) {
          const int k = take();
          if (!ok) break;
          if (turn) {
            scores_few(j & 1, buf, k, (j >> 1) & 1);
          } else {
            scores_few(0, buf, k, j & 1);
            scores_few(1, buf ^ 1, k, j & 1);
          }
          commit(&ctl.empty[k]);
        }
        if (j + 1 == u.nt) {
          commit(&ctl.q_empty[buf]);
          if (!turn) commit(&ctl.q_empty[buf ^ 1]);
        }
      }
      if (!ok) break;
      commit(&ctl.o_full[0]);
      commit(&ctl.o_full[1]);
    }
    walk.done(ctl);
  }
  return ok;
}

// Whether a row sees a page outside the cache among the unit's tiles done here.
__device__ __noinline__ bool at_row_bad(const AtParams& a, const AtControl& ctl, int slot, int r) {
  const AtUnit& u = ctl.unit[slot];  // (not a copy: a caller's registers)
  const int t = at_token(a, u.r0 + r);
  int lo, hi;
  at_span(a.p, u.n, u.len, t, t, lo, hi);
  lo = max(lo, u.tile0 * kAtTile);
  hi = min(hi, (u.tile0 + u.nt) * kAtTile);
  const int32_t* table = a.p.c.page_table + (size_t)u.b * a.p.c.max_pages;
  for (int i = lo >> a.page_bits; lo < hi && i <= (hi - 1) >> a.page_bits; ++i)
    if (table[i] < 0 || table[i] >= a.p.c.num_pages) return true;
  return false;
}

// The values that were set to 0 join a row's results of dimensions e0 .. e1 - 1, which this
// thread has written.  (The row's weights for them are above 0: a sum that one enters is it.)
template <int D>
__device__ __noinline__ void at_join_odd(const AtParams& a, const AtControl& ctl, int slot, int r,
                                         int e0, int e1) {
  const AtUnit& u = ctl.unit[slot];
  const AtOdd& odd = ctl.odd[slot];
  const spec_paged_cache_t& c = a.p.c;
  int lo, hi;
  const int t = at_token(a, u.r0 + r);
  at_span(a.p, u.n, u.len, t, t, lo, hi);
  uint16_t* out = a.p.out + at_head(a, u.first, u.h, u.r0 + r) * D;
  float* part = a.parts + ((size_t)u.slot * a.slot_rows + r) * D;
  for (int i = 0; i < odd.tiles; ++i)
    for (int w = 0; w < kAtTile / 32; ++w)
      for (uint32_t bits = odd.entries[i][w]; bits != 0; bits &= bits - 1) {
        const int at = odd.tile[i] * kAtTile + w * 32 + __ffs(bits) - 1;
        if (at < lo || at >= hi) continue;
        const int page = c.page_table[(size_t)u.b * c.max_pages + (at >> a.page_bits)];
        const uint16_t* x = static_cast<const uint16_t*>(c.v_cache) + page * c.v_page +
                            (at & (c.page_size - 1)) * c.v_slot + u.h * c.v_head;
        for (int e = e0; e < e1; ++e) {
          if ((x[e] & 0x7f80) != 0x7f80) continue;
          const float v = __uint_as_float((uint32_t)x[e] << 16);
          if (u.slot >= 0) {
            part[e] += v;
          } else {
            const float y = __uint_as_float((uint32_t)out[e] << 16);
            out[e] = (uint16_t)(pack_bf16(y + v, 0.0f) & 0xffff);
          }
        }
      }
}

// 32 results of a row, scaled.
template <int kWords>
__device__ __forceinline__ void at_store_row(uint16_t* out, const float (&x)[kWords]) {
#pragma unroll
  for (int c = 0; c < kWords; c += 8)
    *reinterpret_cast<uint4*>(out + c) = pack_vec<uint16_t>(x + c);
}

// A softmax warp: which lanes of tensor memory it has, and how often it has waited for what.
struct AtSoft {
  int s, quarter;  // the stream; the warp's 32 lanes
  int tiles, units, few_units, meets, votes;
  int sets[2], weights;  // scores of either set, weights of units of few rows
  bool ok;
  __device__ __forceinline__ void wait(AtControl& ctl, uint64_t* bar, int parity) {
    if (!at_wait(bar, parity & 1, &ctl.abort_flag)) ok = false;
    ok = __all_sync(0xffffffffu, ok);
    tmem_fence_after();
  }
  // All warps of both streams, or of one: barriers whose waits are bounded.
  __device__ __forceinline__ void meet(AtControl& ctl) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl.meet);
    wait(ctl, &ctl.meet, meets++);
  }
  __device__ __forceinline__ void vote(AtControl& ctl) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl.vote[s]);
    wait(ctl, &ctl.vote[s], votes++);
  }
};

// Units of many rows: a thread has a row of its stream's half.
template <int D>
__device__ __forceinline__ void at_unit_rows(const AtParams& a, AtControl& ctl, uint32_t tmem,
                                             AtSoft& w, const AtUnit& u, int slot) {
  const int lane = threadIdx.x & 31, s = w.s, row = w.quarter * 32 + lane;
  const uint32_t lanes = (uint32_t)(w.quarter * 32) << 16;
  const uint32_t scores = tmem + s * kAtTile + lanes, sums = tmem + 2 * kAtTile + lanes;
  const float nan = __int_as_float(0x7fc00000);
  const int r = s * kAtTile + row;
  const bool live = r < u.rows;
  const bool dead = r - lane >= u.rows;  // the whole warp
  int lo, hi;
  {
    const int t = at_token(a, u.r0 + r);
    at_span(a.p, u.n, u.len, t, t, lo, hi);
    if (!live) hi = 0;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = 0; j < u.nt; ++j, ++w.tiles) {
    w.wait(ctl, &ctl.s_full[s][0], w.sets[0]++);
    if (!w.ok) return;
    if (!dead) {
      // Twice through the scores, 64 registers of them at a time: for the maximum, and for
      // the weights.
      const int at = (u.tile0 + j) * kAtTile;
      const bool edge = !__all_sync(0xffffffffu, lo <= at && at + kAtTile <= hi);
      const int from = lo - at, to = hi - at;
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int h = 0; h < kAtTile; h += 64) {
        uint32_t x[64];
        tmem_issue32(scores + h, x);
        tmem_issue32(scores + h + 32, x + 32);
        tmem_wait_load(x);
        if (edge) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (h + c < from || h + c >= to) x[c] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int c = 0; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(x[c]));
      }
      const float top =
          __fmul_rn(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), a.scale2);
      float fix = 1.0f;
      if (m == -INFINITY) {
        m = top;  // no sums yet
      } else if (top > m + kAtRaise) {
        fix = ex2(__fsub_rn(m, top));
        m = top;
      }
      if (__any_sync(0xffffffffu, fix != 1.0f)) {
        // (All earlier products are done: this tile's scores came behind them.)
        l = __fmul_rn(l, fix);
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_issue32(sums + s * kAtTile + c, o);
          tmem_wait_load(o);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), fix));
          tmem_store32(sums + s * kAtTile + c, o);
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      const float2 sc = make_float2(a.scale2, a.scale2), mm = make_float2(-ref, -ref);
      float2 add[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) add[c] = make_float2(0.0f, 0.0f);
      // (The weights take the first half of the columns, those of scores read already.)
#pragma unroll
      for (int h = 0; h < kAtTile; h += 64) {
        uint32_t x[64];
        tmem_issue32(scores + h, x);
        tmem_issue32(scores + h + 32, x + 32);
        tmem_wait_load(x);
        if (edge) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (h + c < from || h + c >= to) x[c] = 0xff800000u;
        }
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 e = ex2x2(
              f32x2_fma(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc, mm));
          add[(c >> 1) & 3] = f32x2_add(add[(c >> 1) & 3], e);
          x[c >> 1] = pack_bf16(e.x, e.y);
        }
        tmem_store32(scores + h / 2, x);
        if (h == 0) {
          tmem_wait_store();
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.p_half[s]);
        }
      }
      const float2 t = f32x2_add(f32x2_add(add[0], add[1]), f32x2_add(add[2], add[3]));
      l = __fadd_rn(l, __fadd_rn(t.x, t.y));
      tmem_wait_store();
    } else if (lane == 0) {
      mbar_arrive(&ctl.p_half[s]);
    }
    tmem_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.p_ready[s]);
  }
  if (!w.ok) return;
  w.wait(ctl, &ctl.o_full[s], w.units++);
  if (!w.ok) return;
  const bool bad = *(volatile int*)&ctl.unit[slot].bad && live && at_row_bad(a, ctl, slot, r);
  if (bad) l = nan;
  if (!dead) {
    const bool whole = u.slot < 0;
    const float inv = whole ? (l == 0.0f ? 0.0f : __fdividef(1.0f, l)) : 1.0f;
    const long long head = at_head(a, u.first, u.h, u.r0 + r);
    const int slot_row = u.slot * a.slot_rows + r;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      tmem_issue32(sums + s * kAtTile + c, o);
      tmem_wait_load(o);
      float y[32];
#pragma unroll
      for (int e = 0; e < 32; ++e)
        y[e] = bad ? nan : l == 0.0f ? 0.0f : __fmul_rn(__uint_as_float(o[e]), inv);
      if (live) {
        if (whole) {
          at_store_row<32>(a.p.out + head * D + c, y);
        } else {
          float4* dst = reinterpret_cast<float4*>(a.parts + (size_t)slot_row * D + c);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        }
      }
    }
    if (live && !bad && *(volatile int*)&ctl.odd[slot].tiles > 0)
      at_join_odd<D>(a, ctl, slot, r, 0, D);
    if (live) {
      if (!whole) a.stats[slot_row] = make_float2(m, l);
      else if (a.p.lse != nullptr)
        a.p.lse[head] = __fmul_rn(__fadd_rn(m, log2f(l)), kLn2f);
    }
  }
  tmem_fence_before();
}

// 16 columns of the warp's 32 lanes without the wait, and 16 written.
__device__ __forceinline__ void at_issue16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void at_store16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// Units of few rows: a thread has an entry of the tile in the scores, an element of the
// width in the sums, and all rows of either; so a few rows keep all threads busy, where a
// row per thread leaves most of them idle and the others with 128 scores each.
// The maximum in use is the stream's, in shared memory: the warps vote on whether a score
// passes one by more than 2^8, and only then look for the new ones.
template <int D>
__device__ __forceinline__ void at_unit_few(const AtParams& a, AtControl& ctl,
                                            unsigned char* smem, uint32_t tmem, AtSoft& w,
                                            const AtUnit& u, int slot) {
  using S = AtSizes<D>;
  constexpr int kChunks = kAtFewRows / 16;
  const int lane = threadIdx.x & 31, s = w.s, row = w.quarter * 32 + lane;
  const bool turn = at_in_turn(u);
  // The stream's rows.
  const int r0 = u.r0 + (turn || s == 0 ? 0 : at_first_rows(u));
  const int rows = turn || s == 0 ? at_first_rows(u) : u.rows - at_first_rows(u);
  const int chunks = (rows + 15) / 16;
  const uint32_t lanes = (uint32_t)(w.quarter * 32) << 16;
  const uint32_t all_scores = tmem + s * kAtTile + lanes, sums = tmem + 2 * kAtTile + lanes;
  const float nan = __int_as_float(0x7fc00000);
  // This entry's line of weights: 8 rows to 16 bytes, swizzled by the entry.
  unsigned char* store = smem + S::kWeights + s * S::kFewWeights;
  const uint32_t line = smem_addr(store) + row * 128, turnover = (uint32_t)(row & 7) << 4;
  // While no weights are there, what the stream's four warps have found for each row.
  float* found[2] = {reinterpret_cast<float*>(smem + S::kWeights),
                     reinterpret_cast<float*>(smem + S::kWeights + S::kFewWeights)};
  // Entries that every row sees.
  int lo_all, hi_all, unused;
  at_span(a.p, u.n, u.len, 0, at_token(a, r0), unused, hi_all);
  at_span(a.p, u.n, u.len, at_token(a, r0 + rows - 1), 0, lo_all, unused);
  float2 l[kAtFewRows / 2];
#pragma unroll
  for (int c = 0; c < kAtFewRows / 2; ++c) l[c] = make_float2(0.0f, 0.0f);
  if (row < kAtFewRows) {
    ctl.above[s][row] = row < rows ? INFINITY : -FLT_MAX;  // (no row: no weight, no vote)
    ctl.ref[s][row] = row < rows ? 0.0f : -FLT_MAX;
  }
  const float2 sc = make_float2(a.scale2, a.scale2);
  bool first = true;
  for (int j = turn ? s : 0; j < u.nt; j += turn ? 2 : 1, ++w.tiles, first = false) {
    const int set = (turn ? j >> 1 : j) & 1;
    const uint32_t scores = all_scores + set * kAtFewRows;
    w.wait(ctl, &ctl.s_full[s][set], w.sets[set]++);
    if (!w.ok) return;
    const int at = (u.tile0 + j) * kAtTile;
    if (at < lo_all || at + kAtTile > hi_all) {
      // Some row does not see all of the tile: what it does not see becomes -inf.
      const int pos = at + row;
#pragma unroll 1
      for (int c = 0; c < chunks * 16; c += 16) {
        uint32_t x[16];
        at_issue16(scores + c, x);
        tmem_wait_load(x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          int lo, hi;
          const int t = at_token(a, r0 + c + e);
          at_span(a.p, u.n, u.len, t, t, lo, hi);
          if (pos < lo || pos >= hi) x[e] = 0xff800000u;
        }
        at_store16(scores + c, x);
      }
      tmem_wait_store();
    }
    bool raise = first;
    if (!first) {
      float most = -INFINITY;
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        if (q >= chunks) break;
        uint32_t x[16];
        at_issue16(scores + q * 16, x);
        tmem_wait_load(x);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&ctl.above[s][q * 16 + e]);
          const float2 y0 = f32x2_fma(
              make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), sc, make_float2(m.x, m.y));
          const float2 y1 =
              f32x2_fma(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), sc,
                        make_float2(m.z, m.w));
          most = fmaxf(fmaxf(fmaxf(most, y0.x), fmaxf(y0.y, y1.x)), y1.y);
        }
      }
      raise = __any_sync(0xffffffffu, most > kAtRaise);
      // (The word of two tiles ago is read by all before any comes here again.)
      if (raise && lane == 0) *(volatile int*)&ctl.raise[s][w.tiles & 1] = w.tiles;
      w.vote(ctl);
      if (!w.ok) return;
      raise = *(volatile int*)&ctl.raise[s][w.tiles & 1] == w.tiles;
    }
    // The last tile's product has read the weights, and its sums are there.
    if (!first) w.wait(ctl, &ctl.pv_done[s], w.weights - 1);
    ++w.weights;
    if (!w.ok) return;
    if (raise) {
#pragma unroll 1
      for (int c = 0; c < chunks * 16; c += 16) {
        uint32_t x[16];
        at_issue16(scores + c, x);
        tmem_wait_load(x);
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float y = __fmul_rn(__uint_as_float(x[e]), a.scale2);
          const uint32_t most = __reduce_max_sync(0xffffffffu, y != y ? 0u : order_bits(y));
          if (lane == e) top = from_order_bits(most);
        }
        if (lane < 16) found[s][w.quarter * kAtFewRows + c + lane] = top;
      }
      w.vote(ctl);
      if (!w.ok) return;
      if (row < kAtFewRows) {
        float fix = 1.0f;
        if (row < rows) {
          const float m = -ctl.above[s][row];
          const float top =
              fmaxf(fmaxf(found[s][row], found[s][kAtFewRows + row]),
                    fmaxf(found[s][2 * kAtFewRows + row], found[s][3 * kAtFewRows + row]));
          if (m == -INFINITY || top > m + kAtRaise) {
            if (m != -INFINITY) fix = ex2(__fsub_rn(m, top));
            ctl.above[s][row] = -top;
            ctl.ref[s][row] = top == -INFINITY ? 0.0f : -top;
          }
        }
        ctl.fix[s][row] = fix;
      }
      w.vote(ctl);
      if (!w.ok) return;
      if (!first) {
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
          if (q >= chunks) break;
          uint32_t o[16];
          at_issue16(sums + s * kAtTile + q * 16, o);
          tmem_wait_load(o);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float f0 = ctl.fix[s][q * 16 + e], f1 = ctl.fix[s][q * 16 + e + 1];
            l[q * 8 + e / 2] = f32x2_mul(l[q * 8 + e / 2], make_float2(f0, f1));
            o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), f0));
            o[e + 1] = __float_as_uint(__fmul_rn(__uint_as_float(o[e + 1]), f1));
          }
          at_store16(sums + s * kAtTile + q * 16, o);
        }
        tmem_wait_store();
      }
    }
#pragma unroll
    for (int q = 0; q < kChunks; ++q) {
      if (q >= chunks) break;
      uint32_t x[16];
      at_issue16(scores + q * 16, x);
      tmem_wait_load(x);
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 m = *reinterpret_cast<const float4*>(&ctl.ref[s][q * 16 + e]);
        const float2 p0 = ex2x2(f32x2_fma(
            make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), sc, make_float2(m.x, m.y)));
        const float2 p1 =
            ex2x2(f32x2_fma(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), sc,
                            make_float2(m.z, m.w)));
        l[q * 8 + e / 2] = f32x2_add(l[q * 8 + e / 2], p0);
        l[q * 8 + e / 2 + 1] = f32x2_add(l[q * 8 + e / 2 + 1], p1);
        x[e / 2] = pack_bf16(p0.x, p0.y);
        x[e / 2 + 1] = pack_bf16(p1.x, p1.y);
      }
      st_shared16(line + ((uint32_t)(q * 32) ^ turnover), make_uint4(x[0], x[1], x[2], x[3]));
      st_shared16(line + ((uint32_t)(q * 32 + 16) ^ turnover), make_uint4(x[4], x[5], x[6], x[7]));
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tmem_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.p_ready[s]);
  }
  w.wait(ctl, &ctl.o_full[s], w.units++);
  if (!w.ok) return;
  // (No product reads weights any more.)  The sums of the weights, over the 32 lanes: each
  // exchange leaves a lane half of the columns, in the end the one of its number.
#pragma unroll
  for (int g = 0; g < kAtFewRows; g += 32) {
    if (g >= rows) break;
    float y[32];
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      y[c] = l[(g + c) / 2].x;
      y[c + 1] = l[(g + c) / 2].y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int c = 0; c < o; ++c) {
        const float mine = up ? y[c + o] : y[c], theirs = up ? y[c] : y[c + o];
        y[c] = __fadd_rn(mine, __shfl_xor_sync(0xffffffffu, theirs, o));
      }
    }
    found[s][w.quarter * kAtFewRows + g + lane] = y[0];
  }
  const bool bad = *(volatile int*)&ctl.unit[slot].bad, whole = u.slot < 0;
  if (turn) w.meet(ctl);
  else w.vote(ctl);
  if (!w.ok) return;
  // What either stream's sums are multiplied by, a thread per row; where both have the same
  // rows, they are joined.
  if (row < rows) {
    const float m0 = -ctl.above[turn ? 0 : s][row], m1 = turn ? -ctl.above[1][row] : -INFINITY;
    const float top = fmaxf(m0, m1), ref = top == -INFINITY ? 0.0f : top;
    const float w0 = ex2(__fsub_rn(m0, ref)), w1 = ex2(__fsub_rn(m1, ref));
    // (A weight of 0 is no reason to leave a stream out: its sums may hold what is not finite.)
    float all = 0.0f;
    if (m0 != -INFINITY) {
      const float* f = found[turn ? 0 : s] + row;
      all = __fadd_rn(__fadd_rn(f[0], f[kAtFewRows]), __fadd_rn(f[2 * kAtFewRows], f[3 * kAtFewRows]));
      all = __fmul_rn(all, w0);
    }
    if (m1 != -INFINITY) {
      const float* f = found[1] + row;
      const float l1 =
          __fadd_rn(__fadd_rn(f[0], f[kAtFewRows]), __fadd_rn(f[2 * kAtFewRows], f[3 * kAtFewRows]));
      all = fmaf(l1, w1, all);
    }
    const bool bad_row = bad && at_row_bad(a, ctl, slot, r0 - u.r0 + row);
    if (bad_row) all = nan;
    const float inv = whole ? (all == 0.0f ? 0.0f : __fdividef(1.0f, all)) : 1.0f;
    // (Below 0: a stream in which the row has seen nothing, and whose sums may be anything.)
    const bool mine = (turn && s == 1 ? m1 : m0) != -INFINITY;
    ctl.fix[s][row] = bad_row ? nan : mine ? __fmul_rn(turn && s == 1 ? w1 : w0, inv) : -1.0f;
    if (!turn || s == 0) {
      if (!whole)
        a.stats[(size_t)u.slot * a.slot_rows + r0 - u.r0 + row] = make_float2(top, all);
      else if (a.p.lse != nullptr)
        a.p.lse[at_head(a, u.first, u.h, r0 + row)] = __fmul_rn(__fadd_rn(top, log2f(all)), kLn2f);
    }
  }
  if (turn) w.meet(ctl);
  else w.vote(ctl);
  if (!w.ok) return;
  // (In turn: the streams' threads share the chunks of 16 rows.)
#pragma unroll 1
  for (int c = turn ? s * 16 : 0; c < rows; c += turn ? 32 : 16) {
    uint32_t o0[16], o1[16];
    at_issue16(sums + (turn ? 0 : s * kAtTile) + c, o0);
    at_issue16(sums + kAtTile + c, o1);
    tmem_wait_load(o0);
    tmem_wait_load(o1);
    if (row >= D) continue;  // (a width of 64: the product's other rows)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int r = c + e;
      if (r >= rows) break;
      const float w0 = ctl.fix[turn ? 0 : s][r], w1 = turn ? ctl.fix[1][r] : -1.0f;
      const float y = __fadd_rn(w0 < 0.0f ? 0.0f : __fmul_rn(__uint_as_float(o0[e]), w0),
                                w1 < 0.0f ? 0.0f : __fmul_rn(__uint_as_float(o1[e]), w1));
      if (whole)
        a.p.out[at_head(a, u.first, u.h, r0 + r) * D + row] =
            (uint16_t)(pack_bf16(y, 0.0f) & 0xffff);
      else
        a.parts[((size_t)u.slot * a.slot_rows + r0 - u.r0 + r) * D + row] = y;
    }
  }
  if (row < D && *(volatile int*)&ctl.odd[slot].tiles > 0)
    for (int c = turn ? s * 16 : 0; c < rows; c += turn ? 32 : 16)
      for (int r = c; r < min(c + 16, rows); ++r)
        if (ctl.fix[turn ? 0 : s][r] == ctl.fix[turn ? 0 : s][r])  // (else it is NaN already)
          at_join_odd<D>(a, ctl, slot, r0 - u.r0 + r, row, row + 1);
  tmem_fence_before();
  // Neither stream's next products may write sums that the other still reads, nor queries
  // what is in the weights' place.
  if (turn) w.meet(ctl);
  else w.vote(ctl);
  if (w.ok && w.quarter == 0 && lane == 0) mbar_arrive(&ctl.few_done[w.few_units & 1]);
  ++w.few_units;
}

template <int D>
__device__ __forceinline__ bool at_softmax(const AtParams& a, AtControl& ctl, unsigned char* smem,
                                           uint32_t tmem) {
  const int warp = threadIdx.x >> 5;
  AtWalk walk;
  AtSoft w = {};
  w.s = (warp - kAtSoftmax) >> 2;
  w.quarter = warp & 3;
  w.ok = true;
  AtUnit u;
  while (walk.next(ctl, u, w.ok)) {
    if (at_few(u)) at_unit_few<D>(a, ctl, smem, tmem, w, u, walk.slot);
    else at_unit_rows<D>(a, ctl, tmem, w, u, walk.slot);
    if (!w.ok) break;
    walk.done(ctl);
  }
  return w.ok;
}

template <int D>
__global__ void __launch_bounds__(kAtThreads, 1)
    paged_attention_kernel(const __grid_constant__ AtMaps maps, const __grid_constant__ AtParams a) {
  using S = AtSizes<D>;
  extern __shared__ __align__(1024) unsigned char at_smem_raw[];
  const uint32_t base = smem_addr(at_smem_raw);
  AtControl& ctl =
      *reinterpret_cast<AtControl*>(at_smem_raw + S::kTotal);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i][0], 1);
      mbar_init(&ctl.s_full[i][1], 1);
      mbar_init(&ctl.pv_done[i], 1);
      mbar_init(&ctl.p_ready[i], 4);
      mbar_init(&ctl.p_half[i], 4);
      mbar_init(&ctl.o_full[i], 1);
      mbar_init(&ctl.q_full[i], 1);
      mbar_init(&ctl.q_empty[i], 1);
    }
    for (int i = 0; i < kAtUnits; ++i) {
      mbar_init(&ctl.u_full[i], 1);
      mbar_init(&ctl.u_empty[i], kAtReaders);
    }
    mbar_init(&ctl.meet, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.few_done[i], 2);
      mbar_init(&ctl.vote[i], 4);
      ctl.raise[i][0] = ctl.raise[i][1] = 0;
    }
    ctl.abort_flag = ctl.bad_page = 0;
    for (int i = 0; i < kAtTile / 32; ++i) ctl.found_odd[i] = 0;
    fence_mbar_init();
  }
  if (warp == kAtIssuer) tmem1_alloc(&ctl.tmem, 512);
  if (warp == kAtProducer && lane < 2) tma_prefetch_map(lane ? &maps.v : &maps.k);
  pdl_wait();
  pdl_launch_dependents();
  tmem_fence_before();
  at_share(a, ctl);
  tmem_fence_after();
  const uint32_t tmem = ctl.tmem;
  bool ok = (base & 1023) == 0;  // (the tiles' swizzle counts from there)
  if (ok) {
    if (warp == kAtProducer) ok = at_produce<D>(a, maps, ctl, base);
    else if (warp == kAtIssuer) ok = at_issue<D>(a, ctl, base, tmem);
    else if (warp == kAtQueries) ok = at_load_queries<D>(a, ctl, base);
    else if (warp >= kAtSoftmax) ok = at_softmax<D>(a, ctl, at_smem_raw, tmem);
    else if (lane == 0) ok = at_plan(a, ctl);
  }
  if (!ok) *(volatile int*)&ctl.abort_flag = 1;
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (threadIdx.x == 0) {
    a.met[blockIdx.x] = (ctl.abort_flag ? kAtLate : 0) | (ctl.bad_page ? kAtBadPage : 0);
  }
  if (warp == kAtIssuer) tmem1_free(tmem, 512);
}

// Joins the parts of units that lie across CTAs' borders, one warp per row; then the
// rows that belong to no unit: of requests out of range (NaN), and those that see nothing.
// The first CTA writes the workspace's header.
constexpr int kAtJoinThreads = 256;

template <int D>
__device__ __forceinline__ void at_fill(const AtParams& a, long long row, float x, float lse,
                                        int from, int step) {
  const uint32_t w = pack_bf16(x, x);
  uint4* out = reinterpret_cast<uint4*>(a.p.out + row * a.p.heads * D);
  for (int i = from; i < a.p.heads * (D / 8); i += step) out[i] = make_uint4(w, w, w, w);
  if (a.p.lse != nullptr)
    for (int i = from; i < a.p.heads; i += step) a.p.lse[row * a.p.heads + i] = lse;
}

// The rows of a unit that lies across CTAs, one warp each.
template <int D>
__device__ __forceinline__ void at_join(const AtParams& a, const AtPart& u, int c, int share) {
  const PagedParams& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = u.end - c + 1;  // CTAs c .. end have parts (but for such with none)
  for (int r = share * (kAtJoinThreads / 32) + warp; r < u.rows;
       r += a.join_share * (kAtJoinThreads / 32)) {
    // 32 parts at a time, a lane the statistics of each; of further ones the sums so far are
    // rescaled.
    float m = -INFINITY, l = 0.0f, x[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) x[e] = 0.0f;
    for (int i0 = 0; i0 < parts; i0 += 32) {
      const int i = i0 + lane;
      float2 st = make_float2(-INFINITY, 0.0f);
      if (i < parts) {
        // (Of a CTA without a part nothing counts; both loads go together.)
        const int used = i == 0 ? 1 : a.ctas[c + i].part[0].used;
        const float2 x = a.stats[(size_t)(2 * (c + i) + (i == 0 ? 1 : 0)) * a.slot_rows + r];
        if (used) st = x;
      }
      float top = st.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmaxf(top, m);
      const float ref = top == -INFINITY ? 0.0f : top;
      const float fix = ex2(__fsub_rn(m, ref));
      m = top;
      const float w = ex2(__fsub_rn(st.x, ref));
      // (Parts of weight 0 as well: their sums may hold what is not finite.  A NaN in the
      // statistics marks one in which the row sees a page outside the cache.)
      const bool counts = st.x != -INFINITY || st.y != st.y;
      float add = counts ? __fmul_rn(st.y, w) : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) add = __fadd_rn(add, __shfl_xor_sync(0xffffffffu, add, o));
      l = fmaf(l, fix, add);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) x[e] = __fmul_rn(x[e], fix);
      uint32_t some = __ballot_sync(0xffffffffu, counts);
      while (some != 0) {
        // Eight parts' sums at a time: their loads go together.
        float v[8][D / 32], wk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int j = some != 0 ? __ffs(some) - 1 : -1;
          some &= some - 1;
          wk[k] = __shfl_sync(0xffffffffu, w, max(j, 0));
          const float* src =
              a.parts +
              ((size_t)(2 * (c + i0 + j) + (i0 + j == 0 ? 1 : 0)) * a.slot_rows + r) * D;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) v[k][e] = j >= 0 ? src[e * 32 + lane] : 0.0f;
          if (j < 0) wk[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < D / 32; ++e) x[e] = fmaf(v[k][e], wk[k], x[e]);
      }
    }
    const long long head = at_head(a, u.first, u.h, u.r0 + r);
    const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
      p.out[head * D + e * 32 + lane] =
          (uint16_t)(pack_bf16(l == 0.0f ? 0.0f : __fmul_rn(x[e], inv), 0.0f) & 0xffff);
    if (lane == 0 && p.lse != nullptr)
      p.lse[head] = __fmul_rn(__fadd_rn(m, log2f(l)), kLn2f);
  }
}

template <int D>
__global__ void __launch_bounds__(kAtJoinThreads)
    paged_join_kernel(const __grid_constant__ AtParams a) {
  const int c = blockIdx.x / a.join_share, share = blockIdx.x % a.join_share;
  const float nan = __int_as_float(0x7fc00000);
  pdl_wait();
  pdl_launch_dependents();
  const PagedParams& p = a.p;
  const AtPart u = a.ctas[c].part[1];
  int met = 0;
  for (int i = threadIdx.x; i < a.main_ctas; i += kAtJoinThreads) met |= a.met[i];
  int late = met & kAtLate;
#ifdef SPEC_DEBUG
  late |= g_debug_inject == SPEC_ERR_TIMEOUT;
#endif
  late = __syncthreads_or(late);
  if (blockIdx.x == 0) {
    const int bad_page = __syncthreads_or(met & kAtBadPage);
    int bad = 0;
    for (int b = threadIdx.x; b < p.c.B; b += kAtJoinThreads)
      bad += !request_ok(p, p.c.new_start[b], p.c.new_start[b + 1], p.c.kv_len[b]);
    __shared__ int count;
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    if (bad) atomicAdd(&count, bad);
    __syncthreads();
    if (threadIdx.x == 0) {
      p.header->status = late               ? SPEC_ERR_TIMEOUT
                         : count || bad_page ? SPEC_ERR_BAD_INPUT
                                             : SPEC_OK;
      p.header->bad_requests = count;
      p.header->first_bad = INT32_MAX;
    }
  }
  if (!late && u.used) at_join<D>(a, u, c, share);
  // Rows that nobody computed.
  for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
    const int first = p.c.new_start[b], last = p.c.new_start[b + 1], len = p.c.kv_len[b];
    const bool good = request_ok(p, first, last, len);
    if (late || !good) {
      for (int r = max(first, 0); r < min(last, p.rows); ++r)
        at_fill<D>(a, r, nan, nan, threadIdx.x, kAtJoinThreads);
      continue;
    }
    const int n = last - first;
    for (int r0 = 0; r0 < n * a.group; r0 += kAtUnitRows) {
      const AtSpan s = at_unit_span(a, n, len, r0);
      if (s.tiles > 0) break;  // (and none behind it)
      for (int i = threadIdx.x; i < s.rows * p.c.kv_heads * (D / 8); i += kAtJoinThreads) {
        const int e = i % (D / 8), x = i / (D / 8), r = r0 + x % s.rows, h = x / s.rows;
        const long long head = at_head(a, first, h, r);
        reinterpret_cast<uint4*>(p.out + head * D)[e] = make_uint4(0, 0, 0, 0);
        if (e == 0 && p.lse != nullptr) p.lse[head] = -INFINITY;
      }
    }
  }
}

}  // namespace specv
