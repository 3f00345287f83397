// Block tables, positions and slot maps of a step built on the GPU from
// request lengths, and the blocks of finished requests returned.
//
// The bookkeeping is that of "PagedAttention 核心创新深度分析" §3.2 (BlockPool:
// a request takes blocks from the head of the free list only when its last
// block is full; freed blocks go to the tail) and §2.3 (slot mapping), for
// blocks that one request owns. The free list is a ring of block ids with
// two running counters, head and tail: entry i sits at ring[i mod size], so
// head .. tail - 1 are the free blocks in the order they will be handed out.
//
// extend: request r holds c_r tokens and gets n_r more. With
//     qsl_r = sum_{x<r} n_x,   b_r = ceil((c_r + n_r) / B) - ceil(c_r / B),
//     bsl_r = sum_{x<r} b_x,
// new token t of request r is at p = c_r + t - qsl_r in logical block p / B;
// blocks below ceil(c_r / B) are in the table already, block
// ceil(c_r / B) + k is ring entry head + bsl_r + k. Two exclusive sums and a
// search per token, all integers, so results do not depend on the schedule.
//
// Both calls are bound by latency: a decode step of 128 requests moves 5 KB.
// Small steps are therefore ONE launch of one thread-block cluster (up to 8
// CTAs): each CTA sums its share of the requests, the totals meet through
// distributed shared memory, and the same threads then fill the token rows.
// Steps with more token rows run the fill on the whole GPU in a second launch
// that overlaps its start with programmatic dependent launch; a release of
// more requests than the cluster has warps is a count, a scan and a return.
//
// Replayed from a graph: extend of 128 single tokens 6.3 us; of 8,192
// requests with 1.05 million rows 18.3 us (17.5 MB, 2.6 us at the copy rate:
// the plan takes 7, then loads that depend on one another: start rows,
// request, block, slot); release of 32 of 128 requests 5.3 us, of 4,096 of
// 8,192 (33.7 MB of entries read and written, 5 us) 25 us: its three launches
// cost 7 us with nothing to move, the entries are read twice, and a row's
// 2,048 entries are four dependent rounds of its warp.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launchers.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanMaxCluster = 8;
constexpr int kFillThreads = 512;
constexpr int kFillGroups = 4;    // 64-row groups a warp takes at a time
// Table entries a lane has in flight: with 8, 16 and 32 the small release
// takes 5.6, 5.3 and 8.3 us, the large one 25.1, 25.3 and 27.7.
constexpr int kAtOnce = 16;
// Requests whose query_start_loc is staged in shared memory for the searches:
// the 48 KB that a launch has without asking for more, less 1 KB for the
// kernels' own.
constexpr int kStagedSeqs = 12 * 1024 - 256 - 1;

struct Sum2 {
  int64_t a, b;
};

// Exclusive sum over the CTA of one pair per thread; *total gets the CTA's
// sum. `warp_sums` is shared, one pair per warp; the caller syncs between
// two calls.
__device__ __forceinline__ Sum2 block_exclusive(Sum2 v, Sum2* warp_sums, Sum2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sum2 inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, inc.a, o);
    const int64_t b = __shfl_up_sync(0xffffffffu, inc.b, o);
    if (lane >= o) { inc.a += a; inc.b += b; }
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    Sum2 w = lane < kPlanWarps ? warp_sums[lane] : Sum2{0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, w.a, o);
      const int64_t b = __shfl_up_sync(0xffffffffu, w.b, o);
      if (lane >= o) { w.a += a; w.b += b; }
    }
    if (lane < kPlanWarps) warp_sums[lane] = w;
  }
  __syncthreads();
  const Sum2 before = warp > 0 ? warp_sums[warp - 1] : Sum2{0, 0};
  *total = warp_sums[kPlanWarps - 1];
  return Sum2{before.a + inc.a - v.a, before.b + inc.b - v.b};
}

// Sums of the CTAs before this one in the cluster and of all of them; every
// thread of every CTA calls it. The cluster has synchronised once in here.
struct ClusterSums {
  Sum2 before, all;
};
__device__ __forceinline__ ClusterSums cluster_sums(Sum2 mine, Sum2* slot) {
  cg::cluster_group cl = cg::this_cluster();
  if (threadIdx.x == 0) *slot = mine;
  cl.sync();
  ClusterSums r{{0, 0}, {0, 0}};
  const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
  for (int i = 0; i < n; ++i) {
    const Sum2 s = *cl.map_shared_rank(slot, i);
    if (i < rank) { r.before.a += s.a; r.before.b += s.b; }
    r.all.a += s.a;
    r.all.b += s.b;
  }
  return r;
}

// The share [lo, hi) of n items that CTA `rank` of `count` takes: whole
// tiles of kPlanThreads.
__device__ __forceinline__ void cta_share(int n, int rank, int count, int* lo, int* hi) {
  const int tiles = (n + kPlanThreads - 1) / kPlanThreads;
  const int per = (tiles + count - 1) / count;
  *lo = (int)min((int64_t)n, (int64_t)rank * per * kPlanThreads);
  *hi = (int)min((int64_t)n, (int64_t)(rank + 1) * per * kPlanThreads);
}

// index base + i into a ring of `size` entries; base < size, 0 <= i <= size
__device__ __forceinline__ int64_t ring_at(int64_t base, int64_t i, int64_t size) {
  const int64_t x = base + i;
  return x >= size ? x - size : x;
}

__device__ __forceinline__ bool ring_ok(int64_t head, int64_t tail, int64_t size) {
  return head >= 0 && tail >= head && tail - head <= size;
}

// New tokens and new blocks of request r; a request with a length that is
// negative or past its table row gets neither.
__device__ __forceinline__ Sum2 request_need(const ExtendArgs& a, int r) {
  const int64_t c = a.context_lens[r], n = a.new_tokens[r];
  if (c < 0 || n < 0 || c + n > 0x7fffffffll || c + n > a.table_stride * a.block_size) {
    latch(a.err, PA_ERR_OUT_OF_RANGE);
    return Sum2{0, 0};
  }
  if (n == 0) return Sum2{0, 0};
  const uint32_t B = (uint32_t)a.block_size;
  const uint32_t held = ((uint32_t)c + (B - 1)) / B;
  const uint32_t need = ((uint32_t)(c + n) + (B - 1)) / B;
  return Sum2{n, (int64_t)need - held};
}

// Last request in [lo, hi) that starts at or before row t (query_start_loc[lo]
// <= t).
__device__ __forceinline__ int request_of(const int32_t* qsl, int64_t t, int lo, int hi) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)qsl[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// p / B, by a shift where B is a power of two (shift >= 0)
__device__ __forceinline__ uint32_t block_of(uint32_t p, uint32_t B, int shift) {
  return shift >= 0 ? p >> shift : p / B;
}

// Where token row t of request r goes: its position, and the entry (of the
// table, or of the ring when it opens or continues a new block) that names
// its block.
struct RowPlace {
  int64_t pos;
  uint32_t row;
  const int32_t* src;
  int32_t* opens;            // table entry to write, or nullptr
};
__device__ __forceinline__ RowPlace place_row(const ExtendArgs& a, const int32_t* qsl, int r,
                                              int64_t t, int64_t base, int shift) {
  const uint32_t B = (uint32_t)a.block_size;
  const int64_t q0 = qsl[r];
  const int n = (int)(qsl[r + 1] - q0);
  const uint32_t ctx = (uint32_t)(a.seq_lens[r] - n);
  const uint32_t p = ctx + (uint32_t)(t - q0);
  const uint32_t lb = block_of(p, B, shift);
  const uint32_t held = block_of(ctx + (B - 1), B, shift);
  int32_t* entry = a.block_tables + (int64_t)r * a.table_stride + lb;
  RowPlace w;
  w.pos = p;
  w.row = p - lb * B;
  w.src = lb < held ? entry
                    : a.free_ring + ring_at(base, a.block_start_loc[r] + (int64_t)(lb - held),
                                            a.ring_size);
  w.opens = lb >= held && w.row == 0 ? entry : nullptr;
  return w;
}
__device__ __forceinline__ int64_t slot_of(const ExtendArgs& a, const RowPlace& w, int32_t blk) {
  if (w.opens != nullptr) *w.opens = blk;
  if (blk < 0 || blk >= a.num_blocks) {
    latch(a.err, PA_ERR_OUT_OF_RANGE);
    return -1;
  }
  return (int64_t)blk * a.block_size + w.row;
}

// Token rows: warp `first` of `step` takes `groups` x 32 ROWS consecutive rows
// at a time, a lane ROWS (1 or 2) of each group. The requests of the warp's first and last row
// are searched once (every lane the same loads); a lane then searches between
// them, which for prompts is next to no search. Rows behind the last token are
// padding (position 0, slot -1). `qsl` is query_start_loc or a copy in shared
// memory, `head` the ring head before this step.
template <int ROWS>
__device__ __forceinline__ void fill_tokens(const ExtendArgs& a, const int32_t* qsl, int64_t head,
                                            int64_t first, int64_t step, int groups) {
  const int lane = threadIdx.x & 31;
  const int64_t total = qsl[a.num_seqs];
  const int64_t base = a.ring_size > 0 ? head % a.ring_size : 0;
  const int shift = (a.block_size & (a.block_size - 1)) == 0 ? __ffs(a.block_size) - 1 : -1;
  const bool pairs = (reinterpret_cast<uintptr_t>(a.positions) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.slot_mapping) & 15) == 0;
  const int64_t span = 32 * ROWS * (int64_t)groups;
  for (int64_t t0 = first * span; t0 < a.num_tokens; t0 += step * span) {
    int lo = 0, hi = a.num_seqs;
    if (t0 < total) {
      lo = request_of(qsl, t0, 0, a.num_seqs);
      hi = request_of(qsl, min(t0 + span, total) - 1, lo, a.num_seqs) + 1;
    }
#pragma unroll 2
    for (int g = 0; g < groups; ++g) {
      const int64_t t = t0 + 32 * ROWS * g + ROWS * lane;
      longlong2 pos = make_longlong2(0, 0), slot = make_longlong2(-1, -1);
      if (t < total) {
        // both rows' loads before either's stores
        const int r = request_of(qsl, t, lo, hi);
        const RowPlace w0 = place_row(a, qsl, r, t, base, shift);
        const bool two = ROWS == 2 && t + 1 < total;
        RowPlace w1 = w0;
        if (two)
          w1 = place_row(a, qsl, (int64_t)qsl[r + 1] <= t + 1 ? request_of(qsl, t + 1, r, hi) : r,
                         t + 1, base, shift);
        const int32_t b0 = *w0.src, b1 = *w1.src;
        pos.x = w0.pos;
        slot.x = slot_of(a, w0, b0);
        if (two) {
          pos.y = w1.pos;
          slot.y = slot_of(a, w1, b1);
        }
      }
      if (ROWS == 2 && pairs && t + 1 < a.num_tokens) {
        *reinterpret_cast<longlong2*>(a.positions + t) = pos;
        *reinterpret_cast<longlong2*>(a.slot_mapping + t) = slot;
      } else {
        if (t < a.num_tokens) { a.positions[t] = pos.x; a.slot_mapping[t] = slot.x; }
        if (ROWS == 2 && t + 1 < a.num_tokens) {
          a.positions[t + 1] = pos.y;
          a.slot_mapping[t + 1] = slot.y;
        }
      }
    }
  }
}

// query_start_loc in shared memory, if it fits: the searches are chains of
// dependent loads.
__device__ __forceinline__ const int32_t* stage_starts(const ExtendArgs& a, int32_t* staged) {
  if (a.num_seqs > kStagedSeqs) return a.query_start_loc;
  for (int i = threadIdx.x; i <= a.num_seqs; i += blockDim.x) staged[i] = a.query_start_loc[i];
  __syncthreads();
  return staged;
}
static_assert((kStagedSeqs + 1) * 4 + 1024 <= 48 * 1024, "staged rows and the kernels' own");
int staged_bytes(int num_seqs) { return num_seqs > kStagedSeqs ? 0 : (num_seqs + 1) * 4; }

// ROWS: token rows of a lane at a time in the same launch, 0: in the next one.
template <int ROWS>
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const ExtendArgs a) {
  extern __shared__ int32_t staged[];
  __shared__ Sum2 warp_sums[kPlanWarps];
  __shared__ Sum2 slot;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), count = (int)cl.num_blocks();
  griddep_launch();
  griddep_wait();
  const int64_t head = a.ring_state[0], tail = a.ring_state[1];
  int lo, hi;
  cta_share(a.num_seqs, rank, count, &lo, &hi);

  // this CTA's sums; the first tile's values stay in registers
  Sum2 mine{0, 0}, first{0, 0};
  for (int r = lo + (int)threadIdx.x; r < hi; r += kPlanThreads) {
    const Sum2 v = request_need(a, r);
    if (r < lo + kPlanThreads) first = v;
    mine.a += v.a;
    mine.b += v.b;
  }
  Sum2 total;
  Sum2 ex = block_exclusive(mine, warp_sums, &total);
  const ClusterSums cs = cluster_sums(total, &slot);

  // the whole step fits, or nothing changes
  const bool sane = ring_ok(head, tail, a.ring_size) && cs.all.a <= a.num_tokens;
  const bool ok = sane && cs.all.b <= tail - head;
  if (rank == 0 && threadIdx.x == 0) {
    if (!ok) latch(a.err, sane ? PA_ERR_NO_BLOCKS : PA_ERR_OUT_OF_RANGE);
    a.query_start_loc[a.num_seqs] = ok ? (int32_t)cs.all.a : 0;
    a.block_start_loc[a.num_seqs] = ok ? (int32_t)cs.all.b : 0;
    // every CTA has read the state (cluster barrier above), so the output
    // may be the same array
    a.ring_state_out[0] = ok ? head + cs.all.b : head;
    a.ring_state_out[1] = tail;
  }
  Sum2 carry = cs.before;
  const bool one_tile = hi - lo <= kPlanThreads;
  for (int r0 = lo; r0 < hi; r0 += kPlanThreads) {
    const int r = r0 + (int)threadIdx.x;
    Sum2 v = first;
    if (!one_tile) {
      // one pair per thread again: the sums above were over whole columns
      if (r0 > lo) v = r < hi ? request_need(a, r) : Sum2{0, 0};
      __syncthreads();
      ex = block_exclusive(v, warp_sums, &total);
    }
    if (r < hi) {
      const int32_t c = a.context_lens[r];
      a.query_start_loc[r] = ok ? (int32_t)(carry.a + ex.a) : 0;
      a.block_start_loc[r] = ok ? (int32_t)(carry.b + ex.b) : 0;
      a.seq_lens[r] = ok ? c + (int32_t)v.a : c;
    }
    carry.a += total.a;
    carry.b += total.b;
  }
  if (ROWS > 0) __threadfence();
  cl.sync();            // shared memory of this CTA is no longer read; ROWS: sums visible
  if (ROWS > 0)
    fill_tokens<ROWS>(a, stage_starts(a, staged), head,
                (int64_t)rank * kPlanWarps + (threadIdx.x >> 5), (int64_t)count * kPlanWarps, 1);
}

__global__ void __launch_bounds__(kFillThreads) extend_fill_kernel(const ExtendArgs a) {
  extern __shared__ int32_t staged[];
  griddep_launch();
  griddep_wait();
  const int64_t head = a.ring_state_out[0] - a.block_start_loc[a.num_seqs];
  fill_tokens<2>(a, stage_starts(a, staged), head,
                 (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5),
                 (int64_t)gridDim.x * (blockDim.x >> 5), kFillGroups);
}

// Table entries that request r holds, 0 if it is not finished; a length
// that is negative or past the table row is reported and holds none.
__device__ __forceinline__ int held_entries(const ReleaseArgs& a, int r) {
  if (a.finished[r] == 0) return 0;
  const int64_t L = a.seq_lens[r];
  if (L < 0 || L > a.table_stride * a.block_size) {
    latch(a.err, PA_ERR_OUT_OF_RANGE);
    return 0;
  }
  return (int)((L + a.block_size - 1) / a.block_size);
}

__device__ __forceinline__ bool is_block(const ReleaseArgs& a, int32_t id) {
  return id >= 0 && id < a.num_blocks;
}

// ---- rows of table entries, a warp each
__device__ __forceinline__ int count_ids(const ReleaseArgs& a, const int32_t (&id)[kAtOnce]) {
  int c = 0;
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    if (is_block(a, id[k])) ++c;
    else if (id[k] >= 0) latch(a.err, PA_ERR_OUT_OF_RANGE);
  }
  return c;
}
__device__ __forceinline__ void load_ids(const int32_t* row, int64_t j0, int64_t end,
                                         int32_t (&id)[kAtOnce]) {
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const int64_t j = j0 + 32 * k + (threadIdx.x & 31);
    id[k] = j < end ? row[j] : -1;
  }
}

// Valid entries among the first `held` of a row, the first of which are in
// id.
__device__ __forceinline__ int count_row(const ReleaseArgs& a, const int32_t* row, int held,
                                         const int32_t (&id)[kAtOnce]) {
  int c = count_ids(a, id);
  for (int j0 = 32 * kAtOnce; j0 < held; j0 += 32 * kAtOnce) {
    int32_t more[kAtOnce];
    load_ids(row, j0, held, more);
    c += count_ids(a, more);
  }
  return __reduce_add_sync(0xffffffffu, c);
}

// Counts of the rows into release_start_loc[r + 1].
__device__ __forceinline__ void count_rows(const ReleaseArgs& a, int first, int step) {
  for (int r = first; r < a.num_seqs; r += step) {
    const int held = held_entries(a, r);
    const int32_t* row = a.block_tables + (int64_t)r * a.table_stride;
    int32_t id[kAtOnce];
    load_ids(row, 0, held, id);
    const int c = count_row(a, row, held, id);
    if ((threadIdx.x & 31) == 0) a.release_start_loc[r + 1] = c;
  }
}

// Counts to inclusive sums, in place, the ring's new tail and the rows' new
// lengths. The whole release fits the ring, or nothing changes.
__device__ __forceinline__ void scan_rows(const ReleaseArgs& a, Sum2* warp_sums, Sum2* slot) {
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), count = (int)cl.num_blocks();
  const int64_t head = a.ring_state[0], tail = a.ring_state[1];
  int lo, hi;
  cta_share(a.num_seqs, rank, count, &lo, &hi);
  Sum2 mine{0, 0}, total;
  for (int r = lo + (int)threadIdx.x; r < hi; r += kPlanThreads)
    mine.a += a.release_start_loc[r + 1];
  Sum2 ex = block_exclusive(mine, warp_sums, &total);
  const ClusterSums cs = cluster_sums(total, slot);
  const bool ok =
      ring_ok(head, tail, a.ring_size) && cs.all.a <= a.ring_size - (tail - head);
  if (rank == 0 && threadIdx.x == 0) {
    if (!ok) latch(a.err, PA_ERR_OUT_OF_RANGE);
    a.release_start_loc[0] = 0;
    a.ring_state_out[0] = head;
    a.ring_state_out[1] = ok ? tail + cs.all.a : tail;
  }
  int64_t carry = cs.before.a;
  for (int r0 = lo; r0 < hi; r0 += kPlanThreads) {
    const int r = r0 + (int)threadIdx.x;
    Sum2 v = mine;
    if (hi - lo > kPlanThreads) {
      v = Sum2{r < hi ? a.release_start_loc[r + 1] : 0, 0};
      __syncthreads();
      ex = block_exclusive(v, warp_sums, &total);
    }
    if (r < hi) {
      a.release_start_loc[r + 1] = ok ? (int32_t)(carry + ex.a + v.a) : 0;
      const int32_t L = a.seq_lens[r];
      const bool gone = ok && a.finished[r] != 0 && L >= 0 && L <= a.table_stride * a.block_size;
      a.seq_lens_out[r] = gone ? 0 : L;
    }
    carry += total.a;
  }
}

// Ring entries of a warp's 32 x kAtOnce table entries, of which `done` valid
// ones came before in the row; the row returns n, the first to ring entry
// base + at.
__device__ __forceinline__ void put_ids(const ReleaseArgs& a, const int32_t (&id)[kAtOnce],
                                        int64_t base, int64_t at, int n, int& done) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const bool mine = is_block(a, id[k]);
    const unsigned m = __ballot_sync(0xffffffffu, mine);
    const int x = done + __popc(m & ((1u << lane) - 1u));
    if (mine && x < n) a.free_ring[ring_at(base, at + x, a.ring_size)] = id[k];
    done += __popc(m);
  }
}
// One warp per row: its valid entries, in table order, to the ring behind
// the rows before it. The row's count says how far to look, so the lengths
// may have been cleared in place.
__device__ __forceinline__ void return_rows(const ReleaseArgs& a, int first, int step) {
  const int64_t total = a.release_start_loc[a.num_seqs];
  const int64_t tail = a.ring_state_out[1] - total;
  const int64_t base = a.ring_size > 0 ? tail % a.ring_size : 0;
  for (int r = first; r < a.num_seqs; r += step) {
    const int64_t at = a.release_start_loc[r];
    const int n = (int)(a.release_start_loc[r + 1] - at);
    const int32_t* row = a.block_tables + (int64_t)r * a.table_stride;
    int done = 0;
    for (int64_t j0 = 0; done < n && j0 < a.table_stride; j0 += 32 * kAtOnce) {
      int32_t id[kAtOnce];
      load_ids(row, j0, a.table_stride, id);
      put_ids(a, id, base, at, n, done);
    }
  }
}

// The whole release in one cluster, a warp per row: the rows' counts meet
// through distributed shared memory, every CTA sums all of them, and the
// entries that were counted (the first 512 of a row, from registers) go to
// the ring.
__global__ void __launch_bounds__(kPlanThreads) release_one_kernel(const ReleaseArgs a) {
  __shared__ Sum2 warp_sums[kPlanWarps];
  __shared__ int counts[kPlanWarps];
  __shared__ int starts[kPlanMaxCluster * kPlanWarps];
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = (int)cl.block_rank() * kPlanWarps + warp;
  griddep_launch();
  griddep_wait();
  const int64_t head = a.ring_state[0], tail = a.ring_state[1];
  const bool row_is = r < a.num_seqs;
  const int L = row_is ? a.seq_lens[r] : 0;
  const int held = row_is ? held_entries(a, r) : 0;
  const int32_t* row = a.block_tables + (int64_t)r * a.table_stride;
  int32_t id[kAtOnce];
  load_ids(row, 0, held, id);
  const int n = count_row(a, row, held, id);
  if (lane == 0) counts[warp] = n;
  cl.sync();
  const int other = (int)threadIdx.x / kPlanWarps;
  const Sum2 v{other < (int)cl.num_blocks() ? cl.map_shared_rank(counts, other)[lane] : 0, 0};
  Sum2 total;
  const Sum2 ex = block_exclusive(v, warp_sums, &total);
  if (threadIdx.x < kPlanMaxCluster * kPlanWarps)
    starts[threadIdx.x] = (int)min(ex.a, (int64_t)0x7fffffff);
  __syncthreads();
  const bool ok =
      ring_ok(head, tail, a.ring_size) && total.a <= a.ring_size - (tail - head);
  if (r == 0 && lane == 0) {
    if (!ok) latch(a.err, PA_ERR_OUT_OF_RANGE);
    a.release_start_loc[0] = 0;
    // every CTA has read the state (cluster barrier above)
    a.ring_state_out[0] = head;
    a.ring_state_out[1] = ok ? tail + total.a : tail;
  }
  if (row_is) {
    const int at = starts[r];
    if (lane == 0) {
      a.release_start_loc[r + 1] = ok ? at + n : 0;
      const bool gone = ok && a.finished[r] != 0 && L >= 0 && L <= a.table_stride * a.block_size;
      a.seq_lens_out[r] = gone ? 0 : L;
    }
    if (ok && n > 0) {
      const int64_t base = tail % a.ring_size;
      int done = 0;
      put_ids(a, id, base, at, n, done);
      for (int64_t j0 = 32 * kAtOnce; done < n && j0 < held; j0 += 32 * kAtOnce) {
        load_ids(row, j0, held, id);
        put_ids(a, id, base, at, n, done);
      }
    }
  }
  cl.sync();            // no CTA leaves while another reads its counts
}

__global__ void __launch_bounds__(256) release_count_kernel(const ReleaseArgs a) {
  griddep_launch();
  griddep_wait();
  count_rows(a, (int)(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)),
             (int)(gridDim.x * (blockDim.x >> 5)));
}

__global__ void __launch_bounds__(kPlanThreads) release_scan_kernel(const ReleaseArgs a) {
  __shared__ Sum2 warp_sums[kPlanWarps];
  __shared__ Sum2 slot;
  griddep_launch();
  griddep_wait();
  scan_rows(a, warp_sums, &slot);
  cg::this_cluster().sync();     // no CTA leaves while another reads its shared memory
}

__global__ void __launch_bounds__(256) release_return_kernel(const ReleaseArgs a) {
  griddep_launch();
  griddep_wait();
  return_rows(a, (int)(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)),
              (int)(gridDim.x * (blockDim.x >> 5)));
}

template <typename Args>
cudaError_t launch_cluster(void (*kernel)(Args), int ctas, size_t smem, cudaStream_t st,
                           const Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

int cluster_for(int64_t threads) {
  const int64_t ctas = (threads + kPlanThreads - 1) / kPlanThreads;
  return ctas <= 1 ? 1 : ctas <= 2 ? 2 : ctas <= 4 ? 4 : kPlanMaxCluster;
}

// Token rows that the cluster itself fills: the second launch costs some 2
// us (5 to 7 with many requests, whose sums and table writes it repeats), the
// fill on eight SMs 0.2 us per 1,024 rows. One launch against two: 64
// requests, 16,384 rows 7.9 and 8.9 us, 32,768 rows 10.2 and 9.0; 8,192
// requests, 32,768 rows 15.3 and 18.4, 65,536 rows 21.8 and 18.1.
int64_t fused_tokens(int num_seqs) { return 24 * 1024 + 2 * (int64_t)num_seqs; }
// Requests that one cluster releases, a warp each; three launches take, in
// one launch's place, 7.6 us instead of 5.4 (128 requests of up to 4k tokens
// in blocks of 16), 13.8 instead of 11.8 (256 of up to 32k).
constexpr int kFusedRows = kPlanMaxCluster * kPlanWarps;

}  // namespace

cudaError_t launch_extend_tables(const ExtendArgs& a, int sm_count, cudaStream_t st) {
  // a row per thread while the cluster has one for each: the chain is shorter
  // than with two (128 requests, 128 rows 6.2 and 6.8 us; 64 requests, 4,096
  // rows 6.6 and 7.0, 16,384 rows 8.8 and 7.6)
  if (a.num_tokens <= fused_tokens(a.num_seqs))
    return launch_cluster(a.num_tokens <= kPlanMaxCluster * kPlanThreads ? extend_plan_kernel<1>
                                                                         : extend_plan_kernel<2>,
                          cluster_for(a.num_tokens > a.num_seqs ? a.num_tokens : a.num_seqs),
                          staged_bytes(a.num_seqs), st, a);
  cudaError_t e =
      launch_cluster(extend_plan_kernel<0>, cluster_for(a.num_seqs), 0, st, a);
  if (e != cudaSuccess) return e;
  // two CTAs per SM at most: each stages the start rows once
  const int rows = kFillThreads / 32 * 64 * kFillGroups;
  int64_t blocks = (a.num_tokens + rows - 1) / rows;
  if (blocks > (int64_t)sm_count * 2) blocks = (int64_t)sm_count * 2;
  return launch_pdl(extend_fill_kernel, dim3((unsigned)blocks), dim3(kFillThreads),
                    (size_t)staged_bytes(a.num_seqs), st, a);
}

cudaError_t launch_release_tables(const ReleaseArgs& a, int sm_count, cudaStream_t st) {
  if (a.num_seqs <= kFusedRows)
    return launch_cluster(release_one_kernel, cluster_for((int64_t)a.num_seqs * 32), 0, st, a);
  const int threads = 256, rows = threads / 32;
  int64_t blocks = ((int64_t)a.num_seqs + rows - 1) / rows;
  if (blocks > (int64_t)sm_count * 8) blocks = (int64_t)sm_count * 8;
  cudaError_t e =
      launch_pdl(release_count_kernel, dim3((unsigned)blocks), dim3(threads), 0, st, a);
  if (e != cudaSuccess) return e;
  e = launch_cluster(release_scan_kernel, cluster_for(a.num_seqs), 0, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(release_return_kernel, dim3((unsigned)blocks), dim3(threads), 0, st, a);
}

}  // namespace pa
