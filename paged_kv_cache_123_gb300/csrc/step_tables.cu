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
// Steps with more token rows than kFusedTokens run the fill on the whole GPU
// in a second launch that overlaps its start with programmatic dependent
// launch.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launchers.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanMaxCluster = 8;

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

// Token rows first, first + step, ...: position, slot, and the table entry
// of each block that a row opens. Rows behind the last token are padding
// (position 0, slot -1). `head` is the ring head before this step.
__device__ __forceinline__ void fill_tokens(const ExtendArgs& a, int64_t head, int64_t first,
                                            int64_t step) {
  const int64_t total = a.query_start_loc[a.num_seqs];
  const int64_t base = a.ring_size > 0 ? head % a.ring_size : 0;
  const uint32_t B = (uint32_t)a.block_size;
  for (int64_t t = first; t < a.num_tokens; t += step) {
    int64_t pos = 0, slot = -1;
    if (t < total) {
      int lo = 0, hi = a.num_seqs;          // last request that starts at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)a.query_start_loc[mid] <= t) lo = mid; else hi = mid;
      }
      const int64_t q0 = a.query_start_loc[lo];
      const int n = (int)(a.query_start_loc[lo + 1] - q0);
      const uint32_t ctx = (uint32_t)(a.seq_lens[lo] - n);
      const uint32_t p = ctx + (uint32_t)(t - q0);
      const uint32_t lb = p / B, row = p - lb * B;
      const uint32_t held = (ctx + (B - 1)) / B;
      int32_t* entry = a.block_tables + (int64_t)lo * a.table_stride + lb;
      int64_t blk;
      if (lb < held) {
        blk = *entry;
      } else {
        blk = a.free_ring[ring_at(base, a.block_start_loc[lo] + (int64_t)(lb - held),
                                  a.ring_size)];
        if (row == 0) *entry = (int32_t)blk;
      }
      pos = p;
      if (blk < 0 || blk >= a.num_blocks) latch(a.err, PA_ERR_OUT_OF_RANGE);
      else slot = blk * B + row;
    }
    a.positions[t] = pos;
    a.slot_mapping[t] = slot;
  }
}

template <bool FUSED>
__global__ void __launch_bounds__(kPlanThreads) extend_plan_kernel(const ExtendArgs a) {
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
  if (FUSED) __threadfence();
  cl.sync();            // shared memory of this CTA is no longer read; FUSED: sums visible
  if (FUSED)
    fill_tokens(a, head, (int64_t)rank * kPlanThreads + threadIdx.x,
                (int64_t)count * kPlanThreads);
}

__global__ void __launch_bounds__(256) extend_fill_kernel(const ExtendArgs a) {
  griddep_launch();
  griddep_wait();
  const int64_t head = a.ring_state_out[0] - a.block_start_loc[a.num_seqs];
  fill_tokens(a, head, (int64_t)blockIdx.x * blockDim.x + threadIdx.x,
              (int64_t)gridDim.x * blockDim.x);
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

// One warp per row: the row's valid entries, counted into
// release_start_loc[r + 1].
__device__ __forceinline__ void count_rows(const ReleaseArgs& a, int first, int step) {
  const int lane = threadIdx.x & 31;
  for (int r = first; r < a.num_seqs; r += step) {
    const int n = held_entries(a, r);
    const int32_t* row = a.block_tables + (int64_t)r * a.table_stride;
    int c = 0;
    for (int j = lane; j < n; j += 32) {
      const int32_t id = row[j];
      if (is_block(a, id)) ++c;
      else if (id >= 0) latch(a.err, PA_ERR_OUT_OF_RANGE);
    }
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) a.release_start_loc[r + 1] = c;
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
  block_exclusive(mine, warp_sums, &total);
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
    const Sum2 v{r < hi ? a.release_start_loc[r + 1] : 0, 0};
    __syncthreads();
    const Sum2 ex = block_exclusive(v, warp_sums, &total);
    if (r < hi) {
      a.release_start_loc[r + 1] = ok ? (int32_t)(carry + ex.a + v.a) : 0;
      const int32_t L = a.seq_lens[r];
      const bool gone = ok && a.finished[r] != 0 && L >= 0 && L <= a.table_stride * a.block_size;
      a.seq_lens_out[r] = gone ? 0 : L;
    }
    carry += total.a;
  }
}

// One warp per row: its valid entries, in table order, to the ring behind
// the rows before it. The row's count says how far to look, so the lengths
// may have been cleared in place.
__device__ __forceinline__ void return_rows(const ReleaseArgs& a, int first, int step) {
  const int lane = threadIdx.x & 31;
  const int64_t total = a.release_start_loc[a.num_seqs];
  const int64_t tail = a.ring_state_out[1] - total;
  const int64_t base = a.ring_size > 0 ? tail % a.ring_size : 0;
  for (int r = first; r < a.num_seqs; r += step) {
    const int64_t at = a.release_start_loc[r];
    const int n = (int)(a.release_start_loc[r + 1] - at);
    if (n > 0) {
      const int32_t* row = a.block_tables + (int64_t)r * a.table_stride;
      int done = 0;
      for (int j0 = 0; done < n; j0 += 32) {
        const int32_t id = j0 + lane < a.table_stride ? row[j0 + lane] : -1;
        const unsigned m = __ballot_sync(0xffffffffu, is_block(a, id));
        const int k = done + __popc(m & ((1u << lane) - 1u));
        if (((m >> lane) & 1u) && k < n)
          a.free_ring[ring_at(base, at + k, a.ring_size)] = id;
        done += __popc(m);
        if (j0 + 32 >= a.table_stride) break;
      }
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) release_one_kernel(const ReleaseArgs a) {
  __shared__ Sum2 warp_sums[kPlanWarps];
  __shared__ Sum2 slot;
  cg::cluster_group cl = cg::this_cluster();
  griddep_launch();
  griddep_wait();
  const int w = (int)cl.block_rank() * kPlanWarps + (int)(threadIdx.x >> 5);
  const int nw = (int)cl.num_blocks() * kPlanWarps;
  count_rows(a, w, nw);
  __threadfence();
  cl.sync();
  scan_rows(a, warp_sums, &slot);
  __threadfence();
  cl.sync();
  return_rows(a, w, nw);
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
cudaError_t launch_cluster(void (*kernel)(Args), int ctas, cudaStream_t st, const Args& a) {
  cudaLaunchConfig_t cfg = {};
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

// token rows that the cluster itself fills; table entries that it returns
constexpr int64_t kFusedTokens = 4 * kPlanMaxCluster * kPlanThreads;
constexpr int64_t kFusedEntries = 64 * 1024;

}  // namespace

cudaError_t launch_extend_tables(const ExtendArgs& a, int sm_count, cudaStream_t st) {
  if (a.num_tokens <= kFusedTokens)
    return launch_cluster(extend_plan_kernel<true>,
                          cluster_for(a.num_tokens > a.num_seqs ? a.num_tokens : a.num_seqs), st,
                          a);
  cudaError_t e =
      launch_cluster(extend_plan_kernel<false>, cluster_for(a.num_seqs), st, a);
  if (e != cudaSuccess) return e;
  const int threads = 256;
  int64_t blocks = (a.num_tokens + threads - 1) / threads;
  if (blocks > (int64_t)sm_count * 8) blocks = (int64_t)sm_count * 8;
  return launch_pdl(extend_fill_kernel, dim3((unsigned)blocks), dim3(threads), 0, st, a);
}

cudaError_t launch_release_tables(const ReleaseArgs& a, int sm_count, cudaStream_t st) {
  if ((int64_t)a.num_seqs * a.table_stride <= kFusedEntries)
    return launch_cluster(release_one_kernel, cluster_for((int64_t)a.num_seqs * 32), st, a);
  const int threads = 256, rows = threads / 32;
  int64_t blocks = ((int64_t)a.num_seqs + rows - 1) / rows;
  if (blocks > (int64_t)sm_count * 8) blocks = (int64_t)sm_count * 8;
  cudaError_t e =
      launch_pdl(release_count_kernel, dim3((unsigned)blocks), dim3(threads), 0, st, a);
  if (e != cudaSuccess) return e;
  e = launch_cluster(release_scan_kernel, cluster_for(a.num_seqs), st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(release_return_kernel, dim3((unsigned)blocks), dim3(threads), 0, st, a);
}

}  // namespace pa
