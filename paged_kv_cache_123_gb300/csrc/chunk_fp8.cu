// Causal attention of chunks of new tokens over fp8 (E4M3) KV pools, with an
// optional sliding window, on the fifth-generation tensor cores.
//
// New token i of sequence s (n_s new tokens, L_s tokens in the pool with
// them) sits at p = L_s - n_s + i and attends to max(0, p - W + 1) .. p (W =
// 0: from 0), through the block table:
//     x_j = scale <q, K_j>,  out = sum_j softmax(x)_j V_j,
// K = code * k_scale, V = code * v_scale with one scale per pool or one
// power-of-two scale per (block, KV head). ("vLLM 的 PagedAttention：显存管理如何
// 撑起大模型推理" §2.5: one token budget covers prefill chunks and single
// tokens; "PagedAttention 核心创新深度分析" §3.5: the KV spec carries a
// quantisation mode.)
//
// One CTA owns up to 256 rows, (new token, query head) pairs of one KV head,
// as two tiles of 128 (the MMA's M), and walks their keys in tiles of 128
// tokens. Two chains, each with its scores, its output in tensor memory and
// four softmax warps, keep the tensor core busy: while one chain's softmax
// runs, the core works for the other. With more than 128 rows each chain has
// its row tile and takes every key tile (a key tile is loaded and widened
// once for 256 rows); with fewer, both have the same rows and take the key
// tiles in turn, and their results meet at the end.
//   * two producer warps bring the tiles' codes (K and V) by 3-D TMA boxes,
//     one per block piece, into a ring of raw stages;
//   * four converter warps widen each raw tile to fp16 (E4M3 is exact in
//     fp16) into the 128-byte-swizzled operand layout of the MMA, two stages
//     each of K and V, and clear rows without a token on the way;
//   * the Q tiles are fp16 with each row divided by a power of two, so that a
//     bf16 query keeps its 8 significant bits down to 2^-24 of the row's
//     largest value;
//   * one thread issues S = Q K^T into the chain's TMEM scores and O += P V
//     with P (fp16, over the scores) read from TMEM;
//   * a softmax thread owns one row: scores in registers, running maximum
//     and sum in fp32; the output in TMEM is rescaled only when the maximum
//     grew by more than 2^8.
// The steps are halves of a key tile, which makes four streams of scores
// (all in flight: a stream's next scores are issued one step late, behind the
// next stream's P V). A key tile takes 256 rows some 3,700 clocks, of which
// the MMAs need 2,590 by their measured rates (64 clocks for 128 x 128 x 16,
// 49 for the scores' 128 x 64 x 16); what is left is each stream's chain of
// scores, maximum, exponentials, P, P V and next scores, which four streams
// do not quite cover.
//
// Replayed from a graph (64 query and 8 KV heads of 128, bf16, blocks of 16,
// one scale): 8 x 512 tokens after 4k 523 us, 1,116 TFLOP/s, 0.58 of the
// measured bf16 rate; 4 tokens x 128 sequences of 1k
// to 8k 357 us, 3.5 TB/s of codes, 0.52 of the copy rate: a 32-row tile costs
// the softmax and the MMAs as much as a full one. 4 x 256 tokens (32 heads,
// fp16) over 32k with scales per block 598 us, 924 TFLOP/s; 16 ragged chunks
// of up to 511 with a window of 1,000 208 us: with ten key tiles per CTA its
// start (some 10,000 clocks: Q) and end (4,000) are a quarter.
// Measured and dropped: whole-row softmax steps of 128 keys with larger
// register shares (669 us for the 8 x 512 case, then at 609), one step that
// finds the maximum and redoes the exponentials where it grew (540 against
// 533), eight converter warps (536 against 526), an MMA warp that takes
// whichever stream is ready (636 against 531), waits by one lane (749 against
// 609).
//
// fp16 products for both query types: weights are rounded to 11 bits, one
// rounding, in [0, 2^8].
//
// Per-block scales: the converters multiply a block's codes by its scale over
// a reference, at most 1: for K the tile's largest scale, which then joins
// the logit factor, for V the largest so far, which the output is in units of
// (it is rescaled when that reference grows). Powers of two keep this exact
// down to 2^-15 of the reference; below, low bits go as they would with one
// scale equal to the reference. (With the factors on the scores and
// weights in the softmax warps 4 x 256 tokens over 32k took 660 us instead of
// 611.)
//
// NaN codes: a masked weight is 0, but 0 x NaN is NaN inside the MMA, so a
// NaN in V could reach rows that do not see its token. Tiles that some row
// sees only in part are cleared of NaN codes while being widened; if there
// were any, the rows that do see them get their NaNs at the end by a look at
// the codes themselves.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "launchers.h"
#include "mma_util.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;                // rows of a chain (MMA M)
// Rows of a CTA. Two row tiles share each key tile's widening; with CTAs of
// one tile 8 x 512 tokens after 4k take 1,036 us instead of 529, and one
// chunk of 32 tokens x 8 heads after 2k, with twice the CTAs for its two
// tiles, 27.7 instead of 26.6.
constexpr int kCtaRows = 2 * kRows;
constexpr int kKv = 128;                  // KV tokens per tile
constexpr int kMmaWarp = 0;
constexpr int kProducerWarp = 1;          // K, and 2: V
constexpr int kConvWarp = 4;              // 4-7: converters
constexpr int kConvWarps = 4;
constexpr int kSoftmaxWarp = 8;           // 8-11, 12-15: the chains' softmax
constexpr int kThreads = 512;
constexpr int kHalf = kKv / 2;            // tokens of a softmax step
constexpr int kMaxRaw = 4;                // raw stages with one row tile; 2 with two
constexpr uint32_t kTmemCols = 512;       // scores: chain c at 128 c; outputs: 256 + 128 c
constexpr uint32_t kOCol = 256;
constexpr long long kWaitCycles = 4000000000LL;
constexpr float kLazyLog2 = 8.f;
#define kNegInfC (-__int_as_float(0x7f800000))

// barriers; kSFull, kPFull and kODone have one per chain and half (2 c + h),
// each with one phase per tile of the chain
enum : int {
  kRawFull = 0, kRawEmpty = kMaxRaw, kKFull = 2 * kMaxRaw, kKEmpty = kKFull + 2,
  kVFull = kKEmpty + 2, kVEmpty = kVFull + 2, kSFull = kVEmpty + 2, kPFull = kSFull + 4,
  kODone = kPFull + 4, kDone = kODone + 4, kQFull, kConvDone, kBars
};

// Per-block scales of a tile: pieces over the references, and the references.
// A slot is written with the K tile's copies; the writer is at most five
// tiles ahead of the softmax warps (two raw tiles, one in the converters'
// registers, two operand stages).
struct TileScales {
  float k[16], v[16];
  float k_ref, v_ref, unused[2];
};
constexpr int kScaleSlots = 8;
constexpr int kMaxOrdered = kThreads / 4;  // sequences taken by length at most

template <int D>
struct ChunkLayout {
  // small things first, so that the 1024-byte aligned tiles end exactly at
  // the limit of 227 KB for head size 128
  static constexpr int BAR_OFF = 0;
  // words: 0 tmem base, 1 abort flag, 2-5 piece masks of the raw stages, 6
  // NaN codes met, 7 the sequence, 8-11 piece masks of the last four K tiles
  static constexpr int MISC_OFF = (kBars * 8 + 15) / 16 * 16;
  static constexpr int ROW_OFF = MISC_OFF + 64;                 // float [2][128] Q row factors
  static constexpr int SCALE_OFF = ROW_OFF + 2 * kRows * 4;     // TileScales of the last tiles
  static constexpr int SMALL = SCALE_OFF + kScaleSlots * (int)sizeof(TileScales);
  static constexpr int HALVES = D / 64;
  static constexpr int HALF = kKv * 128;                        // 128 rows x 64 fp16
  static constexpr int TILE = HALVES * HALF;
  static constexpr int RAW = kKv * D;
  static constexpr int Q_OFF = 0;                               // from the aligned base
  static constexpr int K_OFF = TILE;
  static constexpr int V_OFF = K_OFF + 2 * TILE;
  static constexpr int RAW_OFF = V_OFF + 2 * TILE;              // two raw stages, then
  static constexpr int Q2_OFF = RAW_OFF + 2 * RAW;              // Q tile 2 or two more
  static constexpr int TILES = Q2_OFF + TILE;
  static constexpr int SMEM = 3 * 1024 + TILES;
  static_assert(2 * RAW <= TILE, "two raw stages where Q tile 2 is");
  static_assert(kRows * D * 4 <= 2 * TILE, "the second chain's output where K is");
  static_assert(2 * kRows * 4 <= 2 * RAW, "its maxima and sums where the raw stages are");
  static_assert(2 * kRows * D * 2 <= 2 * TILE, "the output rows where V is");
  static_assert(SMALL <= 3 * 1024 - 16, "small region");
  static_assert(SMEM <= 232448, "over the shared memory of one CTA");
};

__device__ __forceinline__ float cfmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float cex2(float x) {      // -inf gives +0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ uint32_t pack_out(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack_out<__half>(float a, float b) {
  return pack_half(a, b);
}
template <>
__device__ __forceinline__ uint32_t pack_out<__nv_bfloat16>(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

__host__ __device__ inline int64_t row_tiles_of(int max_query_len, int group) {
  return ((int64_t)max_query_len * group + kCtaRows - 1) / kCtaRows;
}

// What a row tile covers: tokens i_first .. i_last of the sequence's new
// ones, keys kv_base (a multiple of the tile) .. kv_all - 1, of which those
// before kv_first are in no row's window; `count` partitions.
struct TileSpan {
  int i_first, i_last, kv_first, kv_base, kv_all, count;
};
__device__ __forceinline__ TileSpan tile_span(const ChunkArgs& a, int G, int n, int L, int qt) {
  TileSpan t;
  const int r0 = qt * kCtaRows;
  t.i_first = r0 / G;
  t.i_last = min(n - 1, (r0 + kCtaRows - 1) / G);
  t.kv_all = L - n + t.i_last + 1;
  const int p0 = L - n + t.i_first;
  t.kv_first = a.window > 0 && p0 + 1 > a.window ? p0 + 1 - a.window : 0;
  t.kv_base = t.kv_first & ~(kKv - 1);
  t.count = (t.kv_all - t.kv_base - 1) / a.partition + 1;
  return t;
}
__device__ __forceinline__ bool lengths_ok(const ChunkArgs& a, int q0, int n, int L) {
  return n >= 0 && n <= a.max_query_len && L >= n && L <= a.max_seq_len && q0 >= 0 &&
         (int64_t)q0 + n <= a.num_tokens && (int64_t)L <= a.table_stride * a.block_size;
}

// Order of the raw tiles: K0 V0 K1 V1 ..., so that a V never waits behind a K
// whose place the scores still use. Item `it` of 2n: V if odd, tile it / 2.

// Table entry of this lane's block piece of tile t (-1: none, or a piece
// that no row's window reaches, which is never looked up).
struct Pieces {
  const int32_t* trow;
  int bshift, R, npieces, kv_lo, kv_end, kv_first, ntiles;
  __device__ __forceinline__ int entry(int t, int lane) const {
    const int ts = kv_lo + t * kKv;
    const int tok = ts + lane * R;
    if (t < ntiles && lane < npieces && tok < min(kv_end, ts + kKv) && tok + R > kv_first)
      return trow[tok >> bshift];
    return -1;
  }
};

// Producer warp of K (items 0, 2, ...) or V (1, 3, ...): lane p loads piece p
// of a tile. One warp each: a box costs its lane some 90 clocks to issue, and
// a tile of 16-token blocks has eight.
// SCALED: the K warp also reads the pieces' scales, a tile ahead, and writes
// the tile's TileScales before its copies are announced.
template <int D, bool SCALED>
__device__ void produce(const ChunkArgs& a, const CUtensorMap* tm, bool isv, const Pieces& pc,
                        int kvh, uint32_t tiles, uint32_t bar, volatile uint32_t* masks,
                        TileScales* scales, volatile int* abort_flag, int raw_log2, int lane) {
  using Ly = ChunkLayout<D>;
  if (lane == 0) prefetch_tensormap(tm);
  const int n = pc.ntiles, nraw = 1 << raw_log2;
  // entries of this tile and the next are read ahead
  int e0 = pc.entry(0, lane), e1 = pc.entry(1, lane);
  int issued = 0;
  const bool with_scales = SCALED && !isv;
  float ks = 0.f, vs = 0.f, v_ref = 0.f;
  auto load_scales = [&](int e, float& k, float& v) {
    k = v = 0.f;
    if (with_scales && e >= 0 && e < a.num_blocks) {
      k = a.k_scales[(int64_t)e * a.num_kv_heads + kvh];
      v = a.v_scales[(int64_t)e * a.num_kv_heads + kvh];
    }
  };
  load_scales(e0, ks, vs);
  for (int j = 0; j < n; ++j) {
    const int it = 2 * j + (isv ? 1 : 0);
    const int ent = e0;
    e0 = e1;
    e1 = pc.entry(j + 2, lane);
    float ks_next, vs_next;
    load_scales(e0, ks_next, vs_next);
    const int ts = pc.kv_lo + j * kKv;
    const int tok = ts + lane * pc.R;
    const bool mine = ent >= 0 && ent < a.num_blocks;
    if (!isv && !mine && lane < pc.npieces && tok < min(pc.kv_end, ts + kKv) &&
        tok + pc.R > pc.kv_first)
      latch(a.err, PA_ERR_OUT_OF_RANGE);
    const unsigned pm = __ballot_sync(0xffffffffu, mine);
    const int st = it & (nraw - 1);
    int ok = 1;
    if (lane == 0 && it >= nraw)
      ok = mbar_wait_bounded(bar + 8u * (kRawEmpty + st), ((it >> raw_log2) - 1) & 1, abort_flag,
                             kWaitCycles);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) break;
    // the copies are on their way before they are announced: the barrier's
    // phase also needs the announcement's arrival
    if (mine)
      tma_load_3d(tiles + Ly::RAW_OFF + st * Ly::RAW + lane * pc.R * D, tm, 0,
                  tok & (a.block_size - 1), (int)((int64_t)ent * a.num_kv_heads + kvh),
                  bar + 8u * (kRawFull + st));
    if (with_scales) {
      // scales are positive: their bits order as they do
      float k_ref =
          __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mine ? ks : 0.f)));
      v_ref = fmaxf(v_ref, __uint_as_float(__reduce_max_sync(
                               0xffffffffu, __float_as_uint(mine ? vs : 0.f))));
      if (!(k_ref > 0.f)) k_ref = 1.f;
      TileScales* ts_out = scales + (j & (kScaleSlots - 1));
      if (lane < 16) {
        ts_out->k[lane] = ks / k_ref;
        ts_out->v[lane] = v_ref > 0.f ? vs / v_ref : 0.f;
      }
      if (lane == 0) {
        ts_out->k_ref = k_ref;
        ts_out->v_ref = v_ref;
      }
      ks = ks_next;
      vs = vs_next;
      __syncwarp();
    }
    if (lane == 0) {
      masks[st] = pm;
      mbar_arrive_expect_tx(bar + 8u * (kRawFull + st),
                            (uint32_t)__popc(pm) * (uint32_t)(pc.R * D));
    }
    issued = j + 1;
  }
  // this warp's copies land before the CTA can leave, also after a timeout: the
  // last item of each of its nraw / 2 stages (an older one's phase is over)
  if (lane == 0)
    for (int j = max(0, issued - nraw / 2); j < issued; ++j) {
      const int it = 2 * j + (isv ? 1 : 0);
      mbar_wait_drain(bar + 8u * (kRawFull + (it & (nraw - 1))), (it >> raw_log2) & 1,
                      kWaitCycles);
    }
}

// Q rows of a tile to fp16, each divided by the power of two of its largest
// magnitude (bf16 only: fp16 queries are exact as they are); the sign of a
// negative scale goes into Q, a zero scale makes it zero. `factor` gets what
// was taken out of each row. A warp takes ROWS rows from row0, D / 8 lanes to
// a row: each lane copies its 16-byte pieces to their places asynchronously
// (rows without a token are filled with zeros), then works on its own pieces
// in place, several steps at a time: one step is a chain of some 400 clocks.
template <typename T, int D, int G, int ROWS>
__device__ __forceinline__ void convert_q_rows(const ChunkArgs& a, int q0, int n, int kvh,
                                               int tile_row0, int row0, uint32_t qbase,
                                               float* factor, int lane) {
  using Ly = ChunkLayout<D>;
  constexpr int LPR = D / 8;                        // lanes of a row
  constexpr int RPS = 32 / LPR;                     // rows of a step
  constexpr int STEPS = ROWS / RPS;
  const int sub = lane / LPR, c = lane % LPR;
  const uint32_t dst0 = qbase + (c >> 3) * Ly::HALF;
#pragma unroll 4
  for (int s = 0; s < STEPS; ++s) {
    const int r = row0 + s * RPS + sub;
    const int rr = tile_row0 + r;
    const bool live = rr / G < n;
    const T* src =
        reinterpret_cast<const T*>(a.q) +
        ((int64_t)(q0 + (live ? rr / G : 0)) * a.num_q_heads + (int64_t)kvh * G + rr % G) * D +
        8 * c;
    const uint32_t dst = dst0 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(dst), "l"(src), "r"(live ? 16u : 0u) : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  const float sign = a.scale < 0.f ? -1.f : a.scale == 0.f ? 0.f : 1.f;
  constexpr int AT_ONCE = STEPS < 8 ? STEPS : 8;
#pragma unroll 1
  for (int s0 = 0; s0 < STEPS; s0 += AT_ONCE) {
    const int r0 = row0 + s0 * RPS + sub;             // rows of the steps: RPS apart
    uint4 u[AT_ONCE];
    uint32_t top[AT_ONCE];
#pragma unroll
    for (int s = 0; s < AT_ONCE; ++s) {
      const int r = r0 + s * RPS;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u[s].x), "=r"(u[s].y), "=r"(u[s].z), "=r"(u[s].w)
                   : "r"(dst0 + r * 128 + (((c & 7) ^ (r & 7)) << 4)));
    }
    if (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
      for (int s = 0; s < AT_ONCE; ++s) {
        const uint32_t w[4] = {u[s].x, u[s].y, u[s].z, u[s].w};
        top[s] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          top[s] = max(top[s], max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
      }
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
        for (int s = 0; s < AT_ONCE; ++s)
          top[s] = max(top[s], __shfl_xor_sync(0xffffffffu, top[s], o));
    }
#pragma unroll
    for (int s = 0; s < AT_ONCE; ++s) {
      const int r = r0 + s * RPS;
      float mul = sign, back = 1.f;
      if (std::is_same<T, __nv_bfloat16>::value) {
        const int ef = (int)(top[s] >> 7);           // biased exponent of the largest
        if (top[s] != 0 && ef != 255) {
          const int e = max(ef, 1);                  // factor 2^(e - 127)
          back = __uint_as_float((uint32_t)e << 23);
          // 2^(127 - e); at e = 254 it has no normal encoding
          mul *= __uint_as_float(e < 254 ? (uint32_t)(254 - e) << 23 : 1u << 22);
        }
      }
      uint32_t h[4] = {0u, 0u, 0u, 0u};
      if (sign != 0.f) {
        float f[8];
        Vec<T>::to_f32(u[s], f);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = pack_half(f[2 * k] * mul, f[2 * k + 1] * mul);
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                   ::"r"(dst0 + r * 128 + (((c & 7) ^ (r & 7)) << 4)), "r"(h[0]), "r"(h[1]),
                     "r"(h[2]), "r"(h[3]) : "memory");
      if (c == 0) factor[r] = back;
    }
  }
}

// bytes of w that hold a NaN code (x.1111.111), as 0x80 in those bytes
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// A converter lane's place: in each step the four warps take 16 token rows,
// 16 codes per lane. Codes 16c .. 16c+15 of row r become the 16-byte chunks
// 2c and 2c + 1 of the row's 64-element line (c / 4), stored at chunk ^ (r &
// 7); steps are 16 rows apart, so the places only move by whole lines. With
// head size 128, eight consecutive lanes take the first half of one row and
// the second half of the next: their 16-byte loads and their stores then hit
// eight different bank groups.
template <int D>
struct ConvLane {
  using Ly = ChunkLayout<D>;
  static constexpr int UNITS = D / 16;
  static constexpr int ROWS = 32 / UNITS * kConvWarps;   // rows per step
  static constexpr int STEPS = kKv / ROWS;
  int row;                     // row in step 0
  uint32_t src, dst0, dst1;    // byte offsets in the raw and the fp16 tile
  __device__ __forceinline__ ConvLane(int cw, int lane) {
    int c;
    if (D == 128) {
      const int b = (lane >> 2) & 1, q = lane >> 3;
      row = cw * 4 + 2 * (q >> 1) + b;
      c = (lane & 3) + 4 * (b ^ (q & 1));
    } else {
      row = cw * 8 + (lane >> 2);
      c = lane & 3;
    }
    src = row * D + c * 16;
    const int k = (2 * c) & 7;
    const uint32_t line = (c >> 2) * Ly::HALF + row * 128;
    dst0 = line + ((k ^ (row & 7)) << 4);
    dst1 = line + (((k + 1) ^ (row & 7)) << 4);
  }
};
static_assert(ConvLane<128>::ROWS % 8 == 0 && ConvLane<64>::ROWS % 8 == 0, "swizzle period");

// Raw tile -> fp16 operand tile, through registers, so that the raw stage is
// free as soon as it is read. Rows without a token become zero. clean: NaN
// codes become zero; returns whether this lane met any. SCALED: each row
// times its piece's entry of piece_scale.
template <int D>
__device__ __forceinline__ void load_raw(const ConvLane<D>& ln, uint32_t raw,
                                         uint32_t (&w)[ConvLane<D>::STEPS][4]) {
#pragma unroll
  for (int s = 0; s < ConvLane<D>::STEPS; ++s)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[s][0]), "=r"(w[s][1]), "=r"(w[s][2]), "=r"(w[s][3])
                 : "r"(raw + ln.src + s * ConvLane<D>::ROWS * D) : "memory");
}
template <int D, bool SCALED>
__device__ __forceinline__ bool convert_tile(const ConvLane<D>& ln,
                                             uint32_t (&w)[ConvLane<D>::STEPS][4], uint32_t dst,
                                             bool whole, int rows, unsigned pm, int rshift,
                                             bool clean, const float* piece_scale) {
  using CL = ConvLane<D>;
  bool seen = false;
  if (!whole) {
#pragma unroll
    for (int s = 0; s < CL::STEPS; ++s) {
      const int r = ln.row + s * CL::ROWS;
      if (!(r < rows && ((pm >> (r >> rshift)) & 1u))) w[s][0] = w[s][1] = w[s][2] = w[s][3] = 0u;
    }
  }
  if (clean) {
#pragma unroll
    for (int s = 0; s < CL::STEPS; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t nb = nan_bytes(w[s][k]);
        if (nb != 0u) {
          seen = true;
          w[s][k] &= ~((nb >> 7) * 0xffu);
        }
      }
  }
#pragma unroll
  for (int s = 0; s < CL::STEPS; ++s) {
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) e4m3x4_to_f16x2x2(w[s][k], h[2 * k], h[2 * k + 1]);
    if (SCALED) {
      const __half2 f = __float2half2_rn(piece_scale[(ln.row + s * CL::ROWS) >> rshift]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __half2 x = __hmul2(*reinterpret_cast<__half2*>(&h[k]), f);
        h[k] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(dst + ln.dst0 + s * CL::ROWS * 128), "r"(h[0]), "r"(h[1]), "r"(h[2]),
                   "r"(h[3]) : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(dst + ln.dst1 + s * CL::ROWS * 128), "r"(h[4]), "r"(h[5]), "r"(h[6]),
                   "r"(h[7]) : "memory");
  }
  return seen;
}

// MMA issue (the MMA warp, converged; its elected lane issues). The whole of
// tensor memory is allocated, so its base is 0.
//
// A chain works in halves of a key tile, 64 tokens: scores, weights over
// them, P V. That makes four streams (chain c, half h) whose S -> softmax ->
// P V -> next S cycles overlap; a stream's next scores may only be written
// once its P V has completed, so they are issued one step later, behind the
// next stream's P V. ALT: the chains take the key tiles in turn (the same Q
// tile); otherwise each takes every tile with its own Q tile.
//
// ALT and the tile count from a warp reduction keep the loop's control and
// every operand warp-uniform for the compiler.
template <int D, bool ALT>
__device__ __forceinline__ void issue(int ntiles_any, uint32_t tiles, uint32_t bar,
                                      volatile int* abort_flag) {
  using Ly = ChunkLayout<D>;
  constexpr uint32_t idS = idesc_f16(false, kRows, kHalf, false, false);
  constexpr uint32_t idO = idesc_f16(false, kRows, D, false, true);
  const int ntiles = __reduce_max_sync(0xffffffffu, ntiles_any);
  // descriptors of the first operands; the others differ by whole 16-byte
  // units in the address field (no carry: it counts the 227 KB of a CTA)
  const uint64_t q_desc = smem_desc_sw128(tiles + Ly::Q_OFF, 16, 1024);
  const uint64_t k_desc = smem_desc_sw128(tiles + Ly::K_OFF, 16, 1024);
  const uint64_t v_desc = smem_desc_sw128(tiles + Ly::V_OFF, Ly::HALF, 1024);
  const uint32_t leader = elect_one();
  auto wait = [&](int b, int parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar + 8u * b, parity & 1, abort_flag,
                                                     kWaitCycles));
  };
  constexpr int DJ = ALT ? 2 : 1;
  constexpr int PER = ALT ? 2 : 4;                  // steps of a key tile
  // scores of stream (c, h), tile j; the tile's last scores free its K
  auto issue_s = [&](int c, int h, int j) {
    if (h == 0 && (ALT || c == 0) &&
        !wait(kKFull + (j & 1), j >> 1))            // first scores of the tile
      return false;
    tc_fence_after();
    const uint64_t qd = q_desc + (c == 1 && !ALT ? (Ly::Q2_OFF - Ly::Q_OFF) >> 4 : 0);
    const uint64_t kd =
        k_desc + (uint32_t)(j & 1) * (Ly::TILE >> 4) + h * (kHalf * 128 >> 4);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      constexpr int step = Ly::HALF >> 4;
      mma_f16_ss_if(leader, c * kKv + h * kHalf, qd + (ks >> 2) * step + (ks & 3) * 2,
                    kd + (ks >> 2) * step + (ks & 3) * 2, idS, ks > 0 ? 1u : 0u);
    }
    mma_commit_if(leader, bar + 8u * (kSFull + 2 * c + h));
    if (h == 1 && (ALT || c == 1)) mma_commit_if(leader, bar + 8u * (kKEmpty + (j & 1)));
    return true;
  };
  auto issue_pv = [&](int c, int h, int j) {
    tc_fence_after();
    const uint64_t vd = v_desc + (uint32_t)(j & 1) * (Ly::TILE >> 4) + h * (kHalf * 128 >> 4);
    const uint32_t p = c * kKv + h * kHalf;
    const uint32_t more = h > 0 || j >= DJ ? 1u : 0u;
#pragma unroll
    for (int ks = 0; ks < kHalf / 16; ++ks)
      mma_f16_ts_if(leader, kOCol + c * kKv, p + ks * 8, vd + ks * (2048 >> 4), idO,
                    ks > 0 ? 1u : more);
    mma_commit_if(leader, bar + 8u * (kODone + 2 * c + h));
    if (h == 1 && (ALT || c == 1)) mma_commit_if(leader, bar + 8u * (kVEmpty + (j & 1)));
  };
  // the stream of step x (of the round's tile i in {0, 1} when ALT)
  auto chain_of = [](int i, int x) { return ALT ? i : x & 1; };
  auto half_of = [](int x) { return ALT ? x : x >> 1; };
  bool ok = wait(kQFull, 0);
  // first scores of the four streams, in the order of the steps
#pragma unroll
  for (int i = 0; i < DJ; ++i)
#pragma unroll
    for (int x = 0; x < PER; ++x)
      if (ok && i < ntiles) ok = issue_s(chain_of(i, x), half_of(x), i);
  for (int j0 = 0; ok && j0 < ntiles; j0 += DJ) {
#pragma unroll
    for (int i = 0; i < DJ; ++i) {
      const int j = j0 + i;
      if (!ok || j >= ntiles) break;
      ok = wait(kVFull + (j & 1), j >> 1);
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        const int c = chain_of(i, x), h = half_of(x);
        const int t = ALT ? j >> 1 : j;
        if (ok) ok = wait(kPFull + 2 * c + h, t);
        if (!ok) break;
        issue_pv(c, h, j);
        // the next scores of the step before this one
        const int jl = x > 0 ? j : j - 1;
        const int cl = x > 0 ? chain_of(i, x - 1) : chain_of(DJ - 1 - i, PER - 1);
        const int hl = x > 0 ? half_of(x - 1) : half_of(PER - 1);
        if (jl >= 0 && jl + DJ < ntiles)
          ok = wait(kODone + 2 * cl + hl, ALT ? jl >> 1 : jl) && issue_s(cl, hl, jl + DJ);
      }
    }
  }
  // every MMA issued above has completed once this barrier fires (waited
  // for also after a timeout, before the CTA frees its TMEM)
  mma_commit_if(leader, bar + 8u * kDone);
  mbar_wait_drain(bar + 8u * kDone, 0, kWaitCycles);
}

template <typename T, int D, int G, bool SCALED>
__global__ void __launch_bounds__(kThreads, 1)
chunk_fp8_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV) {
  using Ly = ChunkLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sbase = smem_u32(smem_raw);
  const uint32_t bar = sbase + Ly::BAR_OFF;
  const uint32_t tiles = (sbase + Ly::SMALL + 1023u) & ~1023u;
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem_raw + Ly::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + Ly::MISC_OFF + 4);
  volatile uint32_t* masks = misc + 2;
  volatile uint32_t* tile_mask = misc + 8;
  float* row_factor = reinterpret_cast<float*>(smem_raw + Ly::ROW_OFF);   // [2][128]
  TileScales* scales = reinterpret_cast<TileScales*>(smem_raw + Ly::SCALE_OFF);
  if (tiles + Ly::TILES > sbase + Ly::SMEM) {       // base too far off 1024 bytes
    if (threadIdx.x == 0) latch(a.err, PA_ERR_CUDA);
    return;
  }

  int s = blockIdx.z;
  const int kvh = blockIdx.y;
  if (a.by_length) {
    // sequence number blockIdx.z in falling order of length
    uint32_t* keys = reinterpret_cast<uint32_t*>(row_factor);
    // the length's 24 leading bits (of those max_seq_len has) and the index:
    // no two alike, and the words behind the last sequence outrank none
    const int drop = max(0, 8 - __clz(a.max_seq_len));
    if (threadIdx.x < kMaxOrdered) {
      uint32_t key = 0;
      if (threadIdx.x < a.num_seqs)
        key = (uint32_t)(min(max(a.seq_lens[threadIdx.x], 0), a.max_seq_len) >> drop) << 8 |
              (kMaxOrdered - 1 - threadIdx.x);
      keys[threadIdx.x] = key;
    }
    __syncthreads();
    // a sequence's place is the number of larger keys, counted by four threads
    const int u = threadIdx.x >> 2;
    const uint32_t mine = keys[u];
    int rank = 0;
#pragma unroll 4
    for (int x = threadIdx.x & 3; 4 * x < a.num_seqs; x += 4) {
      const uint4 k = reinterpret_cast<const uint4*>(keys)[x];
      rank += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
    }
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    if (u < a.num_seqs && rank == (int)blockIdx.z) misc[7] = u;
    __syncthreads();
    s = misc[7];
  }
  const int row_tiles = (int)row_tiles_of(a.max_query_len, G);
  const int qt = row_tiles - 1 - (int)(blockIdx.x % row_tiles);    // longest rows first
  const int split = (int)(blockIdx.x / row_tiles);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q0 = a.qsl[s];
  const int n = a.qsl[s + 1] - q0;
  const int L = a.seq_lens[s];
  if (!lengths_ok(a, q0, n, L)) {
    if (blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0) latch(a.err, PA_ERR_OUT_OF_RANGE);
    return;
  }
  const int r0 = qt * kCtaRows;
  if (r0 >= n * G) return;
  const TileSpan sp = tile_span(a, G, n, L, qt);
  if (split >= sp.count) return;
  const int kv_lo = sp.kv_base + split * a.partition;
  const int kv_end = kv_lo + min(sp.kv_all - kv_lo, a.partition);
  const int ntiles = (kv_end - kv_lo + kKv - 1) / kKv;
  const bool alt = n * G - r0 <= kRows;             // one row tile: key tiles in turn
  const int raw_log2 = alt ? 2 : 1, nraw = 1 << raw_log2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxRaw; ++i) {
      mbar_init(bar + 8u * (kRawFull + i), 1);
      mbar_init(bar + 8u * (kRawEmpty + i), kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + 8u * (kKFull + i), kConvWarps);
      mbar_init(bar + 8u * (kKEmpty + i), 1);
      mbar_init(bar + 8u * (kVFull + i), kConvWarps);
      mbar_init(bar + 8u * (kVEmpty + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar + 8u * (kSFull + i), 1);
      mbar_init(bar + 8u * (kPFull + i), 4);
      mbar_init(bar + 8u * (kODone + i), 1);
    }
    mbar_init(bar + 8u * kDone, 1);
    mbar_init(bar + 8u * kQFull, 8);
    mbar_init(bar + 8u * kConvDone, kConvWarps);
    *abort_flag = 0;
    misc[6] = 0;                                    // NaN codes cleared in this CTA
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sbase + Ly::MISC_OFF, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  const int B = a.block_size;
  Pieces pc;
  pc.trow = a.tables + (int64_t)s * a.table_stride;
  pc.bshift = __ffs(B) - 1;
  pc.R = B < kKv ? B : kKv;
  pc.npieces = kKv / pc.R;
  pc.kv_lo = kv_lo;
  pc.kv_end = kv_end;
  pc.kv_first = sp.kv_first;
  pc.ntiles = ntiles;
  const int rshift = __ffs(pc.R) - 1;
  const unsigned full_mask = (1u << pc.npieces) - 1u;              // at most 16 pieces
  // a tile that every row sees whole ends at or before pos_first and starts
  // at or after lo_last
  const int pos_first = L - n + sp.i_first;
  const int lo_last = a.window > 0 ? max(0, L - n + sp.i_last + 1 - a.window) : 0;

  if (warp < kSoftmaxWarp) {
    if (warp == kProducerWarp || warp == kProducerWarp + 1) {
      const bool isv = warp > kProducerWarp;
      produce<D, SCALED>(a, isv ? &tmV : &tmK, isv, pc, kvh, tiles, bar, masks, scales,
                         abort_flag, raw_log2, lane);
    } else if (warp == kMmaWarp) {
      if (tmem != 0) *abort_flag = 1;
      else if (alt) issue<D, true>(ntiles, tiles, bar, abort_flag);
      else issue<D, false>(ntiles, tiles, bar, abort_flag);
      __syncwarp();
    } else if (warp >= kConvWarp) {
      const int cw = warp - kConvWarp;
      const ConvLane<D> ln(cw, lane);
      for (int it = 0; it < 2 * ntiles; ++it) {
        const int j = it >> 1;
        const bool isv = (it & 1) != 0;
        const int rs = it & (nraw - 1), st = j & 1;
        bool ok = mbar_wait_bounded(bar + 8u * (kRawFull + rs), (it >> raw_log2) & 1, abort_flag,
                                    kWaitCycles);
        if (!__all_sync(0xffffffffu, ok)) break;
        const unsigned pm = masks[rs];
        uint32_t w[ConvLane<D>::STEPS][4];
        load_raw<D>(ln, tiles + Ly::RAW_OFF + rs * Ly::RAW, w);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + 8u * (kRawEmpty + rs));
        if (j >= 2)
          ok = mbar_wait_bounded(bar + 8u * ((isv ? kVEmpty : kKEmpty) + st), ((j >> 1) - 1) & 1,
                                 abort_flag, kWaitCycles);
        if (!__all_sync(0xffffffffu, ok)) break;
        const int ts = kv_lo + j * kKv;
        const int rows = min(kKv, kv_end - ts);
        const bool clean = isv && (ts + kKv - 1 > pos_first || ts < lo_last);
        const bool seen =
            convert_tile<D, SCALED>(ln, w, tiles + (isv ? Ly::V_OFF : Ly::K_OFF) + st * Ly::TILE,
                                    pm == full_mask && rows == kKv, rows, pm, rshift, clean,
                                    isv ? scales[j & (kScaleSlots - 1)].v
                                        : scales[j & (kScaleSlots - 1)].k);
        if (seen) misc[6] = 1;
        // (a slot is used again four tiles on, when S of the tile two on, and
        // so the softmax of this one, is long over)
        if (!isv && cw == 0 && lane == 0) tile_mask[j & 3] = pm;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar + 8u * ((isv ? kVFull : kKFull) + st));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + 8u * kConvDone);
    }
  } else {
    // ---- softmax of chain c: thread = row r of its tile
    const int c = (warp - kSoftmaxWarp) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int rr = r0 + (alt ? 0 : c * kRows) + r;
    const int i = rr / G;
    const bool rv = i < n;
    const int pos = rv ? L - n + i : -1;
    const int lo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
    const bool idle = __all_sync(0xffffffffu, !rv);   // no row here holds a token
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sadr = tmem + lanes + c * kKv;
    const uint32_t oadr = tmem + lanes + kOCol + c * kKv;
    // the Q tiles: each chain its own, or both the one
    if (alt)
      convert_q_rows<T, D, G, 16>(a, q0, n, kvh, r0, (warp - kSoftmaxWarp) * 16,
                                  tiles + Ly::Q_OFF, row_factor, lane);
    else
      convert_q_rows<T, D, G, 32>(a, q0, n, kvh, r0 + c * kRows, (warp & 3) * 32,
                                  tiles + (c == 0 ? Ly::Q_OFF : Ly::Q2_OFF),
                                  row_factor + c * kRows, lane);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + 8u * kQFull);
    bool ok = mbar_wait_bounded(bar + 8u * kQFull, 0, abort_flag, kWaitCycles);
    // logit factor in the log2 domain (Q carries the scale's sign and zero)
    const float f0 = (a.scale == 0.f ? 1.f : fabsf(a.scale)) * kLog2e *
                     (SCALED ? 1.f : a.k_scale) * row_factor[(alt ? 0 : c * kRows) + r];

    // this chain's tiles: j = j0, j0 + dj, ...; those that begin at fast_lo or
    // later and end by fast_hi are seen whole by every row of the warp
    const int j0 = alt ? c : 0, dj = alt ? 2 : 1;
    const int fast_lo = __reduce_max_sync(0xffffffffu, rv ? lo : 0);
    const int fast_hi = __reduce_min_sync(0xffffffffu, rv ? pos + 1 : 0x7fffffff);
    float m_use = kNegInfC, l = 0.f, vref = 0.f;
    int t = 0;
    for (int j = j0; j < ntiles; j += dj, ++t) {
      const int ts = kv_lo + j * kKv;
      const int te = min(kv_end, ts + kKv);
      float alpha_v = 1.f, f = f0;
      // the tile in two steps of 64 tokens
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        ok = mbar_wait_bounded(bar + 8u * (kSFull + 2 * c + h), t & 1, abort_flag, kWaitCycles);
        ok = __all_sync(0xffffffffu, ok);
        if (__builtin_expect(!ok, 0)) break;
        tc_fence_after();
        if (!idle) {
          uint32_t v[kHalf];
          const unsigned pm = tile_mask[j & 3];
          if (SCALED && h == 0) {
            const TileScales& sc = scales[j & (kScaleSlots - 1)];
            f = f0 * sc.k_ref;
            if (vref > 0.f) alpha_v = vref / sc.v_ref;
            vref = sc.v_ref;
          }
          tmem_ld64(sadr + h * kHalf, v);
          const bool whole = pm == full_mask && te - ts == kKv;
          // rare paths are marked as such, which keeps the common one together
          if (__builtin_expect(!(whole && ts >= fast_lo && te <= fast_hi), 0)) {
            // what a row does not see becomes -inf in place: weight 0 below;
            // rows without a token keep their scores, 0
            const int hi = rv ? min(pos, te - 1) - ts : kKv;     // last column in sight
            const int first = rv ? lo - ts : 0;                  // first column in sight
#pragma unroll
            for (int ch = 0; ch < kHalf / 32; ++ch) {
              const int c0 = h * kHalf + ch * 32;
              uint32_t m = hi < c0 ? 0u : hi >= c0 + 31 ? 0xffffffffu : (2u << (hi - c0)) - 1u;
              if (first > c0) m &= first > c0 + 31 ? 0u : 0xffffffffu << (first - c0);
              if (!whole) {
                uint32_t p = 0;
                if (pc.R >= 32) {
                  p = ((pm >> (c0 >> rshift)) & 1u) ? 0xffffffffu : 0u;
                } else {
                  for (int k = 0; k < 32 / pc.R; ++k)
                    if ((pm >> ((c0 >> rshift) + k)) & 1u) p |= ((1u << pc.R) - 1u) << (k * pc.R);
                }
                m &= p;
              }
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((m >> e) & 1u)) v[ch * 32 + e] = __float_as_uint(kNegInfC);
            }
          }
          // pass 1: the maximum
          float m4[4] = {kNegInfC, kNegInfC, kNegInfC, kNegInfC};
#pragma unroll
          for (int e = 0; e < kHalf; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m4[k] = cfmax3(m4[k], __uint_as_float(v[e + 2 * k]),
                             __uint_as_float(v[e + 2 * k + 1]));
          const float mx = cfmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]) * f;
          const float m_new = fmaxf(m_use, mx);
          float alpha = 1.f;
          if (m_use == kNegInfC) {
            m_use = m_new;                           // nothing accumulated yet
          } else if (m_new > m_use + kLazyLog2) {
            alpha = exp2f(m_use - m_new);
            m_use = m_new;
          }
          // pass 2: P = 2^(x - m_use) in fp16 over this row's own scores; a
          // row that has seen nothing has only -inf scores and weights of 0
          const float nm = m_use == kNegInfC ? 0.f : -m_use;
          uint64_t sum0 = pair(0.f, 0.f), sum1 = sum0;
          const uint64_t cm = pair(nm, nm);
          const uint64_t fm = pair(f, f);
#pragma unroll
          for (int ch = 0; ch < kHalf / 32; ++ch) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              unpair(fma_pair(pair(__uint_as_float(v[ch * 32 + e]),
                                   __uint_as_float(v[ch * 32 + e + 1])), fm, cm), x0, x1);
              x0 = cex2(x0);
              x1 = cex2(x1);
              const uint64_t p = pair(x0, x1);
              if (e & 2) sum1 = add_pair(sum1, p); else sum0 = add_pair(sum0, p);
              pk[e >> 1] = pack_half(x0, x1);
            }
            tmem_st16(sadr + h * kHalf + ch * 16, pk);
          }
          float s0, s1;
          unpair(add_pair(sum0, sum1), s0, s1);
          l = l * alpha + (s0 + s1);
          const float alpha_o = SCALED && h == 0 ? alpha * alpha_v : alpha;
          if (__builtin_expect(t + h >= 1 && __any_sync(0xffffffffu, alpha_o != 1.f), 0)) {
            // after the P V of the step before
            ok = mbar_wait_bounded(bar + 8u * (kODone + 2 * c + (h ^ 1)), (t - 1 + h) & 1,
                                   abort_flag, kWaitCycles);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (ok) {
#pragma unroll 1
              for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t o[32];
                tmem_ld32(oadr + ch * 32, o);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha_o);
                tmem_st32(oadr + ch * 32, o);
              }
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + 8u * (kPFull + 2 * c + h));
      }
      if (!ok) break;
    }
    if (ok) ok = mbar_wait_bounded(bar + 8u * kDone, 0, abort_flag, kWaitCycles);
    if (ok) ok = mbar_wait_bounded(bar + 8u * kConvDone, 0, abort_flag, kWaitCycles);
    tc_fence_after();
    ok = __all_sync(0xffffffffu, ok);
    const float unit = SCALED ? vref : a.v_scale;
    // one row tile: the second chain hands its row over (its output where
    // the K tiles were: 16-byte pieces of a row, spread over the banks)
    float4* second_o =
        reinterpret_cast<float4*>(smem_raw + (tiles - sbase) + Ly::K_OFF);
    constexpr int PIECES = D / 4;
    float* second_ml =
        reinterpret_cast<float*>(smem_raw + (tiles - sbase) + Ly::RAW_OFF);   // [2][128]
    if (alt && c == 1) {
      if (ok && t > 0 && !idle) {
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tmem_ld32(oadr + ch * 32, o);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            second_o[r * PIECES + ((ch * 8 + k) ^ (r & 7))] =
                make_float4(__uint_as_float(o[4 * k]) * unit, __uint_as_float(o[4 * k + 1]) * unit,
                            __uint_as_float(o[4 * k + 2]) * unit,
                            __uint_as_float(o[4 * k + 3]) * unit);
        }
      }
      second_ml[r] = t > 0 ? m_use : kNegInfC;
      second_ml[kRows + r] = t > 0 ? l : 0.f;
    }
    if (alt) asm volatile("bar.sync 1, 256;" ::: "memory");
    if (ok && !idle && !(alt && c == 1)) {
      float w1 = 1.f, w2 = 0.f;                      // the chains' weights
      if (alt) {
        const float m2 = second_ml[r], l2 = second_ml[kRows + r];
        if (!(m2 == kNegInfC && l2 == 0.f)) {
          const float m = fmaxf(m_use, m2);
          w1 = m_use == kNegInfC && l == 0.f ? 0.f : exp2f(m_use - m);
          w2 = exp2f(m2 - m);
          l = l * w1 + l2 * w2;
          m_use = m;
        }
      }
      const int64_t tok = q0 + i;
      const int head = kvh * G + rr % G;
      const bool direct = rv && sp.count == 1;
      const bool partial = rv && sp.count > 1;
      const float inv = direct ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
      const float mul1 = unit * w1 * inv, mul2 = w2 * inv;
      const bool second = alt && ntiles > 1 && w2 != 0.f;
      const bool nans = misc[6] != 0;
      const int64_t slot = (tok * a.num_q_heads + head) * a.num_splits + split;
      // where the V tiles were: 32 rows of this warp
      constexpr int OUTS = D / 8;                    // 16-byte pieces of an output row
      uint4* strip = reinterpret_cast<uint4*>(smem_raw + (tiles - sbase) + Ly::V_OFF) +
                     (warp - kSoftmaxWarp) * 32 * OUTS;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        const int c0 = ch * 32;
        uint32_t o[32];
        tmem_ld32(oadr + c0, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * mul1);
        if (second) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 f = second_o[r * PIECES + ((ch * 8 + k) ^ (r & 7))];
            o[4 * k] = __float_as_uint(fmaf(f.x, mul2, __uint_as_float(o[4 * k])));
            o[4 * k + 1] = __float_as_uint(fmaf(f.y, mul2, __uint_as_float(o[4 * k + 1])));
            o[4 * k + 2] = __float_as_uint(fmaf(f.z, mul2, __uint_as_float(o[4 * k + 2])));
            o[4 * k + 3] = __float_as_uint(fmaf(f.w, mul2, __uint_as_float(o[4 * k + 3])));
          }
        }
        if (nans && rv) {
          // columns in which a token that this row sees, in a cleared tile,
          // holds a NaN
          uint32_t bad = 0;
          for (int j = 0; j < ntiles; ++j) {
            const int ts = kv_lo + j * kKv;
            if (!(ts + kKv - 1 > pos_first || ts < lo_last)) continue;
            for (int x = max(ts, lo); x <= min(min(ts + kKv, kv_end) - 1, pos); ++x) {
              const int64_t b = pc.trow[x >> pc.bshift];
              if (b < 0 || b >= a.num_blocks) continue;
              const uint32_t* codes = reinterpret_cast<const uint32_t*>(
                  static_cast<const uint8_t*>(a.vc) +
                  ((b * a.num_kv_heads + kvh) * B + (x & (B - 1))) * D + c0);
              for (int k = 0; k < 8; ++k) {
                const uint32_t nb = nan_bytes(codes[k]);
                for (int z = 0; z < 4; ++z)
                  if ((nb >> (8 * z + 7)) & 1u) bad |= 1u << (4 * k + z);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((bad >> e) & 1u) o[e] = 0x7fffffffu;
        }
        if (direct) {
          // own row to this warp's strip, 16-byte pieces spread over the banks
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 w;
            w.x = pack_out<T>(__uint_as_float(o[8 * q + 0]), __uint_as_float(o[8 * q + 1]));
            w.y = pack_out<T>(__uint_as_float(o[8 * q + 2]), __uint_as_float(o[8 * q + 3]));
            w.z = pack_out<T>(__uint_as_float(o[8 * q + 4]), __uint_as_float(o[8 * q + 5]));
            w.w = pack_out<T>(__uint_as_float(o[8 * q + 6]), __uint_as_float(o[8 * q + 7]));
            strip[lane * OUTS + ((ch * 4 + q) ^ (lane & 7))] = w;
          }
        } else if (partial) {
          uint4* acc = reinterpret_cast<uint4*>(a.ws_acc + slot * D + c0);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            acc[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      if (partial) {
        a.ws_ml[2 * slot] = m_use;
        a.ws_ml[2 * slot + 1] = l;
      }
      if (sp.count == 1) {
        // whole rows to memory: a row per D / 8 lanes
        T* out = reinterpret_cast<T*>(a.out);
        __syncwarp();
#pragma unroll 4
        for (int x = lane; x < 32 * OUTS; x += 32) {
          const int wr = x / OUTS, q = x % OUTS;
          const int row = rr - lane + wr;            // row of the sequence
          if (row / G < n)
            reinterpret_cast<uint4*>(
                out + ((int64_t)(q0 + row / G) * a.num_q_heads + kvh * G + row % G) * D)[q] =
                strip[wr * OUTS + (q ^ (wr & 7))];
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) latch(a.err, PA_ERR_TIMEOUT);
}

// Log-sum-exp merge of the partitions of one (new token, query head) row;
// rows of tiles with one partition were written by the attention kernel.
template <typename T, int D, int G>
__global__ void __launch_bounds__(D) chunk_combine_kernel(const ChunkArgs a) {
  const int64_t t = blockIdx.x;
  const int head = blockIdx.y, d = threadIdx.x;
  int lo = 0, hi = a.num_seqs + 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)a.qsl[mid] <= t) lo = mid + 1; else hi = mid;
  }
  const int s = lo - 1;
  if (s < 0 || s >= a.num_seqs) return;
  const int q0 = a.qsl[s], n = a.qsl[s + 1] - q0, L = a.seq_lens[s];
  if (!lengths_ok(a, q0, n, L)) return;
  const TileSpan sp = tile_span(a, G, n, L, (int)(((t - q0) * G + head % G) / kCtaRows));
  if (sp.count <= 1) return;
  const int64_t base = (t * a.num_q_heads + head) * a.num_splits;
  float M = kNegInfC;
  for (int p = 0; p < sp.count; ++p) M = fmaxf(M, a.ws_ml[2 * (base + p)]);
  float Ls = 0.f, O = 0.f;
  for (int p = 0; p < sp.count; ++p) {
    const float mp = a.ws_ml[2 * (base + p)];
    const float lp = a.ws_ml[2 * (base + p) + 1];
    if (mp == kNegInfC && lp == 0.f) continue;      // this row sees nothing there
    const float w = exp2f(mp - M);
    Ls += lp * w;
    O += a.ws_acc[(base + p) * D + d] * w;
  }
  reinterpret_cast<T*>(a.out)[(t * a.num_q_heads + head) * D + d] =
      Vec<T>::cvt_out(Ls != 0.f ? O / Ls : 0.f);
}

PFN_cuTensorMapEncodeTiled_v12000 g_chunk_encode = nullptr;
std::once_flag g_chunk_encode_once;

bool chunk_encoder() {
  std::call_once(g_chunk_encode_once, []() {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_chunk_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_chunk_encode != nullptr;
}

// pool [NB][Hkv][B][D] of codes as {D, B, NB*Hkv}: a box is R rows of a slice
bool encode_codes(CUtensorMap* map, const void* base, int D, int B, uint64_t planes, int R) {
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)B, planes};
  cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)B * D};
  cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)R, 1u};
  cuuint32_t es[3] = {1, 1, 1};
  return g_chunk_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims,
                        strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int G, bool SCALED>
cudaError_t launch_chunk(const ChunkArgs& a, cudaStream_t st) {
  using Ly = ChunkLayout<D>;
  if (!chunk_encoder()) return cudaErrorNotSupported;
  const uint64_t planes = (uint64_t)a.num_blocks * a.num_kv_heads;
  if (planes == 0 || planes > 0x7fffffffull) return cudaErrorInvalidValue;
  const int R = a.block_size < kKv ? a.block_size : kKv;
  CUtensorMap tk, tv;
  if (!encode_codes(&tk, a.kc, D, a.block_size, planes, R) ||
      !encode_codes(&tv, a.vc, D, a.block_size, planes, R))
    return cudaErrorInvalidValue;
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, []() {
    attr = cudaFuncSetAttribute(chunk_fp8_kernel<T, D, G, SCALED>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::SMEM);
  });
  if (attr != cudaSuccess) return attr;
  const int64_t row_tiles = row_tiles_of(a.max_query_len, G);
  if (row_tiles * a.num_splits > 0x7fffffffll) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(row_tiles * a.num_splits), a.num_kv_heads, a.num_seqs);
  chunk_fp8_kernel<T, D, G, SCALED><<<grid, kThreads, Ly::SMEM, st>>>(a, tk, tv);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.num_splits <= 1) return e;
  const dim3 cgrid((unsigned)a.num_tokens, a.num_q_heads);
  chunk_combine_kernel<T, D, G><<<cgrid, D, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D, int G>
cudaError_t launch_chunk_s(const ChunkArgs& a, cudaStream_t st) {
  return a.k_scales != nullptr ? launch_chunk<T, D, G, true>(a, st)
                               : launch_chunk<T, D, G, false>(a, st);
}

template <typename T, int D>
cudaError_t launch_chunk_g(const ChunkArgs& a, cudaStream_t st) {
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch_chunk_s<T, D, 1>(a, st);
    case 2: return launch_chunk_s<T, D, 2>(a, st);
    case 4: return launch_chunk_s<T, D, 4>(a, st);
    case 8: return launch_chunk_s<T, D, 8>(a, st);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_chunk_d(const ChunkArgs& a, cudaStream_t st) {
  if (a.head_size == 64) return launch_chunk_g<T, 64>(a, st);
  if (a.head_size == 128) return launch_chunk_g<T, 128>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace

// Keys a CTA's rows can span (the kernel's tile_span).
static int64_t span_of(int group, int max_query_len, int max_seq_len, int window) {
  const int64_t len = max_seq_len > 0 ? max_seq_len : 1;
  if (window <= 0) return len;
  const int64_t toks =
      std::min<int64_t>(max_query_len, kCtaRows / group);
  return std::min<int64_t>(len, (int64_t)window - 1 + toks + kKv - 1);
}

// Whether CTAs take the sequences in falling order of length. A ragged batch
// in the order given leaves some SMs with a long sequence at the end; with
// CTAs for one to sixteen waves (more even out by themselves) the longest
// first shortens that tail, for a search of some 1,000 clocks per CTA, which
// short sequences would feel. In the order given and by length: 128 sequences
// of 1k to 8k tokens 385 and 362 us, 32 chunks of 128 after 0 to 4k 312 and
// 294; all of 4k 315 and 320; 128 of 100 to 400 tokens 75.6 and 78.8.
bool chunk_by_length(int num_seqs, int num_kv_heads, int group, int max_query_len, int max_seq_len,
                     int sm_count, int splits) {
  const int64_t ctas = row_tiles_of(max_query_len, group) * num_kv_heads * num_seqs;
  return num_seqs > 1 && num_seqs <= kMaxOrdered && max_seq_len >= 2048 && splits == 1 &&
         ctas > sm_count && ctas <= 16 * (int64_t)sm_count;
}

// Partitions of the keys, where the CTAs alone would leave SMs idle: the
// number that minimises the waves' keys, with 256 tokens' time for the start
// of a CTA and again for the merge. With a wave of CTAs or more there is
// little to gain, and the parts of ragged sequences cannot be taken longest
// first; unsplit against split (4 tokens a sequence, 8 KV heads): 32
// sequences of 1k to 8k tokens 98 and 134 us, 64 of them 182 and 225, 36 of
// 6k 129 and 129, 24 of 6k 127 and 112. Below a wave: 12 of 1k to 8k 83 and
// 69, 8 of 4k 47 and 32, one of 8k 82 and 17.
void chunk_plan(int num_seqs, int num_kv_heads, int group, int max_query_len, int max_seq_len,
                int window, int partition_size, int sm_count, int* splits, int* tokens) {
  const int64_t len = span_of(group, max_query_len, max_seq_len, window);
  auto round_up = [](int64_t x) { return (x + kKv - 1) / kKv * kKv; };
  int64_t P = round_up(len);
  if (partition_size > 0) {
    P = std::min(P, round_up(partition_size));
  } else {
    const int64_t ctas = std::max<int64_t>(
        1, row_tiles_of(max_query_len, group) * num_kv_heads * num_seqs);
    if (ctas < (int64_t)sm_count) {
      int64_t best = -1;
      for (int64_t k = 1; k <= 64 && (k == 1 || len / k >= 256); ++k) {
        const int64_t p = round_up((len + k - 1) / k);
        const int64_t waves = (ctas * k + sm_count - 1) / sm_count;
        const int64_t cost = waves * (p + 256) + (k > 1 ? 256 : 0);
        if (best < 0 || cost < best) {
          best = cost;
          P = p;
        }
      }
    }
  }
  P = std::min<int64_t>(P, 1 << 30);
  *tokens = (int)P;
  *splits = (int)((len + P - 1) / P);
}

cudaError_t launch_chunk_fp8(const ChunkArgs& a, cudaStream_t st) {
  if (a.dtype == PA_BF16) return launch_chunk_d<__nv_bfloat16>(a, st);
  if (a.dtype == PA_F16) return launch_chunk_d<__half>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace pa
