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
// One CTA owns 128 rows, (new token, query head) pairs of one KV head, and
// walks their keys in tiles of 128 tokens:
//   * a producer warp brings the tiles' codes (K and V in the order in which
//     the MMAs need them) by 3-D TMA boxes, one per block piece, into a ring
//     of four raw stages;
//   * four converter warps widen each raw tile to fp16 (E4M3 is exact in
//     fp16) into the 128-byte-swizzled operand layout of the MMA, two stages
//     each of K and V, and clear rows without a token on the way. They also
//     build the Q tile: fp16 with each row divided by a power of two, so
//     that a bf16 query keeps its 8 significant bits down to 2^-24 of the
//     row's largest value;
//   * one thread issues S = Q K^T into one of two TMEM score buffers and
//     O += P V with P (fp16, over the scores) read from TMEM;
//   * eight softmax warps, half a row per thread, keep the running maximum
//     and the sum in fp32 registers; the output in TMEM is rescaled only
//     when a row's maximum grew by more than 2^8.
// fp16 products for both query types: weights are rounded to 11 bits, one
// rounding, in [0, 2^8].
//
// Per-block scales: a K scale multiplies the scores of its block's columns
// in fp32; a V scale relative to the largest one seen so far (at most 1)
// multiplies the weights before their rounding, and the output is rescaled
// when that reference grows, so no weight overflows and none loses more than
// with one scale equal to the reference. The sums use the unscaled weights.
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

constexpr int kRows = 128;                // query rows per CTA (MMA M)
constexpr int kKv = 128;                  // KV tokens per tile
constexpr int kRaw = 4;                   // raw stages
constexpr int kSoftmaxWarps = 8;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kConvWarp = 10;             // first of four
constexpr int kConvWarps = 4;
constexpr int kThreads = (kConvWarp + kConvWarps) * 32;
constexpr int kCols = kKv / 2;            // score columns per softmax thread
constexpr uint32_t kTmemCols = 512;       // S0 [0,128), S1 [128,256), O [256,256+D)
constexpr uint32_t kOCol = 256;
constexpr long long kWaitCycles = 4000000000LL;
constexpr float kLazyLog2 = 8.f;
#define kNegInfC (-__int_as_float(0x7f800000))

enum : int {
  kRawFull = 0, kRawEmpty = kRaw, kKFull = 2 * kRaw, kKEmpty = kKFull + 2, kVFull = kKEmpty + 2,
  kVEmpty = kVFull + 2, kSFull = kVEmpty + 2, kPFull = kSFull + 2, kODone, kDone, kQFull, kConvDone,
  kBars
};

template <int D>
struct ChunkLayout {
  // small things first, so that the 1024-byte aligned tiles end exactly at
  // the limit of 227 KB for head size 128
  static constexpr int BAR_OFF = 0;
  static constexpr int MISC_OFF = (kBars * 8 + 15) / 16 * 16;   // tmem base, abort, masks, NaN
  static constexpr int XCH_OFF = MISC_OFF + 32;                 // float [2][2][128]
  static constexpr int SMALL = XCH_OFF + 2 * 2 * kRows * 4;
  static constexpr int HALVES = D / 64;
  static constexpr int HALF = kKv * 128;                        // 128 rows x 64 fp16
  static constexpr int TILE = HALVES * HALF;
  static constexpr int RAW = kKv * D;
  static constexpr int Q_OFF = 0;                               // from the aligned base
  static constexpr int K_OFF = TILE;
  static constexpr int V_OFF = K_OFF + 2 * TILE;
  static constexpr int RAW_OFF = V_OFF + 2 * TILE;
  static constexpr int TILES = RAW_OFF + kRaw * RAW;
  static constexpr int SMEM = 3 * 1024 + TILES;
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
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
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

// Barrier 1 over the softmax warps that also returns whether all passed `ok`.
__device__ __forceinline__ bool softmax_all(bool ok) {
  uint32_t out;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n"
      " barrier.cta.red.and.pred po, 1, 256, pi;\n selp.u32 %0, 1, 0, po;\n}\n"
      : "=r"(out) : "r"((uint32_t)ok) : "memory");
  return out != 0;
}

// What a row tile covers: tokens i_first .. i_last of the sequence's new
// ones, keys kv_base (a multiple of the tile) .. kv_all - 1, of which those
// before kv_first are in no row's window; `count` partitions.
struct TileSpan {
  int i_first, i_last, kv_first, kv_base, kv_all, count;
};
__device__ __forceinline__ TileSpan tile_span(const ChunkArgs& a, int G, int n, int L, int qt) {
  TileSpan t;
  const int r0 = qt * kRows;
  t.i_first = r0 / G;
  t.i_last = min(n - 1, (r0 + kRows - 1) / G);
  t.kv_all = L - n + t.i_last + 1;
  const int p0 = L - n + t.i_first;
  t.kv_first = a.window > 0 && p0 + 1 > a.window ? p0 + 1 - a.window : 0;
  t.kv_base = t.kv_first & ~(kKv - 1);
  t.count = (t.kv_all - t.kv_base + a.partition - 1) / a.partition;
  return t;
}
__device__ __forceinline__ bool lengths_ok(const ChunkArgs& a, int q0, int n, int L) {
  return n >= 0 && n <= a.max_query_len && L >= n && L <= a.max_seq_len && q0 >= 0 &&
         (int64_t)q0 + n <= a.num_tokens && (int64_t)L <= a.table_stride * a.block_size;
}

// Order of the raw tiles: K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1), as the
// MMAs consume them. Item `it` of 2n: true for V, *j its tile.
__device__ __forceinline__ bool item_of(int it, int n, int* j) {
  if (it == 0) { *j = 0; return false; }
  if (it & 1) {
    *j = (it + 1) >> 1;
    if (*j < n) return false;
    *j = n - 1;
    return true;
  }
  *j = (it - 2) >> 1;
  return true;
}

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

template <int D>
__device__ void produce(const ChunkArgs& a, const CUtensorMap* tmK, const CUtensorMap* tmV,
                        const Pieces& pc, int kvh, uint32_t tiles, uint32_t bar,
                        volatile uint32_t* masks, volatile int* abort_flag, int lane) {
  using Ly = ChunkLayout<D>;
  if (lane == 0) {
    prefetch_tensormap(tmK);
    prefetch_tensormap(tmV);
  }
  const int n = pc.ntiles;
  // entries of the K tile to come and of the one behind it are read ahead;
  // the two K tiles gone by are kept for their V
  int e0 = pc.entry(0, lane), e1 = pc.entry(1, lane), h0 = -1, h1 = -1;
  int issued = 0;
  for (int it = 0; it < 2 * n; ++it) {
    int j;
    const bool isv = item_of(it, n, &j);
    int ent;
    if (!isv) {
      ent = e0;
      h1 = h0;
      h0 = e0;
      e0 = e1;
      e1 = pc.entry(j + 2, lane);
    } else {
      ent = j == n - 1 ? h0 : h1;
    }
    const int ts = pc.kv_lo + j * kKv;
    const int tok = ts + lane * pc.R;
    const bool mine = ent >= 0 && ent < a.num_blocks;
    if (!isv && !mine && lane < pc.npieces && tok < min(pc.kv_end, ts + kKv) &&
        tok + pc.R > pc.kv_first)
      latch(a.err, PA_ERR_OUT_OF_RANGE);
    const unsigned pm = __ballot_sync(0xffffffffu, mine);
    const int st = it % kRaw;
    int ok = 1;
    if (lane == 0) {
      if (it >= kRaw)
        ok = mbar_wait_bounded(bar + 8u * (kRawEmpty + st), ((it / kRaw) - 1) & 1, abort_flag,
                               kWaitCycles);
      if (ok) {
        masks[st] = pm;
        mbar_arrive_expect_tx(bar + 8u * (kRawFull + st),
                              (uint32_t)__popc(pm) * (uint32_t)(pc.R * D));
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) break;
    if (mine)
      tma_load_3d(tiles + Ly::RAW_OFF + st * Ly::RAW + lane * pc.R * D, isv ? tmV : tmK, 0,
                  tok & (a.block_size - 1), (int)((int64_t)ent * a.num_kv_heads + kvh),
                  bar + 8u * (kRawFull + st));
    issued = it + 1;
  }
  // this warp's copies land before the CTA can leave, also after a timeout
  if (lane == 0)
    for (int i = issued > kRaw ? issued - kRaw : 0; i < issued; ++i)
      mbar_wait_drain(bar + 8u * (kRawFull + i % kRaw), (i / kRaw) & 1, kWaitCycles);
}

// Q row r of the tile to fp16, divided by the power of two of its largest
// magnitude (bf16 only: fp16 queries are exact as they are); the sign of a
// negative scale goes into Q, a zero scale makes it zero. Returns the factor
// taken out.
template <typename T, int D>
__device__ __forceinline__ float convert_q_row(const T* src, bool live, float scale,
                                               uint32_t qbase, int r) {
  using Ly = ChunkLayout<D>;
  float mul = scale < 0.f ? -1.f : scale == 0.f ? 0.f : 1.f, back = 1.f;
  if (std::is_same<T, __nv_bfloat16>::value && live) {
    uint32_t top = 0;
    for (int c = 0; c < D / 8; ++c) {
      const uint4 u = *reinterpret_cast<const uint4*>(src + 8 * c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
    }
    const int ef = (int)(top >> 7);                  // biased exponent of the largest
    if (top != 0 && ef != 255) {
      const int e = max(ef, 1);                      // factor 2^(e - 127)
      back = __uint_as_float((uint32_t)e << 23);
      // 2^(127 - e), in two steps where it has no normal encoding
      mul *= e < 254 ? __uint_as_float((uint32_t)(254 - e) << 23)
                     : __uint_as_float(1u << 22);
    }
  }
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    uint32_t h[4] = {0u, 0u, 0u, 0u};
    if (live && mul != 0.f) {
      float f[8];
      Vec<T>::to_f32(*reinterpret_cast<const uint4*>(src + 8 * c), f);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = pack_half(f[2 * k] * mul, f[2 * k + 1] * mul);
    }
    const uint32_t dst = qbase + (c >> 3) * Ly::HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(dst), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
  }
  return back;
}

// bytes of w that hold a NaN code (x.1111.111), as 0x80 in those bytes
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Raw tile -> fp16 operand tile: token row r, codes 16c .. 16c+15 become two
// 16-byte chunks of the row's 128-byte line(s), at the swizzled places. Rows
// without a token become zero. CLEAN: NaN codes become zero; returns whether
// there were any.
template <int D>
__device__ __forceinline__ bool convert_tile(uint32_t raw, uint32_t dst, bool whole, int rows,
                                             unsigned pm, int rshift, bool clean, int cw,
                                             int lane) {
  using Ly = ChunkLayout<D>;
  constexpr int UNITS = D / 16;                     // 16-code units per row
  constexpr int RPW = 32 / UNITS;                   // rows per warp and step
  constexpr int STEPS = kKv / (RPW * kConvWarps);
  const int c = lane % UNITS;
  bool seen = false;
#pragma unroll 4
  for (int s = 0; s < STEPS; ++s) {
    const int r = (s * kConvWarps + cw) * RPW + lane / UNITS;
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(raw + r * D + c * 16) : "memory");
    if (!whole && !(r < rows && ((pm >> (r >> rshift)) & 1u))) w[0] = w[1] = w[2] = w[3] = 0u;
    if (clean) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t nb = nan_bytes(w[k]);
        if (nb != 0u) {
          seen = true;
          w[k] &= ~((nb >> 7) * 0xffu);
        }
      }
    }
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) e4m3x4_to_f16x2x2(w[k], h[2 * k], h[2 * k + 1]);
    const uint32_t line = dst + (D == 128 ? (c >> 2) * Ly::HALF : 0) + r * 128;
    const int k0 = (2 * c) & 7;
    // the eight lanes of a store phase cover two half lines: the second half
    // stores its odd chunk first, so that they hit different banks
    const bool swap = D == 128 && c >= 4;
    const uint32_t d0 = line + ((k0 ^ (r & 7)) << 4), d1 = line + (((k0 + 1) ^ (r & 7)) << 4);
    const uint32_t da = swap ? d1 : d0, db = swap ? d0 : d1;
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(da), "r"(swap ? h[4] : h[0]), "r"(swap ? h[5] : h[1]),
                   "r"(swap ? h[6] : h[2]), "r"(swap ? h[7] : h[3]) : "memory");
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(db), "r"(swap ? h[0] : h[4]), "r"(swap ? h[1] : h[5]),
                   "r"(swap ? h[2] : h[6]), "r"(swap ? h[3] : h[7]) : "memory");
  }
  return seen;
}

// MMA issue (one thread).
template <int D>
__device__ void issue(int ntiles, uint32_t tiles, uint32_t bar, uint32_t tmem,
                      volatile int* abort_flag) {
  using Ly = ChunkLayout<D>;
  constexpr uint32_t idS = idesc_f16(false, kRows, kKv, false, false);
  constexpr uint32_t idO = idesc_f16(false, kRows, D, false, true);
  auto issue_s = [&](int t) -> bool {
    const int sb = t & 1;
    if (!mbar_wait_bounded(bar + 8u * (kKFull + sb), (t >> 1) & 1, abort_flag, kWaitCycles))
      return false;
    tc_fence_after();
    const uint32_t qa = tiles + Ly::Q_OFF, kb = tiles + Ly::K_OFF + sb * Ly::TILE;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint64_t ad = smem_desc_sw128(qa + (ks >> 2) * Ly::HALF + (ks & 3) * 32, 16, 1024);
      const uint64_t bd = smem_desc_sw128(kb + (ks >> 2) * Ly::HALF + (ks & 3) * 32, 16, 1024);
      mma_f16_ss(tmem + sb * kKv, ad, bd, idS, ks > 0 ? 1u : 0u);
    }
    mma_commit(bar + 8u * (kSFull + sb));
    mma_commit(bar + 8u * (kKEmpty + sb));
    return true;
  };
  auto issue_pv = [&](int t) -> bool {
    const int vs = t & 1;
    if (!mbar_wait_bounded(bar + 8u * kPFull, t & 1, abort_flag, kWaitCycles)) return false;
    if (!mbar_wait_bounded(bar + 8u * (kVFull + vs), (t >> 1) & 1, abort_flag, kWaitCycles))
      return false;
    tc_fence_after();
    const uint32_t vb = tiles + Ly::V_OFF + vs * Ly::TILE;
    const uint32_t pt = tmem + (uint32_t)(t & 1) * kKv;
#pragma unroll
    for (int ks = 0; ks < kKv / 16; ++ks) {
      const uint64_t bd = smem_desc_sw128(vb + ks * 2048, Ly::HALF, 1024);
      mma_f16_ts(tmem + kOCol, pt + (ks >> 2) * kCols + (ks & 3) * 8, bd, idO,
                 (t > 0 || ks > 0) ? 1u : 0u);
    }
    mma_commit(bar + 8u * kODone);
    mma_commit(bar + 8u * (kVEmpty + vs));
    return true;
  };
  bool ok = mbar_wait_bounded(bar + 8u * kQFull, 0, abort_flag, kWaitCycles);
  for (int t = 0; ok && t < 2 && t < ntiles; ++t) ok = issue_s(t);
  for (int j = 0; ok && j < ntiles; ++j) {
    ok = issue_pv(j);
    if (ok && j + 2 < ntiles) {
      ok = mbar_wait_bounded(bar + 8u * kODone, j & 1, abort_flag, kWaitCycles);
      if (ok) ok = issue_s(j + 2);
    }
  }
  mma_commit(bar + 8u * kDone);
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
  float* xch = reinterpret_cast<float*>(smem_raw + Ly::XCH_OFF);   // [2][2 halves][128]
  if (tiles + Ly::TILES > sbase + Ly::SMEM) {       // base too far off 1024 bytes
    if (threadIdx.x == 0) latch(a.err, PA_ERR_CUDA);
    return;
  }

  const int s = blockIdx.z, kvh = blockIdx.y;
  const int row_tiles = (int)(((int64_t)a.max_query_len * G + kRows - 1) / kRows);
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
  const int r0 = qt * kRows;
  if (r0 >= n * G) return;
  const TileSpan sp = tile_span(a, G, n, L, qt);
  const int kv_lo = sp.kv_base + split * a.partition;
  if (split >= sp.count) return;
  const int kv_end = min(sp.kv_all, kv_lo + a.partition);
  const int ntiles = (kv_end - kv_lo + kKv - 1) / kKv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(bar + 8u * (kRawFull + i), 1);
      mbar_init(bar + 8u * (kRawEmpty + i), kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + 8u * (kKFull + i), kConvWarps);
      mbar_init(bar + 8u * (kKEmpty + i), 1);
      mbar_init(bar + 8u * (kVFull + i), kConvWarps);
      mbar_init(bar + 8u * (kVEmpty + i), 1);
      mbar_init(bar + 8u * (kSFull + i), 1);
    }
    mbar_init(bar + 8u * kPFull, kSoftmaxWarps);
    mbar_init(bar + 8u * kODone, 1);
    mbar_init(bar + 8u * kDone, 1);
    mbar_init(bar + 8u * kQFull, kConvWarps);
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

  if (warp == kProducerWarp) {
    produce<D>(a, &tmK, &tmV, pc, kvh, tiles, bar, masks, abort_flag, lane);
  } else if (warp == kMmaWarp) {
    if (lane == 0) issue<D>(ntiles, tiles, bar, tmem, abort_flag);
    __syncwarp();
  } else if (warp >= kConvWarp) {
    const int cw = warp - kConvWarp;
    {
      const int r = cw * 32 + lane, rr = r0 + r;
      const int i = rr / G;
      const bool live = i < n;
      const T* src = reinterpret_cast<const T*>(a.q) +
                     ((int64_t)(q0 + (live ? i : 0)) * a.num_q_heads + (int64_t)kvh * G + rr % G) * D;
      // the factors sit where the second exchange buffer will be: it is
      // first written after every softmax thread has read its factor
      xch[2 * kRows + r] = convert_q_row<T, D>(src, live, a.scale, tiles + Ly::Q_OFF, r);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + 8u * kQFull);
    }
    for (int it = 0; it < 2 * ntiles; ++it) {
      int j;
      const bool isv = item_of(it, ntiles, &j);
      const int rs = it % kRaw, st = j & 1;
      bool ok = mbar_wait_bounded(bar + 8u * (kRawFull + rs), (it / kRaw) & 1, abort_flag,
                                  kWaitCycles);
      if (ok && j >= 2)
        ok = mbar_wait_bounded(bar + 8u * ((isv ? kVEmpty : kKEmpty) + st), ((j >> 1) - 1) & 1,
                               abort_flag, kWaitCycles);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int ts = kv_lo + j * kKv;
      const int rows = min(kKv, kv_end - ts);
      const unsigned pm = masks[rs];
      const bool clean = isv && (ts + kKv - 1 > pos_first || ts < lo_last);
      const bool seen = convert_tile<D>(
          tiles + Ly::RAW_OFF + rs * Ly::RAW,
          tiles + (isv ? Ly::V_OFF : Ly::K_OFF) + st * Ly::TILE, pm == full_mask && rows == kKv,
          rows, pm, rshift, clean, cw, lane);
      if (seen) misc[6] = 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar + 8u * (kRawEmpty + rs));
        mbar_arrive(bar + 8u * ((isv ? kVFull : kKFull) + st));
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + 8u * kConvDone);
  } else {
    // ---- softmax: thread = (half hf, row r)
    const int hf = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int rr = r0 + r;
    const int i = rr / G;
    const bool rv = i < n;
    const int pos = rv ? L - n + i : -1;
    const int lo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
    const bool idle = __all_sync(0xffffffffu, !rv);   // no row here holds a token
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    bool ok = mbar_wait_bounded(bar + 8u * kQFull, 0, abort_flag, kWaitCycles);
    // logit factor in the log2 domain (Q carries the scale's sign and zero)
    const float f0 = (a.scale == 0.f ? 1.f : fabsf(a.scale)) * kLog2e *
                     (SCALED ? 1.f : a.k_scale) * xch[2 * kRows + r];

    int ent = pc.entry(0, lane), ent_next = pc.entry(1, lane);
    float ksl = 1.f, vsl = 0.f;                       // scales of this lane's piece
    auto load_scales = [&](int e, float& k, float& v) {
      k = 1.f;
      v = 0.f;
      if (SCALED && e >= 0 && e < a.num_blocks) {
        k = a.k_scales[(int64_t)e * a.num_kv_heads + kvh];
        v = a.v_scales[(int64_t)e * a.num_kv_heads + kvh];
      }
    };
    load_scales(ent, ksl, vsl);
    float m_use = kNegInfC, l = 0.f, vref = 0.f;
    for (int j = 0; j < ntiles; ++j) {
      const int sb = j & 1;
      const int ts = kv_lo + j * kKv;
      const int te = min(kv_end, ts + kKv);
      const unsigned pm = __ballot_sync(0xffffffffu, ent >= 0 && ent < a.num_blocks);
      float ks_next, vs_next;
      load_scales(ent_next, ks_next, vs_next);
      const int ent_2 = pc.entry(j + 2, lane);
      if (ok)
        ok = mbar_wait_bounded(bar + 8u * (kSFull + sb), (j >> 1) & 1, abort_flag, kWaitCycles);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const bool whole = pm == full_mask && te - ts == kKv;
      const int hi = min(pos, te - 1) - ts - hf * kCols;     // last own column in sight
      const int first = lo - ts - hf * kCols;                // first own column in sight
      const bool fast = __all_sync(0xffffffffu, (whole && hi >= kCols - 1 && first <= 0) || !rv);
      const uint32_t sadr = tmem + lanes + sb * kKv + hf * kCols;
      uint32_t v[kCols];
      if (ok && !idle) {
        tmem_ld64(sadr, v);
      } else {
#pragma unroll
        for (int e = 0; e < kCols; ++e) v[e] = 0u;
      }
      if (!fast && rv) {
        // what a row does not see becomes -inf in place: weight 0 below
#pragma unroll
        for (int ch = 0; ch < kCols / 32; ++ch) {
          const int c0 = ch * 32;
          uint32_t m = hi < c0 ? 0u : hi >= c0 + 31 ? 0xffffffffu : (2u << (hi - c0)) - 1u;
          if (first > c0) m &= first > c0 + 31 ? 0u : 0xffffffffu << (first - c0);
          if (!whole) {
            const int g0 = hf * kCols + c0;
            uint32_t p = 0;
            if (pc.R >= 32) {
              p = ((pm >> (g0 >> rshift)) & 1u) ? 0xffffffffu : 0u;
            } else {
              for (int k = 0; k < 32 / pc.R; ++k)
                if ((pm >> ((g0 >> rshift) + k)) & 1u) p |= ((1u << pc.R) - 1u) << (k * pc.R);
            }
            m &= p;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((m >> e) & 1u)) v[c0 + e] = __float_as_uint(kNegInfC);
        }
      }
      // the tile's V reference: all warps see the same pieces
      float alpha_v = 1.f;
      float rcp_ref = 0.f;
      if (SCALED) {
        const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vsl)));
        if (top > vref) {
          if (vref > 0.f) alpha_v = vref / top;
          vref = top;
        }
        rcp_ref = vref > 0.f ? 1.f / vref : 0.f;
      }
      // pass 1: the half row's maximum
      float mx = kNegInfC;
      if (ok && !idle) {
        if (!SCALED) {
          float mx0 = kNegInfC, mx1 = kNegInfC;
#pragma unroll
          for (int e = 0; e < kCols; e += 4) {
            mx0 = cfmax3(mx0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            mx1 = cfmax3(mx1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
          }
          mx = fmaxf(mx0, mx1) * f0;
        } else {
#pragma unroll
          for (int g = 0; g < kCols / 8; ++g) {
            const float kf = __shfl_sync(0xffffffffu, ksl, (hf * kCols + 8 * g) >> rshift) * f0;
            float m0 = fmaxf(__uint_as_float(v[8 * g]), __uint_as_float(v[8 * g + 1]));
            float m1 = fmaxf(__uint_as_float(v[8 * g + 2]), __uint_as_float(v[8 * g + 3]));
            m0 = cfmax3(m0, __uint_as_float(v[8 * g + 4]), __uint_as_float(v[8 * g + 5]));
            m1 = cfmax3(m1, __uint_as_float(v[8 * g + 6]), __uint_as_float(v[8 * g + 7]));
            mx = fmaxf(mx, fmaxf(m0, m1) * kf);
          }
        }
      }
      // the two halves meet; the buffers alternate, so one barrier a tile
      xch[(sb * 2 + hf) * kRows + r] = mx;
      ok = softmax_all(ok);
      if (!ok) break;
      mx = fmaxf(mx, xch[(sb * 2 + (hf ^ 1)) * kRows + r]);
      const float m_new = fmaxf(m_use, mx);
      float alpha = 1.f;
      if (m_use == kNegInfC) {
        m_use = m_new;                               // nothing accumulated yet
      } else if (m_new > m_use + kLazyLog2) {
        alpha = exp2f(m_use - m_new);
        m_use = m_new;
      }
      // pass 2: P = 2^(x - m_use) in fp16 over this thread's own scores; a
      // row that has seen nothing has only -inf scores and weights of 0
      const float nm = m_use == kNegInfC ? 0.f : -m_use;
      uint64_t sum = pair(0.f, 0.f);
#pragma unroll
      for (int ch = 0; ch < kCols / 32; ++ch) {
        uint32_t pk[16];
        if (idle) {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
        } else {
          const uint64_t cm = pair(nm, nm);
          uint64_t fm = pair(f0, f0), rm = 0;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            if (SCALED && (e & 7) == 0) {
              const int src = (hf * kCols + ch * 32 + e) >> rshift;
              const float kf = __shfl_sync(0xffffffffu, ksl, src) * f0;
              const float rt = __shfl_sync(0xffffffffu, vsl, src) * rcp_ref;
              fm = pair(kf, kf);
              rm = pair(rt, rt);
            }
            float x0, x1;
            unpair(fma_pair(pair(__uint_as_float(v[ch * 32 + e]),
                                 __uint_as_float(v[ch * 32 + e + 1])), fm, cm), x0, x1);
            x0 = cex2(x0);
            x1 = cex2(x1);
            uint64_t p = pair(x0, x1);
            sum = add_pair(sum, p);
            if (SCALED) unpair(mul_pair(p, rm), x0, x1);
            pk[e >> 1] = pack_half(x0, x1);
          }
        }
        tmem_st16(sadr + ch * 16, pk);
      }
      float s0, s1;
      unpair(sum, s0, s1);
      l = l * alpha + (s0 + s1);
      const float alpha_o = SCALED ? alpha * alpha_v : alpha;
      if (__any_sync(0xffffffffu, alpha_o != 1.f)) {
        if (j >= 1) {
          ok = mbar_wait_bounded(bar + 8u * kODone, (j - 1) & 1, abort_flag, kWaitCycles);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          if (ok) {
#pragma unroll 1
            for (int ch = 0; ch < D / 64; ++ch) {
              const uint32_t oadr = tmem + lanes + kOCol + hf * (D / 2) + ch * 32;
              uint32_t o[32];
              tmem_ld32(oadr, o);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha_o);
              tmem_st32(oadr, o);
            }
          }
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + 8u * kPFull);
      ent = ent_next;
      ent_next = ent_2;
      ksl = ks_next;
      vsl = vs_next;
    }
    // the row's sum, over both halves
    const int xb = (ntiles & 1) * 2;
    xch[(xb + hf) * kRows + r] = l;
    ok = softmax_all(ok);
    l += xch[(xb + (hf ^ 1)) * kRows + r];
    if (ok) ok = mbar_wait_bounded(bar + 8u * kDone, 0, abort_flag, kWaitCycles);
    if (ok) ok = mbar_wait_bounded(bar + 8u * kConvDone, 0, abort_flag, kWaitCycles);
    tc_fence_after();
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      const int64_t t = q0 + i;
      const int head = kvh * G + rr % G;
      const bool direct = rv && sp.count == 1;
      const bool partial = rv && sp.count > 1;
      const float unit = SCALED ? vref : a.v_scale;
      const float mul = direct ? (l != 0.f ? unit / l : 0.f) : unit;
      const bool nans = misc[6] != 0;
      T* out = reinterpret_cast<T*>(a.out);
      const int64_t slot = (t * a.num_q_heads + head) * a.num_splits + split;
#pragma unroll 1
      for (int ch = 0; ch < D / 64; ++ch) {
        const int c0 = hf * (D / 2) + ch * 32;
        uint32_t o[32];
        tmem_ld32(tmem + lanes + kOCol + c0, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * mul);
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
          uint4* op = reinterpret_cast<uint4*>(out + (t * a.num_q_heads + head) * D + c0);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 w;
            w.x = pack_out<T>(__uint_as_float(o[8 * q + 0]), __uint_as_float(o[8 * q + 1]));
            w.y = pack_out<T>(__uint_as_float(o[8 * q + 2]), __uint_as_float(o[8 * q + 3]));
            w.z = pack_out<T>(__uint_as_float(o[8 * q + 4]), __uint_as_float(o[8 * q + 5]));
            w.w = pack_out<T>(__uint_as_float(o[8 * q + 6]), __uint_as_float(o[8 * q + 7]));
            op[q] = w;
          }
        } else if (partial) {
          uint4* acc = reinterpret_cast<uint4*>(a.ws_acc + slot * D + c0);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            acc[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      if (partial && hf == 0) {
        a.ws_ml[2 * slot] = m_use;
        a.ws_ml[2 * slot + 1] = l;
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
  const TileSpan sp = tile_span(a, G, n, L, (int)(((t - q0) * G + head % G) / kRows));
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
  const int64_t row_tiles = ((int64_t)a.max_query_len * G + kRows - 1) / kRows;
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

// Keys a row tile can span (chunk_plan below and the kernel's tile_span).
static int64_t span_of(int group, int max_query_len, int max_seq_len, int window) {
  const int64_t len = max_seq_len > 0 ? max_seq_len : 1;
  if (window <= 0) return len;
  const int64_t toks = std::min<int64_t>(max_query_len, (kRows + group - 1) / group);
  return std::min<int64_t>(len, (int64_t)window - 1 + toks + kKv - 1);
}

void chunk_plan(int num_seqs, int num_kv_heads, int group, int max_query_len, int max_seq_len,
                int window, int partition_size, int sm_count, int* splits, int* tokens) {
  const int64_t len = span_of(group, max_query_len, max_seq_len, window);
  auto round_up = [](int64_t x) { return (x + kKv - 1) / kKv * kKv; };
  int64_t P = round_up(len);
  if (partition_size > 0) {
    P = std::min(P, round_up(partition_size));
  } else {
    const int64_t row_tiles = ((int64_t)max_query_len * group + kRows - 1) / kRows;
    const int64_t ctas = std::max<int64_t>(1, row_tiles * num_kv_heads * num_seqs);
    if (ctas < 4 * (int64_t)sm_count) {
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
  *tokens = (int)P;
  *splits = (int)((len + P - 1) / P);
}

cudaError_t launch_chunk_fp8(const ChunkArgs& a, cudaStream_t st) {
  if (a.dtype == PA_BF16) return launch_chunk_d<__nv_bfloat16>(a, st);
  if (a.dtype == PA_F16) return launch_chunk_d<__half>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace pa
