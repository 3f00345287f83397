// Rotary positions of q and k, with one or several position axes (time,
// height, width of image and video tokens), fused with the KV write.
//
// Pair i of a head's first rot_size dims is turned by
//     angle = positions[axis_of_pair[i]][t] * inv_freq[i],
//     (a, b) -> (a cos - b sin, b cos + a sin),
// in fp32, with (a, b) = (x[i], x[i + rot/2]) or, interleaved,
// (x[2i], x[2i + 1]); the other dims pass. q goes to q_out, k and v to the
// pool slots of the token ("PagedAttention 核心创新深度分析" §2.3), rounded
// once, from fp32 to the stored type.
//
// Angles: a far position times a frequency needs more than fp32, and FP64
// products and range reductions per angle would load the few FP64 units. A
// frequency becomes a 64-bit fixed-point fraction of a turn; position x fraction in
// wrapping 64-bit integers then IS the reduction to one turn, and the top 32
// bits go to sincospif as half turns in [-1, 1).
//
// The kernel moves bytes: per token it reads q, k, v and writes q and the
// two cache rows once. A CTA takes a few tokens, puts their cosines and
// sines into shared memory (each angle computed once, used by every head)
// and then runs over (token, head) rows; a thread keeps its place in the
// row, so its cosines change only with the token.
//
// Replayed from a graph, 64 query and 8 KV heads of 128, bf16, three axes:
// 32,500 tokens into 16-bit pools 215 us (1.33 GB: 6.2 TB/s, 0.91 of the
// measured copy rate); 4,400 tokens into blocks with scales 47.6 us (171 MB,
// 25 us at the copy rate; everything waits for the scales' pass, which reads k
// and v once more); 64 tokens of 32 + 2 x 32 heads, fp16, 3.9 us (3.1 MB: the
// launch). The angle work is what kept it from the
// copy rate: with FP64 frequencies and range reduction the blocks' case took
// 105 us. A persistent grid measured 318 us for the first case, and a table
// of turns in shared memory 240: short CTAs hide one another's start better.
#include <cuda_fp8.h>

#include <algorithm>

#include "block_scale.cuh"
#include "common.cuh"
#include "launchers.h"

namespace pa {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotMaxHalf = 128;     // head_size <= 256

// x as a fraction of a turn, x / (2 pi) mod 1, in 64-bit fixed point: the
// 53-bit mantissa times the first 128 bits of 1 / (2 pi), shifted by the
// exponent. Off by less than 2^-64 of a turn for |x| < 2^62; 0 for zeros,
// subnormals, infinities and NaN. In integers, because the SM has few FP64
// units: a warp's FP64 instruction occupies them for 16 clocks.
__device__ __forceinline__ uint64_t turn_fraction(double x) {
  const uint64_t c_hi = 0x28be60db9391054aull, c_lo = 0x7f09d5f47d4d3770ull;
  const uint64_t bits = (uint64_t)__double_as_longlong(x);
  const int e = (int)(bits >> 52) & 0x7ff;
  const uint64_t m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  // 192-bit product m * (c_hi 2^64 + c_lo), limbs p0 (low) to p2
  const uint64_t p0 = m * c_lo, mid = __umul64hi(m, c_lo), q = m * c_hi;
  const uint64_t p1 = mid + q;
  const uint64_t p2 = __umul64hi(m, c_hi) + (p1 < q ? 1u : 0u);
  // the 64 bits from bit s on
  const int s = 1139 - e;
  if (e == 0 || e == 0x7ff || s < 0 || s >= 192) return 0;
  const uint64_t a = s < 64 ? p0 : s < 128 ? p1 : p2;
  const uint64_t b = s < 64 ? p1 : s < 128 ? p2 : 0;
  const int k = s & 63;
  const uint64_t r = k == 0 ? a : (a >> k) | (b << (64 - k));
  return (bits >> 63) != 0 ? 0 - r : r;
}

__device__ __forceinline__ float2 cos_sin(int64_t pos, uint64_t turn) {
  const uint64_t phase = (uint64_t)pos * turn;      // wraps by whole turns
  const float half_turns = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;   // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ void rotate(float a, float b, float2 cs, float& x, float& y) {
  x = fmaf(a, cs.x, -b * cs.y);
  y = fmaf(b, cs.x, a * cs.y);
}

// N fp32 values to 16 bytes of T, round to nearest
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f) {
  uint4 u;
  T* p = reinterpret_cast<T*>(&u);
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) p[i] = Vec<T>::cvt_out(f[i]);
  return u;
}

// N fp32 values divided by the scale (IEEE fp32) to N E4M3 codes, nearest
// even, saturating. POW2: the scale is a power of two, whose reciprocal is
// exact, so a product gives the quotient.
template <int N, bool POW2>
__device__ __forceinline__ void store_fp8(uint8_t* dst, const float* f, float scale) {
  const float rcp = POW2 ? 1.f / scale : 0.f;
  auto over = [&](float x) { return POW2 ? x * rcp : __fdiv_rn(x, scale); };
  uint32_t w[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    uint32_t a = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_fp8x2_storage_t p = __nv_cvt_float2_to_fp8x2(
          make_float2(over(f[4 * j + 2 * h]), over(f[4 * j + 2 * h + 1])), __NV_SATFINITE,
          __NV_E4M3);
      a |= (uint32_t)p << (16 * h);
    }
    w[j] = a;
  }
  if constexpr (N == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

// Units: a head's D elements are D / (2N) units of two 16-byte vectors; unit
// c < rot / (2N) holds N pairs, the vectors at c*N and rot/2 + c*N (halves)
// or the neighbours at 2c*N and 2c*N + N (interleaved), later units the
// neighbours at 2c*N (dims that pass).
// POOL: 0 pools of T, 1 E4M3 with one scale, 2 E4M3 with per-block scales.
template <typename T, int POOL, bool INTER, int TOK>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ float2 cs[TOK][kRotMaxHalf];
  __shared__ int64_t slot_of[TOK];
  griddep_launch();
  const int half = a.rot_size / 2;
  const int D = a.head_size;
  const int units = D / (2 * N);
  const int rot_units = a.rot_size / (2 * N);
  const int rows_at_once = kRotThreads / units;
  const int c = threadIdx.x % units;
  const int lane_row = threadIdx.x / units;
  const bool active = lane_row < rows_at_once;
  const bool rot = c < rot_units;
  const int e0 = rot && !INTER ? c * N : 2 * c * N;           // first vector's element
  const int e1 = rot && !INTER ? half + c * N : e0 + N;       // second vector's
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int64_t limit = a.num_blocks * a.block_size;
  griddep_wait();
  for (int64_t t0 = (int64_t)blockIdx.x * TOK; t0 < a.num_tokens;
       t0 += (int64_t)gridDim.x * TOK) {
    const int nt = (int)min((int64_t)TOK, a.num_tokens - t0);
    __syncthreads();                                          // cs of the last round is used up
    for (int i = threadIdx.x; i < nt * half; i += kRotThreads) {
      const int tk = i / half, p = i - tk * half;
      int ax = a.axis_of_pair != nullptr ? a.axis_of_pair[p] : 0;
      if (ax < 0 || ax >= a.num_axes) {
        latch(a.err, PA_ERR_OUT_OF_RANGE);
        ax = 0;
      }
      cs[tk][p] = cos_sin(a.positions[ax * a.position_stride + t0 + tk],
                          turn_fraction(a.inv_freq[p]));
    }
    if (threadIdx.x < nt) {
      const int64_t s = a.slots[t0 + threadIdx.x];
      if (s >= limit) latch(a.err, PA_ERR_OUT_OF_RANGE);
      slot_of[threadIdx.x] = s < limit ? s : -1;
    }
    __syncthreads();
    if (!active) continue;
    int tk = 0, h = lane_row;
    while (true) {
      while (h >= heads) { h -= heads; ++tk; }
      if (tk >= nt) break;
      const int64_t t = t0 + tk;
      const int64_t slot = slot_of[tk];
      const int kind = h < a.num_q_heads ? 0 : h < a.num_q_heads + a.num_kv_heads ? 1 : 2;
      const int kvh = h - a.num_q_heads - (kind == 2 ? a.num_kv_heads : 0);
      if (kind == 0 || slot >= 0) {
        const T* src = kind == 0 ? (const T*)a.q + t * a.q_stride + (int64_t)h * D
                     : kind == 1 ? (const T*)a.k + t * a.k_stride + (int64_t)kvh * D
                                 : (const T*)a.v + t * a.v_stride + (int64_t)kvh * D;
        const uint4 u0 = *reinterpret_cast<const uint4*>(src + e0);
        const uint4 u1 = *reinterpret_cast<const uint4*>(src + e1);
        float x[2 * N];
        Vec<T>::to_f32(u0, x);
        Vec<T>::to_f32(u1, x + N);
        if (rot && kind != 2) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float2 w = cs[tk][c * N + i];
            if (INTER) rotate(x[2 * i], x[2 * i + 1], w, x[2 * i], x[2 * i + 1]);
            else rotate(x[i], x[N + i], w, x[i], x[N + i]);
          }
        }
        if (kind == 0) {
          T* dst = (T*)a.q_out + t * a.q_out_stride + (int64_t)h * D;
          *reinterpret_cast<uint4*>(dst + e0) = pack16<T>(x);
          *reinterpret_cast<uint4*>(dst + e1) = pack16<T>(x + N);
        } else {
          const int64_t blk = slot / a.block_size;
          const int64_t dst =
              ((blk * a.num_kv_heads + kvh) * a.block_size + (slot - blk * a.block_size)) * D;
          if (POOL != 0) {
            const float sc =
                POOL == 2 ? (kind == 1 ? a.k_scales : a.v_scales)[blk * a.num_kv_heads + kvh]
                          : (kind == 1 ? a.k_scale : a.v_scale);
            uint8_t* cache = (uint8_t*)(kind == 1 ? a.kc : a.vc) + dst;
            store_fp8<N, POOL == 2>(cache + e0, x, sc);
            store_fp8<N, POOL == 2>(cache + e1, x + N, sc);
          } else {
            T* cache = (T*)(kind == 1 ? a.kc : a.vc) + dst;
            *reinterpret_cast<uint4*>(cache + e0) = pack16<T>(x);
            *reinterpret_cast<uint4*>(cache + e1) = pack16<T>(x + N);
          }
        }
      }
      h += rows_at_once;
    }
  }
}

// First pass of the write into pools with per-block scales, as
// fix_block_scales_kernel of the plain write: for each token whose slot is
// row 0 of its block, the largest magnitude over the run of tokens that this
// call puts into the block, of the ROTATED keys and of the values, fixes the
// block's scales. A CTA looks at kScaleTokens tokens and takes the runs that
// begin there (one, with blocks of 16) one after the other: the run's cosines
// and sines go to shared memory, kRunTokens tokens at a time, and each warp
// takes KV heads, in the units of rotary_kernel (the same arithmetic, so the
// maximum is of exactly the values that the second pass quantises).
constexpr int kScaleTokens = 16;
constexpr int kRunTokens = 16;
constexpr int kHeadsPerWarp = 8;

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRotThreads) rotary_scales_kernel(const RotaryArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr int WARPS = kRotThreads / 32;
  __shared__ float2 cs[kRunTokens][kRotMaxHalf];
  __shared__ uint64_t turn[kRotMaxHalf];
  __shared__ int axis[kRotMaxHalf];
  __shared__ int64_t first_slot[kScaleTokens];
  __shared__ int run_len;
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = a.rot_size / 2, D = a.head_size, B = a.block_size;
  const int units = D / (2 * N), rot_units = a.rot_size / (2 * N);
  const int rows_at_once = 32 / units;
  const int c = lane % units, lane_row = lane / units;
  const bool rot = c < rot_units;
  const int e0 = rot && !INTER ? c * N : 2 * c * N;
  const int e1 = rot && !INTER ? half + c * N : e0 + N;
  const int64_t limit = a.num_blocks * B;
  const int64_t base = (int64_t)blockIdx.x * kScaleTokens;
  for (int p = threadIdx.x; p < half; p += kRotThreads) {
    turn[p] = turn_fraction(a.inv_freq[p]);
    const int ax = a.axis_of_pair != nullptr ? a.axis_of_pair[p] : 0;
    axis[p] = ax < 0 || ax >= a.num_axes ? 0 : ax;    // reported by the second pass
  }
  if (threadIdx.x < kScaleTokens) {
    const int64_t s = base + threadIdx.x < a.num_tokens ? a.slots[base + threadIdx.x] : -1;
    // only slots that begin a block; those past the pool are reported by the
    // second pass
    first_slot[threadIdx.x] = s >= 0 && s < limit && s % B == 0 ? s : -1;
  }
  __syncthreads();
  for (int i = 0; i < kScaleTokens; ++i) {
    const int64_t s0 = first_slot[i], t = base + i;
    if (s0 < 0) continue;                             // the same for every thread
    if (threadIdx.x == 0) run_len = B;
    __syncthreads();
    const int most = (int)min((int64_t)B, a.num_tokens - t);
    for (int k = threadIdx.x; k < B; k += kRotThreads)
      if (k >= most || a.slots[t + k] != s0 + k) atomicMin(&run_len, k);
    __syncthreads();
    const int n = run_len;
    const int64_t blk = s0 / B;
    for (int h0 = 0; h0 < a.num_kv_heads; h0 += WARPS * kHeadsPerWarp) {
      float ka[kHeadsPerWarp] = {}, va[kHeadsPerWarp] = {};
      for (int r0 = 0; r0 < n; r0 += kRunTokens) {
        const int nt = min(kRunTokens, n - r0);
        __syncthreads();                              // cs of the last round is used up
        for (int x = threadIdx.x; x < nt * half; x += kRotThreads) {
          const int tk = x / half, p = x - tk * half;
          cs[tk][p] = cos_sin(a.positions[axis[p] * a.position_stride + t + r0 + tk], turn[p]);
        }
        __syncthreads();
        if (lane_row >= rows_at_once) continue;       // joins the barriers above again
#pragma unroll
        for (int q = 0; q < kHeadsPerWarp; ++q) {
          const int h = h0 + q * WARPS + warp;
          if (h >= a.num_kv_heads) break;
#pragma unroll 4
          for (int tk = lane_row; tk < nt; tk += rows_at_once) {
            const T* k = (const T*)a.k + (t + r0 + tk) * a.k_stride + (int64_t)h * D;
            const T* v = (const T*)a.v + (t + r0 + tk) * a.v_stride + (int64_t)h * D;
            float x[2 * N], y[2 * N];
            Vec<T>::to_f32(*reinterpret_cast<const uint4*>(k + e0), x);
            Vec<T>::to_f32(*reinterpret_cast<const uint4*>(k + e1), x + N);
            Vec<T>::to_f32(*reinterpret_cast<const uint4*>(v + e0), y);
            Vec<T>::to_f32(*reinterpret_cast<const uint4*>(v + e1), y + N);
            if (rot) {
#pragma unroll
              for (int e = 0; e < N; ++e) {
                const float2 w = cs[tk][c * N + e];
                if (INTER) rotate(x[2 * e], x[2 * e + 1], w, x[2 * e], x[2 * e + 1]);
                else rotate(x[e], x[N + e], w, x[e], x[N + e]);
              }
            }
            // fmaxf leaves a NaN out
#pragma unroll
            for (int e = 0; e < 2 * N; ++e) {
              ka[q] = fmaxf(ka[q], fabsf(x[e]));
              va[q] = fmaxf(va[q], fabsf(y[e]));
            }
          }
        }
      }
#pragma unroll
      for (int q = 0; q < kHeadsPerWarp; ++q) {
        const int h = h0 + q * WARPS + warp;
        if (h >= a.num_kv_heads) break;               // the same for the whole warp
        float km = ka[q], vm = va[q];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
          km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
          vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
        }
        if (lane == 0) {
          a.k_scales[blk * a.num_kv_heads + h] = block_scale_of(km);
          a.v_scales[blk * a.num_kv_heads + h] = block_scale_of(vm);
        }
      }
    }
  }
}

template <typename T, int POOL, bool INTER>
cudaError_t launch_rotary_t(const RotaryArgs& a, int sm_count, cudaStream_t st) {
  if (POOL == 2) {
    const int64_t blocks = (a.num_tokens + kScaleTokens - 1) / kScaleTokens;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const cudaError_t e = launch_pdl(rotary_scales_kernel<T, INTER>, dim3((unsigned)blocks),
                                     dim3(kRotThreads), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  // few tokens: one per CTA, so that they spread over the SMs; more: two or
  // four per CTA, which share a round's barriers, as long as that leaves
  // several waves of CTAs (some five are resident per SM). With 1, 2 and 4
  // tokens per CTA (64 + 2 x 8 heads of 128, bf16): 608 tokens 7.0, 9.3, 8.2
  // us; 1,216 tokens 11.8, 10.9, 16.0; 2,432 tokens 23.2, 20.3, 20.2; 4,864
  // tokens 44.6, 40.4, 38.4; 36,000 tokens 289, 249, 237.
  auto go = [&](auto kernel, int tok) {
    const int64_t blocks = std::min<int64_t>((a.num_tokens + tok - 1) / tok, 0x7fffffffll);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kRotThreads), 0, st, a);
  };
  if (a.num_tokens <= (int64_t)sm_count * 5) return go(rotary_kernel<T, POOL, INTER, 1>, 1);
  if (a.num_tokens <= (int64_t)sm_count * 30) return go(rotary_kernel<T, POOL, INTER, 2>, 2);
  return go(rotary_kernel<T, POOL, INTER, 4>, 4);
}

template <typename T, int POOL>
cudaError_t launch_rotary_i(const RotaryArgs& a, int sm_count, cudaStream_t st) {
  return a.interleaved ? launch_rotary_t<T, POOL, true>(a, sm_count, st)
                       : launch_rotary_t<T, POOL, false>(a, sm_count, st);
}

template <typename T>
cudaError_t launch_rotary_d(const RotaryArgs& a, int sm_count, cudaStream_t st) {
  if (a.pool == 0) return launch_rotary_i<T, 0>(a, sm_count, st);
  return a.k_scales == nullptr ? launch_rotary_i<T, 1>(a, sm_count, st)
                               : launch_rotary_i<T, 2>(a, sm_count, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int sm_count, cudaStream_t st) {
  switch (a.dtype) {
    case PA_F32: return launch_rotary_d<float>(a, sm_count, st);
    case PA_F16: return launch_rotary_d<__half>(a, sm_count, st);
    case PA_BF16: return launch_rotary_d<__nv_bfloat16>(a, sm_count, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
