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
// products and range reductions per angle would load the few FP64 units. The
// frequency becomes a 64-bit fixed-point fraction of a turn once per thread
// (two FP64 products, exact to 2^-64 of a turn); position x fraction in
// wrapping 64-bit integers then IS the reduction to one turn, and the top 32
// bits go to sincospif as half turns in [-1, 1).
//
// The kernel moves bytes: per token it reads q, k, v and writes q and the
// two cache rows once. A CTA takes a few tokens, puts their cosines and
// sines into shared memory (each angle computed once, used by every head)
// and then runs over (token, head) rows; a thread keeps its place in the
// row, so its cosines change only with the token.
#include <cuda_fp8.h>

#include "block_scale.cuh"
#include "common.cuh"
#include "launchers.h"

namespace pa {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotMaxHalf = 128;     // head_size <= 256

// inv_freq as a fraction of a turn, 64-bit fixed point: x / (2 pi) with the
// reciprocal split in two doubles, its whole turns dropped.
__device__ __forceinline__ uint64_t turn_fraction(double x) {
  const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;   // 1 / (2 pi)
  const double p = x * hi;
  const double e = fma(x, hi, -p) + x * lo;
  const double f = p - floor(p);                    // exact
  const uint64_t whole = __double2ull_rz(f * 18446744073709551616.0);
  return whole + (uint64_t)__double2ll_rn(e * 18446744073709551616.0);
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
// even, saturating
template <int N>
__device__ __forceinline__ void store_fp8(uint8_t* dst, const float* f, float scale) {
  uint32_t w[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    uint32_t a = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_fp8x2_storage_t p = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(f[4 * j + 2 * h], scale), __fdiv_rn(f[4 * j + 2 * h + 1], scale)),
          __NV_SATFINITE, __NV_E4M3);
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
template <typename T, bool FP8, bool INTER, int TOK>
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
          if (FP8) {
            float sc = kind == 1 ? a.k_scale : a.v_scale;
            if (a.k_scales != nullptr)
              sc = (kind == 1 ? a.k_scales : a.v_scales)[blk * a.num_kv_heads + kvh];
            uint8_t* cache = (uint8_t*)(kind == 1 ? a.kc : a.vc) + dst;
            store_fp8<N>(cache + e0, x, sc);
            store_fp8<N>(cache + e1, x + N, sc);
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
// fix_block_scales_kernel of the plain write: one warp per (token, KV head)
// whose slot is row 0 of its block takes the largest magnitude over the run
// of tokens that this call puts into the block, of the ROTATED keys and of
// the values, and fixes the block's scales. A lane owns pairs lane, lane +
// 32, ..., so it needs their frequencies only once.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRotThreads) rotary_scales_kernel(const RotaryArgs a) {
  constexpr int kMaxPairs = kRotMaxHalf / 32;
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int half = a.rot_size / 2, D = a.head_size;
  const int64_t warps = (int64_t)gridDim.x * (kRotThreads / 32);
  const int64_t limit = a.num_blocks * a.block_size;
  uint64_t turn[kMaxPairs];
  int axis[kMaxPairs];
#pragma unroll
  for (int j = 0; j < kMaxPairs; ++j) {
    const int p = lane + 32 * j;
    turn[j] = p < half ? turn_fraction(a.inv_freq[p]) : 0;
    axis[j] = p < half && a.axis_of_pair != nullptr ? a.axis_of_pair[p] : 0;
    if (axis[j] < 0 || axis[j] >= a.num_axes) axis[j] = 0;    // reported by the second pass
  }
  for (int64_t w = (int64_t)blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5);
       w < a.num_tokens * a.num_kv_heads; w += warps) {
    const int64_t t = w / a.num_kv_heads;
    const int h = (int)(w - t * a.num_kv_heads);
    const int64_t s0 = a.slots[t];
    if (s0 < 0 || s0 >= limit || s0 % a.block_size != 0) continue;
    int n = 1;
    while (n < a.block_size && t + n < a.num_tokens && a.slots[t + n] == s0 + n) ++n;
    float ka = 0.f, va = 0.f;
    for (int r = 0; r < n; ++r) {
      const T* k = (const T*)a.k + (t + r) * a.k_stride + (int64_t)h * D;
      const T* v = (const T*)a.v + (t + r) * a.v_stride + (int64_t)h * D;
#pragma unroll
      for (int j = 0; j < kMaxPairs; ++j) {
        const int p = lane + 32 * j;
        if (p >= half) break;
        float x, y;
        rotate(static_cast<float>(k[INTER ? 2 * p : p]),
               static_cast<float>(k[INTER ? 2 * p + 1 : p + half]),
               cos_sin(a.positions[axis[j] * a.position_stride + t + r], turn[j]), x, y);
        ka = fmaxf(ka, fmaxf(fabsf(x), fabsf(y)));
      }
      for (int e = a.rot_size + lane; e < D; e += 32) ka = fmaxf(ka, fabsf(static_cast<float>(k[e])));
      for (int e = lane; e < D; e += 32) va = fmaxf(va, fabsf(static_cast<float>(v[e])));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
      va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
    }
    if (lane == 0) {
      const int64_t idx = (s0 / a.block_size) * a.num_kv_heads + h;
      a.k_scales[idx] = block_scale_of(ka);
      a.v_scales[idx] = block_scale_of(va);
    }
  }
}

template <typename T, bool FP8, bool INTER>
cudaError_t launch_rotary_t(const RotaryArgs& a, int sm_count, cudaStream_t st) {
  if (FP8 && a.k_scales != nullptr) {
    const int64_t warps = a.num_tokens * a.num_kv_heads;
    int64_t blocks = (warps + kRotThreads / 32 - 1) / (kRotThreads / 32);
    if (blocks > (int64_t)sm_count * 16) blocks = (int64_t)sm_count * 16;
    const cudaError_t e = launch_pdl(rotary_scales_kernel<T, INTER>, dim3((unsigned)blocks),
                                     dim3(kRotThreads), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  // few tokens: one per CTA, so that they spread over the SMs; many: four
  // per CTA, which share a round's barriers
  if (a.num_tokens <= (int64_t)sm_count * 8)
    return launch_pdl(rotary_kernel<T, FP8, INTER, 1>, dim3((unsigned)a.num_tokens),
                      dim3(kRotThreads), 0, st, a);
  int64_t blocks = (a.num_tokens + 3) / 4;
  if (blocks > 0x7fffffffll) blocks = 0x7fffffffll;
  return launch_pdl(rotary_kernel<T, FP8, INTER, 4>, dim3((unsigned)blocks), dim3(kRotThreads), 0,
                    st, a);
}

template <typename T>
cudaError_t launch_rotary_d(const RotaryArgs& a, int sm_count, cudaStream_t st) {
  if (a.pool == 1)
    return a.interleaved ? launch_rotary_t<T, true, true>(a, sm_count, st)
                         : launch_rotary_t<T, true, false>(a, sm_count, st);
  return a.interleaved ? launch_rotary_t<T, false, true>(a, sm_count, st)
                       : launch_rotary_t<T, false, false>(a, sm_count, st);
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
