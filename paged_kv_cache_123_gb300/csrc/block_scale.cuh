// Scale of an fp8 block from its first tokens, shared by the KV writes.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// Power-of-two scale of a block whose first tokens' largest magnitude is
// amax: 2^k with k = ceil(log2(amax)) - 7 kept in [-126, 127], so amax lands
// in (64, 128]; 1 for amax = 0, 2^127 for an infinite amax. Integer work on
// the fp32 encoding: the biased exponent gives floor(log2), and a nonzero
// mantissa moves it up by one.
__device__ __forceinline__ float block_scale_of(float amax) {
  if (amax == 0.f) return 1.f;
  const uint32_t b = __float_as_uint(amax);
  const int ef = (int)(b >> 23);
  int k;
  if (ef == 0) {
    k = -126;                                   // below 2^-126: clamped
  } else if (ef == 255) {
    k = 127;
  } else {
    const int c = (ef - 127) + ((b & 0x7fffffu) != 0u);
    k = min(max(c - 7, -126), 127);
  }
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

}  // namespace pa
