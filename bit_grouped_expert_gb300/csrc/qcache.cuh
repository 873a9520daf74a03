// Device view of the 8-bit paged KV cache (qcache.h) and its numbers.
#pragma once
#include <cuda_fp16.h>

#include "cache.cuh"
#include "qcache.h"

namespace moe {

struct QCacheView {
  CacheView c;  // k, v: the codes, two to a 16-bit word
  float *ks, *vs;
  int heads, dim;
};

// Two values' e4m3 codes (nearest, ties to even; beyond 448 the largest; NaN stays), the first in the low byte.
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
  uint16_t codes;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(codes) : "f"(hi), "f"(lo));
  return codes;
}
// Two codes' values (exact in fp16).
__device__ __forceinline__ float2 from_codes(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

constexpr int Q_MIN_EXP = -100;  // of a scale

// The least e >= Q_MIN_EXP with most <= 448 * 2^e (448 = 1.75 * 2^8), for a
// finite most >= 0: by its exponent and whether its fraction is above 1.75.
__device__ __forceinline__ int scale_exp(float most) {
  const uint32_t bits = __float_as_uint(most);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, Q_MIN_EXP);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // e: -126 .. 127

// Host: the view of a cache, after its dimensions and pointers are checked.
moe_status qcache_view(const attn_qcache *c, QCacheView *out);

}  // namespace moe
