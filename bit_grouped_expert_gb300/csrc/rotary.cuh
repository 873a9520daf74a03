// Rotary positions on the device (rotary.h): a thread turns sixteen values of
// a head at a time, item j of its head_dim / 16.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "rotary.h"

namespace moe {

template <bool FP16>
__device__ __forceinline__ float half_value(uint32_t bits) {  // of the low 16 bits
  if constexpr (FP16)
    return __half2float(__ushort_as_half((uint16_t)bits));
  else
    return __uint_as_float(bits << 16);
}
template <bool FP16>
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  if constexpr (FP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}
template <bool FP16>
__device__ __forceinline__ void unpack8(uint4 a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = half_value<FP16>(w[i] & 0xFFFFu);
    x[2 * i + 1] = half_value<FP16>(w[i] >> 16);
  }
}
template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(half_pair<FP16>(x[0], x[1]), half_pair<FP16>(x[2], x[3]), half_pair<FP16>(x[4], x[5]),
                    half_pair<FP16>(x[6], x[7]));
}

// What a thread knows of its item: the two runs of eight values (a, then b),
// whether they are turned, and how.
struct RotaryItem {
  int a, b;   // offsets in the head
  bool turns, inter;
  float c[8], s[8];  // cos and sin of pairs 8j .. 8j + 7 at the position set last
  uint64_t rate[8];
  float factor;

  __device__ __forceinline__ RotaryItem(const attn_rotary_table *t, int j) {
    turns = t && j < t->dim / 16;
    inter = !turns || t->interleaved;
    a = inter ? 16 * j : 8 * j;
    b = inter ? 16 * j + 8 : t->dim / 2 + 8 * j;
    factor = turns ? t->factor : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) rate[i] = turns ? t->turns[8 * j + i] : 0;
  }
  // p times the rate overflows by whole turns: what is left, read as signed, is
  // the angle within half a turn to either side.
  __device__ __forceinline__ void at(int p) {
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t turn = (uint64_t)(int64_t)p * rate[i];
      sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s[i], &c[i]);
      c[i] *= factor;
      s[i] *= factor;
    }
  }
  // the values of runs a and b, turned where they are
  __device__ __forceinline__ void turn(float (&x)[8], float (&y)[8]) const {
    if (!turns) return;
    if (inter) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float u = x[i], v = y[i];
        x[i] = u * c[i / 2] - x[i + 1] * s[i / 2];
        x[i + 1] = u * s[i / 2] + x[i + 1] * c[i / 2];
        y[i] = v * c[4 + i / 2] - y[i + 1] * s[4 + i / 2];
        y[i + 1] = v * s[4 + i / 2] + y[i + 1] * c[4 + i / 2];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = x[i];
        x[i] = u * c[i] - y[i] * s[i];
        y[i] = u * s[i] + y[i] * c[i];
      }
    }
  }
};

// Host: a table that attn_rotary_plan could have made, for heads of head_dim values.
moe_status rotary_check(const attn_rotary_table *t, int head_dim);

}  // namespace moe
