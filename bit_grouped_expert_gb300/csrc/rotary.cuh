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
    if constexpr (FP16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(half_pair<FP16>(x[0], x[1]), half_pair<FP16>(x[2], x[3]), half_pair<FP16>(x[4], x[5]),
                    half_pair<FP16>(x[6], x[7]));
}

// Cosines and sines of an item's pairs, 8 j .. 8 j + 7, at the position set last.
struct RotaryPairs {
  float c[8], s[8];

  // p times the rate overflows by whole turns: what is left is the angle, whose
  // nearest quarter turn is taken off as a whole number.  The rest, within an eighth of a
  // turn, comes as two signed words, so that fp32 keeps 2^-23 of it however small it is (8,191 rows of
  // 16 heads of 256 26.3 us, as one word of 64 bits 27.6), and the series of sine and cosine to the
  // ninth and tenth power are off by 2^-29 there.
  template <typename F>
  __device__ __forceinline__ void at(int p, F rate, float factor) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t turn = (uint64_t)(int64_t)p * rate(i);
      const uint32_t low = (uint32_t)turn, high = (uint32_t)(turn >> 32) + (low >> 31);  // low as a signed word
      const uint32_t quarter = (high + 0x20000000u) >> 30;
      const float x = fmaf((float)(int32_t)(high - (quarter << 30)), 6.283185307f * 0x1p-32f,
                           (float)(int32_t)low * (6.283185307f * 0x1p-64f)), xx = x * x;
      const float v = fmaf(x * xx, fmaf(xx, fmaf(xx, fmaf(xx, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
      const float u =
          fmaf(xx, fmaf(xx, fmaf(xx, fmaf(xx, fmaf(xx, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
      const float f = quarter & 2 ? -factor : factor;  // half a turn on
      c[i] = (quarter & 1 ? -v : u) * f;               // a quarter turn on
      s[i] = (quarter & 1 ? u : v) * f;
    }
  }
  // the values of the item's two runs
  __device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], bool inter) const {
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

// What a thread knows of its item: the two runs of eight values (a, then b),
// whether they are turned, and how.
struct RotaryItem : RotaryPairs {
  int a, b;   // offsets in the head
  bool turns, inter;
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
  __device__ __forceinline__ void at(int p) {
    if (turns) RotaryPairs::at(p, [&](int i) { return rate[i]; }, factor);
  }
  // sixteen-bit values, turned and rounded once; those that are not turned keep their bits
  template <bool FP16>
  __device__ __forceinline__ void turn_halves(uint4 &p, uint4 &q) const {
    if (!turns) return;
    float x[8], y[8];
    unpack8<FP16>(p, x);
    unpack8<FP16>(q, y);
    turn(x, y, inter);
    p = pack8<FP16>(x);
    q = pack8<FP16>(y);
  }
};

// Host: a table that attn_rotary_plan could have made, for heads of head_dim values.
moe_status rotary_check(const attn_rotary_table *t, int head_dim);

}  // namespace moe
