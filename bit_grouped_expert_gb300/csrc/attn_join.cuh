// Joining the parts of attention units that several CTAs share (tree.cu, qattend.cu).
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

constexpr int JOIN_MAX_CTAS = 320;  // of the kernel before: two for each of 160 SMs at most

// A CTA's split unit that starts with it, for the joining kernel.
struct SplitDesc {
  int32_t parts;   // CTAs it spans (0: none)
  int32_t stride;  // from one of them to the next
  int32_t rows, node0, head0, pad[3];
};

struct JoinArgs {
  SplitDesc *desc;  // [grid]
  float *ml;        // [2 * grid][rows_cap][2]
  float *part;      // [2 * grid][D / 4][rows_cap][4], or with row_major [2 * grid][rows_cap][D]
  uint16_t *o;      // [rows][Hq][D]
  int rows_cap;     // rows of a unit at most
  int row_major;
  int most_groups;  // threads that share a unit's values at most: 8 or 32
  int Hq, G;        // query heads, and of a KV head
};

namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (FP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}
// o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the parts of a split
// unit.  A thread has sixteen values of one row (rows run fastest, in the
// parts as in the threads, so that a warp reads whole lines); up to `most_groups`
// groups of a block's threads share the parts of the same values (a unit is
// split over as few as two CTAs and as many as all of them).
constexpr int JOIN_THREADS = 256;

// (One group always, this rule, eight always, whole calls in us: 1 node over 3,000
// positions 17.4, 14.8, 14.4; 4 x 5 over 9,000 29.8, 25.0, 24.3; 24 x 5 over 6,000
// 63.9, 62.2, 65.9; 48 x 16 over 1,800, fp16, 78.0, 75.9, 93.5.  More than 32 parts, over the 8-bit cache,
// whose units are fewer rows: one row over 131,000 positions in 32 groups 38.4 us, in eight 43.0; five 53.7 and 55.2.)
// The groups' log2.
__device__ __forceinline__ int part_groups(int parts, int most) {
  return parts <= 2 ? 0 : parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 32 || most == 8 ? 3 : 5;
}

template <int D, bool FP16>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ JoinArgs a, int ctas) {
  constexpr int MAXU = JOIN_MAX_CTAS, WARPS = JOIN_THREADS / 32;  // MAXU: split units at most
  __shared__ SplitDesc desc_s[MAXU];
  __shared__ int cta_s[MAXU], item_s[MAXU + 1], wsum[WARPS];
  __shared__ float4 acc_s[4][JOIN_THREADS];
  __shared__ float2 ml_s[JOIN_THREADS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the split units in the CTAs' order, and the items (blocks of cells of sixteen values) before each
  const int cells = D / 16 * a.rows_cap;
  constexpr int PER = (MAXU + JOIN_THREADS - 1) / JOIN_THREADS;
  SplitDesc d[PER];
  auto items_of = [&](const SplitDesc &x) {
    const int each = 8 - part_groups(x.parts, a.most_groups);  // log2 of a group's threads
    static_assert(JOIN_THREADS == 1 << 8, "threads");
    return (cells + (1 << each) - 1) >> each;
  };
  int packed = 0;  // units << 20 | items: at most 320, and 320 * 16 * 128 / 8 below 2^17 of them
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = tid * PER + i;
    d[i].parts = 0;
    if (c < ctas) d[i] = a.desc[c];
    if (d[i].parts > 0) packed += 1 << 20 | items_of(d[i]);
  }
  int before = packed, all = 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += t;
  }
  if (lane == 31) wsum[warp] = before;
  before -= packed;
  __syncthreads();
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += wsum[w];
    all += wsum[w];
  }
  const int units = all >> 20, n_items = all & 0xFFFFF;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (d[i].parts > 0) {
      const int u = before >> 20;
      desc_s[u] = d[i];
      cta_s[u] = tid * PER + i;
      item_s[u] = before & 0xFFFFF;
      before += 1 << 20 | items_of(d[i]);
    }
  if (tid == 0) item_s[units] = n_items;
  __syncthreads();

  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    int u = 0;  // the last unit whose first item is at or before this one
#pragma unroll
    for (int step = 256; step; step >>= 1)
      if (u + step < units && item_s[u + step] <= item) u += step;
    const SplitDesc ds = desc_s[u];
    const int c0 = cta_s[u], group_bits = part_groups(ds.parts, a.most_groups), groups = 1 << group_bits;
    const int each = JOIN_THREADS >> group_bits, grp = tid >> (8 - group_bits);
    const int e = (item - item_s[u]) * each + (tid & (each - 1)), c4 = e / a.rows_cap * 4, r = e % a.rows_cap;
    const bool in = e < cells && r < ds.rows;
    float M = -INFINITY, den = 0.f;
    float4 acc[4] = {};
    // A part in which the row saw nothing has the sum 0.  Its maximum does not
    // tell: that is -infinity as well where every score is NaN (a maximum passes
    // over NaN), and such a part, whose sum is NaN, makes the row NaN.
    auto add = [&](float2 ml, const float4 (&v)[4]) {
      if (ml.y == 0.f) return;
      const float mn = fmaxf(M, ml.x), f = M == -INFINITY ? 0.f : ex2(M - mn), h = ex2(ml.x - mn);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[q].x = fmaf(v[q].x, h, acc[q].x * f);
        acc[q].y = fmaf(v[q].y, h, acc[q].y * f);
        acc[q].z = fmaf(v[q].z, h, acc[q].z * f);
        acc[q].w = fmaf(v[q].w, h, acc[q].w * f);
      }
      den = fmaf(ml.y, h, den * f);
      M = mn;
    };
    if (in) {
      // part 0 lies in its CTA's second slot, the others in their CTAs' first
      for (int i0 = grp; i0 < ds.parts; i0 += 2 * groups) {
        float2 ml[2];
        float4 v[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = i0 + k * groups;
          ml[k] = make_float2(-INFINITY, 0.f);
          if (i < ds.parts) {
            const size_t p = (size_t)2 * (c0 + i * ds.stride) + (i == 0 ? 1 : 0);
            ml[k] = reinterpret_cast<const float2 *>(a.ml)[p * a.rows_cap + r];
            const float4 *src = reinterpret_cast<const float4 *>(a.part) + p * (D / 4) * a.rows_cap +
                                (a.row_major ? r * (D / 4) + c4 : c4 * a.rows_cap + r);
            const int step = a.row_major ? 1 : a.rows_cap;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[k][q] = src[q * step];
          }
        }
        add(ml[0], v[0]);
        add(ml[1], v[1]);
      }
    }
    if (groups > 1) {
      __syncthreads();  // the last item's readers are done
#pragma unroll
      for (int q = 0; q < 4; ++q) acc_s[q][tid] = acc[q];
      ml_s[tid] = make_float2(M, den);
      __syncthreads();
      if (grp == 0 && in)
        for (int g = 1; g < groups; ++g) {
          float4 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = acc_s[q][g * each + tid];
          add(ml_s[g * each + tid], v);
        }
    }
    if (in && grp == 0) {
      const float inv = den == 0.f ? 0.f : 1.f / den;
      const int node = ds.node0 + r / a.G, head = ds.head0 + r % a.G;
      uint4 *out = reinterpret_cast<uint4 *>(a.o + ((size_t)node * a.Hq + head) * D + c4 * 4);
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        uint4 x;
        x.x = pack2<FP16>(acc[q].x * inv, acc[q].y * inv);
        x.y = pack2<FP16>(acc[q].z * inv, acc[q].w * inv);
        x.z = pack2<FP16>(acc[q + 1].x * inv, acc[q + 1].y * inv);
        x.w = pack2<FP16>(acc[q + 1].z * inv, acc[q + 1].w * inv);
        out[q / 2] = x;
      }
    }
  }
}

}  // namespace
}  // namespace moe
