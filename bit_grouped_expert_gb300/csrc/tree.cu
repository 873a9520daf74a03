// Attention of drafted trees over a paged cache (tree.h).
//
// One CTA per (node, query head); its four warps take every fourth position
// with a running maximum and sum and merge at the end.
#include <cuda_fp16.h>
#include <math.h>

#include "cache.cuh"
#include "kernels.h"
#include "tree.h"

namespace moe {
namespace {

constexpr int AT_MAXN = 256;  // nodes of a tree

struct TreeArgs {
  CacheView c;
  const uint16_t *q, *k_new, *v_new;
  const int32_t *slots, *offsets, *parent;
  uint16_t *o;
  int B, n_nodes, max_nodes, Hq, Hkv, layer;
  float scale_log2;
};

template <bool FP16>
__device__ __forceinline__ float to_f32(uint16_t h) {
  if constexpr (FP16)
    return __half2float(__ushort_as_half(h));
  else
    return bf16_to_f32(h);
}
template <bool FP16>
__device__ __forceinline__ uint16_t from_f32(float f) {
  if constexpr (FP16)
    return __half_as_ushort(__float2half_rn(f));
  else
    return f32_to_bf16(f);
}

template <int D, bool FP16>
__global__ void __launch_bounds__(128) tree_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int E = D / 32;
  __shared__ float o_s[4][D], m_s[4], l_s[4];
  const int node = blockIdx.x, h = blockIdx.y, g = h / (a.Hq / a.Hkv), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const CacheView &c = a.c;
  int b = 0;
  while (b < a.B && !(a.offsets[b] <= node && node < a.offsets[b + 1])) ++b;
  if (b == a.B) return;
  const int lo = a.offsets[b], slot = a.slots ? a.slots[b] : b;
  int L = slot >= 0 && slot < c.n_slots ? slot_len(c, slot) : -1;
  if (lo < 0 || a.offsets[b + 1] > a.n_nodes || a.offsets[b + 1] - lo > a.max_nodes || L < 0) {
    if (threadIdx.x == 0) set_status(c.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  if (a.parent[node] == -2) L = 0;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = to_f32<FP16>(a.q[((size_t)node * a.Hq + h) * D + e * 32 + lane]) * a.scale_log2;
  auto take = [&](const uint16_t *k, const uint16_t *v) {
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], to_f32<FP16>(k[e * 32 + lane]), s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, to_f32<FP16>(v[e * 32 + lane]), o[e] * f);
    l = l * f + w;
    m = mn;
  };
  for (int p = warp; p < L; p += 4) {
    const int page = table_page(c, slot, p >> c.page_shift);
    if (page < 0) break;
    const size_t row = ((((size_t)a.layer * c.n_pages + page) << c.page_shift) + (p & ((1 << c.page_shift) - 1))) * c.row;
    take(c.k + row + g * D, c.v + row + g * D);
  }
  int i = node - lo, step = 0;
  if (a.parent[node] == -2) i = -1;
  while (i >= 0) {
    const size_t row = (size_t)(lo + i) * c.row + g * D;
    if ((step++ & 3) == warp) take(a.k_new + row, a.v_new + row);
    const int up = a.parent[lo + i];
    if (up >= i || up < -1) {
      if (threadIdx.x == 0) set_status(c.status, MOE_ERR_DEVICE_BOUNDS);
      break;
    }
    i = up;
  }
  for (int e = 0; e < E; ++e) o_s[warp][e * 32 + lane] = o[e];
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY, den = 0.f;
  for (int w = 0; w < 4; ++w) M = fmaxf(M, m_s[w]);
  for (int w = 0; w < 4; ++w) den += m_s[w] == -INFINITY ? 0.f : exp2f(m_s[w] - M) * l_s[w];
  for (int d = threadIdx.x; d < D; d += 128) {
    float s = 0.f;
    for (int w = 0; w < 4; ++w) s += m_s[w] == -INFINITY ? 0.f : exp2f(m_s[w] - M) * o_s[w][d];
    a.o[((size_t)node * a.Hq + h) * D + d] = from_f32<FP16>(M == -INFINITY ? 0.f : s / den);
  }
}

template <int D>
cudaError_t launch_tree(const TreeArgs &a, bool fp16, cudaStream_t s) {
  const dim3 grid(a.n_nodes, a.Hq);
  return fp16 ? launch_dep(false, tree_kernel<D, true>, grid, dim3(128), 0, s, a)
              : launch_dep(false, tree_kernel<D, false>, grid, dim3(128), 0, s, a);
}

}  // namespace
}  // namespace moe

extern "C" size_t attn_tree_workspace_bytes(const attn_cache *c, int32_t B, int32_t n_nodes, int32_t max_nodes,
                                            int32_t Hq) {
  moe::CacheView v;
  if (moe::cache_view(c, &v) != MOE_OK || B < 1 || n_nodes < 1 || max_nodes < 1 || Hq < 1) return 0;
  return 16;
}

extern "C" moe_status attn_tree(const attn_cache *c, int32_t layer, const void *q_d, const void *k_new_d,
                                const void *v_new_d, const int32_t *slots_d, const int32_t *offsets_d,
                                const int32_t *parent_d, int32_t B, int32_t n_nodes, int32_t max_nodes, int32_t Hq,
                                float scale, void *ws_d, size_t ws_bytes, void *o_d, void *stream) {
  using moe::aligned16;
  moe::TreeArgs a;
  const moe_status st = moe::cache_view(c, &a.c);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= c->n_layers || B < 0 || n_nodes < 0 || max_nodes < 1 || Hq < 1 || !(scale >= 0.f) ||
      isinf(scale))
    return MOE_ERR_INVALID_ARGUMENT;
  if (Hq % c->n_kv_heads || Hq / c->n_kv_heads > 128 || max_nodes > moe::AT_MAXN || B > moe::CACHE_MAX_SEQS)
    return MOE_ERR_UNSUPPORTED;
  if (B == 0 || n_nodes == 0) return MOE_OK;
  if (!q_d || !k_new_d || !v_new_d || !offsets_d || !parent_d || !ws_d || !o_d) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned16(q_d) || !aligned16(k_new_d) || !aligned16(v_new_d) || !aligned16(slots_d) ||
      !aligned16(offsets_d) || !aligned16(parent_d) || !aligned16(ws_d) || !aligned16(o_d))
    return MOE_ERR_MISALIGNED;
  if (ws_bytes < attn_tree_workspace_bytes(c, B, n_nodes, max_nodes, Hq)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (scale == 0.f) scale = 1.f / sqrtf((float)c->head_dim);
  a.q = static_cast<const uint16_t *>(q_d);
  a.k_new = static_cast<const uint16_t *>(k_new_d);
  a.v_new = static_cast<const uint16_t *>(v_new_d);
  a.slots = slots_d;
  a.offsets = offsets_d;
  a.parent = parent_d;
  a.o = static_cast<uint16_t *>(o_d);
  a.B = B;
  a.n_nodes = n_nodes;
  a.max_nodes = max_nodes;
  a.Hq = Hq;
  a.Hkv = c->n_kv_heads;
  a.layer = layer;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp16 = c->dtype == MOE_FP16;
  moe::prof_before(MOE_KERNEL_ATTN_TREE, s);
  const cudaError_t e = c->head_dim == 64    ? moe::launch_tree<64>(a, fp16, s)
                        : c->head_dim == 128 ? moe::launch_tree<128>(a, fp16, s)
                                             : moe::launch_tree<256>(a, fp16, s);
  moe::prof_after(MOE_KERNEL_ATTN_TREE, s);
  return moe::note_cuda_error(e);
}
