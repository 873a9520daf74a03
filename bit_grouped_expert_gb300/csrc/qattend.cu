// Attention over the 8-bit paged KV cache (qcache.h), in its simplest form: a
// CTA a (row, query head), a thread a position, the softmax in one pass with the
// running maximum and sum.
#include <math.h>

#include "kernels.h"
#include "qcache.cuh"
#include "rotary.cuh"

namespace moe {
namespace {

constexpr int AT_THREADS = 128;

struct AttendArgs {
  QCacheView q;
  int layer;
  const uint16_t *x;
  const int32_t *slots, *offsets;
  uint16_t *o;
  int B, n_rows, max_rows, Hq, G;
  float scale_log2;
};

template <bool FP16>
__global__ void __launch_bounds__(AT_THREADS) attend_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ float q_s[256], p_s[AT_THREADS], red[AT_THREADS / 32];
  __shared__ size_t at_s[AT_THREADS];
  start_dependent();
  const CacheView &c = a.q.c;
  const int row = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, D = a.q.dim, tid = threadIdx.x, g = h / a.G;
  int b = -1;
  for (int i = 0; i < a.B; ++i)
    if (a.offsets[i] <= row && row < a.offsets[i + 1]) b = i;
  if (b < 0) return;
  const int slot = a.slots ? a.slots[b] : b, lo = a.offsets[b], hi = a.offsets[b + 1];
  const int L = slot >= 0 && slot < c.n_slots ? slot_len(c, slot) : -1;
  if (L < 0 || lo < 0 || hi < lo || hi > a.n_rows || hi - lo > a.max_rows) {
    if (tid == 0) set_status(c.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  const int sees = L - (hi - lo) + (row - lo) + 1, in_page = (1 << c.page_shift) - 1;
  const size_t base = (size_t)a.layer * c.n_pages;
  const uint8_t *k = reinterpret_cast<const uint8_t *>(c.k), *v = reinterpret_cast<const uint8_t *>(c.v);
  for (int d = tid; d < D; d += AT_THREADS) q_s[d] = half_value<FP16>(a.x[((size_t)row * a.Hq + h) * D + d]);
  float m = -INFINITY, sum = 0.f, o[2] = {0.f, 0.f};
  for (int l0 = 0; l0 < sees; l0 += AT_THREADS) {
    __syncthreads();
    const int l = l0 + tid;
    float s = -INFINITY, vs = 0.f;
    at_s[tid] = 0;
    if (l < sees) {
      const int page = table_page(c, slot, l >> c.page_shift);
      if (page >= 0) {
        const size_t at = (((base + page) << c.page_shift) + (l & in_page)) * a.q.heads * D + (size_t)g * D;
        float dot = 0.f;
        for (int d = 0; d < D; d += 2) {
          const float2 x = from_codes(*reinterpret_cast<const uint16_t *>(k + at + d));
          dot = fmaf(q_s[d], x.x, fmaf(q_s[d + 1], x.y, dot));
        }
        s = dot * a.q.ks[(base + page) * a.q.heads + g] * a.scale_log2;
        vs = a.q.vs[(base + page) * a.q.heads + g];
        at_s[tid] = at;
      }
    }
    float most = s;
    for (int i = 16; i; i >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, i));
    if ((tid & 31) == 0) red[tid >> 5] = most;
    __syncthreads();
    for (int i = 0; i < AT_THREADS / 32; ++i) most = fmaxf(most, red[i]);
    most = fmaxf(most, m);
    const float f = m == -INFINITY ? 0.f : exp2f(m - most), base2 = most == -INFINITY ? 0.f : most;
    m = most;
    float p = l < sees ? exp2f(s - base2) : 0.f;
    p_s[tid] = p * vs;
    for (int i = 16; i; i >>= 1) p += __shfl_xor_sync(0xffffffffu, p, i);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = p;
    __syncthreads();
    sum *= f;
    for (int i = 0; i < AT_THREADS / 32; ++i) sum += red[i];
    for (int j = 0; j < 2; ++j) {
      const int d = tid + j * AT_THREADS;
      if (d >= D) continue;
      o[j] *= f;
      for (int i = 0; i < min(AT_THREADS, sees - l0); ++i)
        o[j] = fmaf(p_s[i], from_codes(v[at_s[i] + d]).x, o[j]);
    }
  }
  for (int j = 0; j < 2; ++j) {
    const int d = tid + j * AT_THREADS;
    if (d < D) a.o[((size_t)row * a.Hq + h) * D + d] = (uint16_t)half_pair<FP16>(sum == 0.f ? 0.f : o[j] / sum, 0.f);
  }
}

}  // namespace
}  // namespace moe

extern "C" size_t attn_qcache_attend_workspace_bytes(const attn_qcache *c, int32_t B, int32_t n_rows, int32_t max_rows,
                                                     int32_t Hq) {
  moe::QCacheView v;
  if (moe::qcache_view(c, &v) != MOE_OK || B < 1 || n_rows < 1 || max_rows < 1 || Hq < 1 || Hq % c->n_kv_heads ||
      Hq / c->n_kv_heads > 128)
    return 0;
  return 16;
}

extern "C" moe_status attn_qcache_attend(const attn_qcache *c, int32_t layer, const void *q_d, int32_t dtype,
                                         const int32_t *slots_d, const int32_t *offsets_d, int32_t B, int32_t n_rows,
                                         int32_t max_rows, int32_t Hq, float scale, void *ws_d, size_t ws_bytes,
                                         void *o_d, void *stream) {
  using moe::aligned16;
  moe::AttendArgs a;
  const moe_status st = moe::qcache_view(c, &a.q);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= c->n_layers || B < 0 || n_rows < 0 || max_rows < 1 || Hq < 1 || !(scale >= 0.f) ||
      isinf(scale))
    return MOE_ERR_INVALID_ARGUMENT;
  const int D = c->head_dim;
  if (Hq % c->n_kv_heads || Hq / c->n_kv_heads > 128 || B > moe::CACHE_MAX_SEQS ||
      (dtype != MOE_BF16 && dtype != MOE_FP16))
    return MOE_ERR_UNSUPPORTED;
  if (B == 0 || n_rows == 0) return MOE_OK;
  if (!q_d || !offsets_d || !ws_d || !o_d) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned16(q_d) || !aligned16(slots_d) || !aligned16(offsets_d) || !aligned16(ws_d) || !aligned16(o_d))
    return MOE_ERR_MISALIGNED;
  const size_t no = (size_t)n_rows * Hq * D * 2;
  const size_t np = (size_t)c->n_layers * c->n_pages * c->page_size * a.q.c.row * 2;
  const size_t ns = (size_t)c->n_layers * c->n_pages * c->n_kv_heads * 4;
  if (moe::ranges_meet(o_d, no, q_d, no) || moe::ranges_meet(o_d, no, c->k_d, np) ||
      moe::ranges_meet(o_d, no, c->v_d, np) || moe::ranges_meet(o_d, no, c->k_scale_d, ns) ||
      moe::ranges_meet(o_d, no, c->v_scale_d, ns))
    return MOE_ERR_INVALID_ARGUMENT;
  if (ws_bytes < attn_qcache_attend_workspace_bytes(c, B, n_rows, max_rows, Hq)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (scale == 0.f) scale = 1.f / sqrtf((float)D);
  a.layer = layer;
  a.x = static_cast<const uint16_t *>(q_d);
  a.slots = slots_d;
  a.offsets = offsets_d;
  a.o = static_cast<uint16_t *>(o_d);
  a.B = B;
  a.n_rows = n_rows;
  a.max_rows = max_rows;
  a.Hq = Hq;
  a.G = Hq / c->n_kv_heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool chain = moe::prof_chain(0);
  const dim3 grid((unsigned)(n_rows * Hq)), block(moe::AT_THREADS);
  return moe::note_cuda_error(dtype == MOE_FP16 ? moe::launch_dep(chain, moe::attend_kernel<true>, grid, block, 0, s, a)
                                                : moe::launch_dep(chain, moe::attend_kernel<false>, grid, block, 0, s, a));
}
