// Appending to the 8-bit paged KV cache (qcache.h); its forks and cuts are the
// 16-bit cache's (cache.cu), which move codes as they are.
//
// After the plan (cache.cu) a CTA takes one part, the rows that the call adds to
// one page, of K or of V in one layer, and as many heads as make up some 16,384
// values: it finds each head's largest value, settles the scales, rounds the
// page's earlier codes anew where their scale grew (or moves them, where the
// page is a copy), and writes the new rows' codes.
#include "qcache.cuh"
#include "rotary.cuh"

namespace moe {
namespace {

constexpr int QA_THREADS = 256;

struct QAppendArgs {
  AppendArgs a;
  QCacheView q;
  attn_rotary_table table;
  int turns;       // K rows are turned
  int heads_job;   // heads of a job
};

__device__ __forceinline__ float largest(const float (&x)[8], const float (&y)[8], float most) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = fabsf(x[i]), v = fabsf(y[i]);
    if (u < INFINITY) most = fmaxf(most, u);  // NaN and infinity do not count
    if (v < INFINITY) most = fmaxf(most, v);
  }
  return most;
}
// Codes of eight values times f; infinities become NaN as well.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float u = x[2 * i] * f, v = x[2 * i + 1] * f;
    w[i] = to_codes(fabsf(u) < INFINITY ? u : NAN, fabsf(v) < INFINITY ? v : NAN);
  }
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

template <bool FP16>
__global__ void __launch_bounds__(QA_THREADS) qcache_append_kernel(const __grid_constant__ QAppendArgs g) {
  __shared__ int parts_s[CACHE_MAX_SEQS], wsum[QA_THREADS / 32], total_s;
  __shared__ unsigned most_s[256];
  __shared__ float inv_s[256], grow_s[256];
  start_dependent();
  const AppendArgs &a = g.a;
  const CacheView &c = a.c;
  const int rows = *a.rows, shift = c.page_shift, in_page = (1 << shift) - 1;
  if (rows == 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto kept = [&](int b) {  // rows the call adds to sequence b
    return (b + 1 < a.B ? a.seg[b + 1].start : rows) - a.seg[b].start - a.seg[b].cow;
  };
  // the parts before each sequence's
  constexpr int PER = CACHE_MAX_SEQS / QA_THREADS;
  int mine[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    mine[i] = sum;
    if (b < a.B) {
      const int n = kept(b), len = a.seg[b].len;
      if (n > 0) sum += ((len + n - 1) >> shift) - (len >> shift) + 1;
    }
  }
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) wsum[warp] = upto;
  __syncthreads();
  int before = upto - sum, total = 0;
  for (int w = 0; w < QA_THREADS / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (tid * PER + i < a.B) parts_s[tid * PER + i] = before + mine[i];
  __syncthreads();

  const int D = g.q.dim, items = D / 16, groups = (g.q.heads + g.heads_job - 1) / g.heads_job;
  const size_t row_bytes = (size_t)c.row * 2;
  const int new_row = g.q.heads * D;  // values of a new row
  const long long jobs = (long long)total * c.n_layers * 2 * groups;
  for (long long job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int part = (int)(job / (c.n_layers * 2 * groups)), rest = (int)(job % (c.n_layers * 2 * groups));
    const int layer = rest / (2 * groups), is_v = rest / groups & 1, h0 = rest % groups * g.heads_job;
    const int heads = min(g.heads_job, g.q.heads - h0);
    // the last sequence whose parts begin at or before this one (those without parts begin where the next does)
    const int b = segment_of(parts_s, a.B, part);
    const AppendSeg seg = a.seg[b];
    const int n = kept(b), nth = part - parts_s[b];
    const int first = nth == 0 ? seg.len : ((seg.len >> shift) + nth) << shift;  // its first new position
    const int count = min(seg.len + n, ((first >> shift) + 1) << shift) - first;
    const int old = nth == 0 ? first & in_page : 0;  // the page's earlier rows
    const int page = c.table[(size_t)seg.slot * c.max_pages + (first >> shift)];
    if ((unsigned)page >= (unsigned)c.n_pages) continue;
    const int from_page = nth == 0 && seg.cow ? seg.old_page : page;
    uint8_t *pool = reinterpret_cast<uint8_t *>(is_v ? c.v : c.k) + (size_t)layer * c.n_pages * (in_page + 1) * row_bytes;
    uint8_t *to = pool + ((size_t)page << shift) * row_bytes;
    const uint8_t *from = pool + ((size_t)from_page << shift) * row_bytes;
    float *scales = (is_v ? g.q.vs : g.q.ks) + (size_t)layer * c.n_pages * g.q.heads;
    const uint16_t *x = (is_v ? a.v_new : a.k_new) + (size_t)layer * a.n_rows * new_row;
    const int per_row = heads * items, lane_item = tid % items;
    // (the threads are a multiple of a head's items: a thread has the same one throughout)
    RotaryItem item(g.turns && !is_v ? &g.table : nullptr, lane_item);
    __syncthreads();  // the last job's readers are done
    if (tid < heads) most_s[tid] = 0;
    __syncthreads();
    auto load = [&](int e, int &head, float (&u)[8], float (&v)[8]) {
      const int r = e / per_row, i = first - seg.len + r;
      head = (e - r * per_row) / items;
      const size_t row = (size_t)seg.src + (a.path ? a.path[(size_t)b * a.path_stride + i] : i);
      const uint16_t *p = x + row * new_row + (h0 + head) * D;
      unpack8<FP16>(*reinterpret_cast<const uint4 *>(p + item.a), u);
      unpack8<FP16>(*reinterpret_cast<const uint4 *>(p + item.b), v);
      item.at(first + r);
      item.turn(u, v);
      return r;
    };
    for (int e = tid; e < count * per_row; e += QA_THREADS) {
      int head;
      float u[8], v[8];
      load(e, head, u, v);
      atomicMax(&most_s[head], __float_as_uint(largest(u, v, 0.f)));
    }
    __syncthreads();
    if (tid < heads) {
      float s = exp2_int(scale_exp(__uint_as_float(most_s[tid]))), was = s;
      if (old) {
        was = scales[(size_t)from_page * g.q.heads + h0 + tid];
        s = fmaxf(s, was);
      }
      scales[(size_t)page * g.q.heads + h0 + tid] = s;
      inv_s[tid] = 1.f / s;
      grow_s[tid] = was / s;
    }
    __syncthreads();
    if (old)
      for (int e = tid; e < old * per_row; e += QA_THREADS) {
        const int r = e / per_row, head = (e - r * per_row) / items;
        const float f = grow_s[head];
        if (f == 1.f && from == to) continue;
        const size_t at = r * row_bytes + (size_t)(h0 + head) * D + lane_item * 16;
        uint4 w = *reinterpret_cast<const uint4 *>(from + at);
        if (f != 1.f) {
          uint32_t *p = &w.x;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 lo = from_codes(p[i] & 0xFFFFu), hi = from_codes(p[i] >> 16);
            p[i] = to_codes(lo.x * f, lo.y * f) | to_codes(hi.x * f, hi.y * f) << 16;
          }
        }
        *reinterpret_cast<uint4 *>(to + at) = w;
      }
    for (int e = tid; e < count * per_row; e += QA_THREADS) {
      int head;
      float u[8], v[8];
      const int r = load(e, head, u, v);
      uint8_t *at = to + ((first & in_page) + r) * row_bytes + (size_t)(h0 + head) * D;
      *reinterpret_cast<uint2 *>(at + item.a) = codes8(u, inv_s[head]);
      *reinterpret_cast<uint2 *>(at + item.b) = codes8(v, inv_s[head]);
    }
  }
}

}  // namespace

moe_status qcache_view(const attn_qcache *c, QCacheView *out) {
  if (!c || !c->k_scale_d || !c->v_scale_d) return MOE_ERR_INVALID_ARGUMENT;
  const moe_status st =
      cache_view_any(c->k_d, c->v_d, c->refs_d, c->table_d, c->lens_d, c->status_d, c->n_layers, c->n_pages,
                     c->page_size, c->n_kv_heads, c->head_dim, c->n_slots, c->max_pages,
                     c->n_kv_heads * c->head_dim / 2, &out->c);
  if (st != MOE_OK) return st;
  if (!aligned16(c->k_scale_d) || !aligned16(c->v_scale_d)) return MOE_ERR_MISALIGNED;
  out->ks = c->k_scale_d;
  out->vs = c->v_scale_d;
  out->heads = c->n_kv_heads;
  out->dim = c->head_dim;
  return MOE_OK;
}

}  // namespace moe

extern "C" size_t attn_qcache_append_workspace_bytes(const attn_qcache *c, int32_t B, int32_t n_rows) {
  moe::QCacheView v;
  if (moe::qcache_view(c, &v) != MOE_OK || B < 1 || B > moe::CACHE_MAX_SEQS || n_rows < 0) return 0;
  size_t at;
  return moe::append_ws(c->page_size, B, n_rows, &at);
}

extern "C" moe_status attn_qcache_append(const attn_qcache *c, const attn_rotary_table *table, const void *k_new_d,
                                         const void *v_new_d, int32_t dtype, const int32_t *slots_d,
                                         const int32_t *offsets_d, const int32_t *n_keep_d, const int32_t *path_d,
                                         int32_t path_stride, int32_t B, int32_t n_rows, void *ws_d, size_t ws_bytes,
                                         void *stream) {
  moe::QAppendArgs g;
  moe_status st = moe::qcache_view(c, &g.q);
  if (st == MOE_OK && table) st = moe::rotary_check(table, c->head_dim);
  if (st != MOE_OK) return st;
  if (dtype != MOE_BF16 && dtype != MOE_FP16) return MOE_ERR_UNSUPPORTED;
  st = moe::append_args(g.q.c, moe::AppendCall{k_new_d, v_new_d, slots_d, offsets_d, n_keep_d, path_d, path_stride, B,
                                               n_rows, ws_d, ws_bytes}, g.q.c.row * 2, &g.a);
  if (st != MOE_OK || g.a.B == 0) return st;
  g.turns = table != nullptr;
  if (table) g.table = *table;
  const int page_values = c->page_size * c->head_dim, fit = 16384 / page_values;
  g.heads_job = fit < 1 ? 1 : fit < c->n_kv_heads ? fit : c->n_kv_heads;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = moe::launch_append_plan(g.a, s);
  if (e != cudaSuccess) return moe::note_cuda_error(e);
  const long long parts = (long long)n_rows / c->page_size + 2ll * B;
  const long long jobs = parts * c->n_layers * 2 * ((c->n_kv_heads + g.heads_job - 1) / g.heads_job);
  const dim3 grid((unsigned)(jobs < moe::COPY_CTAS ? jobs : moe::COPY_CTAS)), block(moe::QA_THREADS);
  const bool pdl = moe::prof_quiet(MOE_KERNEL_CACHE_COPY);
  moe::prof_before(MOE_KERNEL_CACHE_COPY, s);
  e = dtype == MOE_FP16 ? moe::launch_dep(pdl, moe::qcache_append_kernel<true>, grid, block, 0, s, g)
                        : moe::launch_dep(pdl, moe::qcache_append_kernel<false>, grid, block, 0, s, g);
  moe::prof_after(MOE_KERNEL_CACHE_COPY, s);
  return moe::note_cuda_error(e);
}

extern "C" size_t attn_qcache_fork_workspace_bytes(const attn_qcache *c, int32_t n) {
  moe::QCacheView v;
  return moe::qcache_view(c, &v) == MOE_OK ? moe::fork_ws(n) : 0;
}

extern "C" moe_status attn_qcache_fork(const attn_qcache *c, const int32_t *src_d, const int32_t *dst_d, int32_t n,
                                       void *ws_d, size_t ws_bytes, void *stream) {
  moe::QCacheView v;
  const moe_status st = moe::qcache_view(c, &v);
  return st != MOE_OK ? st
                      : moe::fork_call(v.c, src_d, dst_d, n, ws_d, ws_bytes, v.ks, v.vs, v.heads,
                                       static_cast<cudaStream_t>(stream));
}

extern "C" moe_status attn_qcache_trim(const attn_qcache *c, const int32_t *slots_d, const int32_t *new_lens_d,
                                       int32_t n, void *stream) {
  moe::QCacheView v;
  const moe_status st = moe::qcache_view(c, &v);
  return st != MOE_OK ? st : moe::trim_call(v.c, slots_d, new_lens_d, n, static_cast<cudaStream_t>(stream));
}
