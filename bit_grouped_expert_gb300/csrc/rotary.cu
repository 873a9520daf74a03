// Rotary positions (rotary.h): rows turned by their positions, and appending to
// the paged cache with the K rows turned on the way.
//
// A lane turns sixteen values of a head, the same ones of every head that its
// warp goes over, so that a position's cosines and sines are made once: with
// that HBM bounds large calls (8,191 rows of 16 heads of 256, bf16: 26.4 us, 5.1 TB/s; in
// the append, where 24 prompts' 9,318 rows in 10 layers of 2 heads are copied as well as turned, 69.5 us,
// 5.5 TB/s), the host small ones (one row 6.9 us).
#include "rotary.cuh"

#include <math.h>

#include "cache.cuh"

namespace moe {
namespace {

struct RotaryArgs {
  attn_rotary_table table;
  const uint16_t *x;
  uint16_t *o;
  const int32_t *positions;
  int64_t x_stride, o_stride;
  int n_rows, n_heads, head_dim;
  int per_job;  // groups of heads a warp turns of a row
};

constexpr int ROT_THREADS = 256;

template <bool FP16>
__global__ void __launch_bounds__(ROT_THREADS) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  const int lane = threadIdx.x & 31, items = a.head_dim / 16, together = 32 / items;  // heads of a group
  RotaryItem item(&a.table, lane % items);
  start_dependent();
  const int groups = (a.n_heads + together - 1) / together, jobs = (groups + a.per_job - 1) / a.per_job;
  const long long warps = (long long)gridDim.x * (ROT_THREADS / 32);
  for (long long job = (long long)blockIdx.x * (ROT_THREADS / 32) + (threadIdx.x >> 5);
       job < (long long)a.n_rows * jobs; job += warps) {
    const long long row = job / jobs;
    const int g0 = (int)(job - row * jobs) * a.per_job, g1 = min(groups, g0 + a.per_job);
    const int p = a.positions[row];
    const uint16_t *x = a.x + row * a.x_stride;
    uint16_t *o = a.o + row * a.o_stride;
    constexpr int AHEAD = 4;  // groups in flight (2, 4, 8 in the case above: 33.3, 26.9, 37.5 us)
    bool first = true;
    for (int g = g0; g < g1; g += AHEAD) {
      uint4 u[AHEAD], v[AHEAD];
      int at[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int head = (g + i) * together + lane / items;
        at[i] = g + i < g1 && head < a.n_heads ? head * a.head_dim : -1;
        if (at[i] >= 0) {
          u[i] = *reinterpret_cast<const uint4 *>(x + at[i] + item.a);
          v[i] = *reinterpret_cast<const uint4 *>(x + at[i] + item.b);
        }
      }
      if (first) item.at(p);  // (while the values are on their way)
      first = false;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (at[i] < 0) continue;
        item.turn_halves<FP16>(u[i], v[i]);
        *reinterpret_cast<uint4 *>(o + at[i] + item.a) = u[i];
        *reinterpret_cast<uint4 *>(o + at[i] + item.b) = v[i];
      }
    }
  }
}

// As append_copy_kernel, with K turned.
template <bool FP16>
__global__ void __launch_bounds__(COPY_THREADS)
    append_rotary_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ attn_rotary_table table, int head_dim) {
  __shared__ int start_s[CACHE_MAX_SEQS];
  const int lane = threadIdx.x & 31, items = head_dim / 16, together = 32 / items;
  RotaryItem item(&table, lane % items);
  start_dependent();
  const CacheView &c = a.c;
  const int rows = *a.rows, in_page = (1 << c.page_shift) - 1, heads = c.row / head_dim;
  if (rows == 0) return;
  for (int b = threadIdx.x; b < a.B; b += COPY_THREADS) start_s[b] = a.seg[b].start;
  __syncthreads();
  const long long warps = (long long)gridDim.x * (COPY_THREADS / 32);
  const int jobs = (c.n_layers + a.per_job - 1) / a.per_job;
  const size_t pool = ((size_t)c.n_pages << c.page_shift) * c.row;
  for (long long job = (long long)blockIdx.x * (COPY_THREADS / 32) + (threadIdx.x >> 5);
       job < (long long)rows * jobs; job += warps) {
    const int group = (int)(job / rows), r = (int)(job - (long long)group * rows);
    const int layer = group * a.per_job, layers = min(a.per_job, c.n_layers - layer);
    const int b = segment_of(start_s, a.B, r);
    const AppendSeg g = a.seg[b];
    int i = r - g.start;
    const bool copied = i < g.cow;
    const int at = copied ? (g.len & ~in_page) + i : g.len + (i -= g.cow);
    const int page = c.table[(size_t)g.slot * c.max_pages + (at >> c.page_shift)];
    if ((unsigned)page >= (unsigned)c.n_pages) continue;
    const size_t dst = (((size_t)layer * c.n_pages + page) * (in_page + 1) + (at & in_page)) * c.row;
    if (copied) {
      const size_t src = (((size_t)layer * c.n_pages + g.old_page) * (in_page + 1) + i) * c.row;
      copy_rows(c.k + dst, c.v + dst, c.k + src, c.v + src, c.row, layers, pool, pool);
      continue;
    }
    const size_t from = (size_t)a.n_rows * c.row;
    const size_t src = (size_t)layer * from +
                       (size_t)(g.src + (a.path ? a.path[(size_t)b * a.path_stride + i] : i)) * c.row;
    const int groups = (heads + together - 1) / together, all = layers * groups;
    constexpr int AHEAD = 2;  // heads in flight (1, 2, 4: the whole call 89.6, 80.8, 106 us)
    bool first = true;
    for (int n = 0; n < all; n += AHEAD) {
      uint4 k0[AHEAD], k1[AHEAD], v0[AHEAD], v1[AHEAD];
      size_t d[AHEAD];
      bool in[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int l = (n + u) / groups, h = (n + u - l * groups) * together + lane / items;
        in[u] = n + u < all && h < heads;
        if (!in[u]) continue;
        const size_t s = src + l * from + h * head_dim;
        d[u] = dst + l * pool + h * head_dim;
        k0[u] = *reinterpret_cast<const uint4 *>(a.k_new + s + item.a);
        k1[u] = *reinterpret_cast<const uint4 *>(a.k_new + s + item.b);
        v0[u] = *reinterpret_cast<const uint4 *>(a.v_new + s + item.a);
        v1[u] = *reinterpret_cast<const uint4 *>(a.v_new + s + item.b);
      }
      if (first) item.at(at);  // (while the values are on their way)
      first = false;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        if (!in[u]) continue;
        item.turn_halves<FP16>(k0[u], k1[u]);
        *reinterpret_cast<uint4 *>(c.k + d[u] + item.a) = k0[u];
        *reinterpret_cast<uint4 *>(c.k + d[u] + item.b) = k1[u];
        *reinterpret_cast<uint4 *>(c.v + d[u] + item.a) = v0[u];
        *reinterpret_cast<uint4 *>(c.v + d[u] + item.b) = v1[u];
      }
    }
  }
}

}  // namespace

moe_status rotary_check(const attn_rotary_table *t, int head_dim) {
  if (!t || (t->interleaved != 0 && t->interleaved != 1) || !isfinite(t->factor)) return MOE_ERR_INVALID_ARGUMENT;
  if (t->dim < 16 || t->dim % 16 || t->dim > head_dim) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace moe

extern "C" moe_status attn_rotary_plan(const attn_rotary_config *cfg, attn_rotary_table *table) {
  if (!cfg || !table) return MOE_ERR_INVALID_ARGUMENT;
  const double low = cfg->low_turns, high = cfg->high_turns;
  const bool by_turns = high != 0.0 || low != 0.0;
  if (!(cfg->base > 0.0) || !isfinite(cfg->base) || !(cfg->stretch > 0.0) || !isfinite(cfg->stretch) ||
      !isfinite(cfg->factor) || (cfg->interleaved != 0 && cfg->interleaved != 1) ||
      (by_turns && (!(low >= 0.0) || !(high > low) || !isfinite(high) || !(cfg->original_len > 0.0) ||
                    !isfinite(cfg->original_len))))
    return MOE_ERR_INVALID_ARGUMENT;
  if (cfg->dim < 16 || cfg->dim % 16 || cfg->dim > 256) return MOE_ERR_UNSUPPORTED;
  attn_rotary_table t = {};
  t.dim = cfg->dim;
  t.interleaved = cfg->interleaved;
  t.factor = cfg->factor;
  constexpr double TWO_PI = 6.283185307179586476925;
  for (int i = 0; i < cfg->dim / 2; ++i) {
    double f = pow(cfg->base, -2.0 * i / cfg->dim) / TWO_PI, g = 0.0;  // turns a position
    if (by_turns) g = fmin(fmax((cfg->original_len * f - low) / (high - low), 0.0), 1.0);
    f *= g + (1.0 - g) / cfg->stretch;
    if (!isfinite(f)) return MOE_ERR_INVALID_ARGUMENT;
    t.turns[i] = (uint64_t)ldexp(f - floor(f), 64);  // the fraction is below 1 - 2^-54, so this fits
  }
  *table = t;
  return MOE_OK;
}

extern "C" moe_status attn_rotary(const attn_rotary_table *table, const void *x_d, int64_t x_stride, int32_t dtype,
                                  const int32_t *positions_d, int32_t n_rows, int32_t n_heads, int32_t head_dim,
                                  void *o_d, int64_t o_stride, void *stream) {
  using moe::aligned16;
  if (!table || n_rows < 0 || n_heads < 1) return MOE_ERR_INVALID_ARGUMENT;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || n_heads > 65536 ||
      (dtype != MOE_BF16 && dtype != MOE_FP16))
    return MOE_ERR_UNSUPPORTED;
  const moe_status st = moe::rotary_check(table, head_dim);
  if (st != MOE_OK) return st;
  const int64_t row = (int64_t)n_heads * head_dim;
  if (x_stride < row || o_stride < row || x_stride > INT64_MAX / 2 / (n_rows + 1ll) ||
      o_stride > INT64_MAX / 2 / (n_rows + 1ll))
    return MOE_ERR_INVALID_ARGUMENT;
  if (n_rows == 0) return MOE_OK;
  if (!x_d || !positions_d || !o_d) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned16(x_d) || !aligned16(positions_d) || !aligned16(o_d) || x_stride % 8 || o_stride % 8)
    return MOE_ERR_MISALIGNED;
  const size_t nx = (size_t)((n_rows - 1) * x_stride + row) * 2, no = (size_t)((n_rows - 1) * o_stride + row) * 2;
  if (((x_d != o_d || x_stride != o_stride) && moe::ranges_meet(x_d, nx, o_d, no)) ||
      moe::ranges_meet(positions_d, (size_t)n_rows * 4, o_d, no))
    return MOE_ERR_INVALID_ARGUMENT;
  moe::RotaryArgs a;
  a.table = *table;
  a.x = static_cast<const uint16_t *>(x_d);
  a.o = static_cast<uint16_t *>(o_d);
  a.positions = positions_d;
  a.x_stride = x_stride;
  a.o_stride = o_stride;
  a.n_rows = n_rows;
  a.n_heads = n_heads;
  a.head_dim = head_dim;
  // A warp's groups of heads of a row: all of them where the rows alone fill half of
  // the GPU, so that a position's angles are made once (8,191 rows of 16 heads of 256: one
  // group a warp 45.7 us, all 26); else as many as leave the GPU half full.
  const int together = 512 / head_dim, groups = (n_heads + together - 1) / together;
  const long long per = (long long)n_rows * groups * 2 / moe::COPY_WARPS;
  a.per_job = (int)(per < 1 ? 1 : per > groups ? groups : per);
  const long long jobs = (long long)n_rows * ((groups + a.per_job - 1) / a.per_job);
  const long long ctas = (jobs + moe::ROT_THREADS / 32 - 1) / (moe::ROT_THREADS / 32);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool chain = moe::prof_chain(0);
  const dim3 grid((unsigned)(ctas < moe::COPY_CTAS ? ctas : moe::COPY_CTAS));
  return moe::note_cuda_error(
      dtype == MOE_FP16 ? moe::launch_dep(chain, moe::rotary_kernel<true>, grid, dim3(moe::ROT_THREADS), 0, s, a)
                        : moe::launch_dep(chain, moe::rotary_kernel<false>, grid, dim3(moe::ROT_THREADS), 0, s, a));
}

extern "C" moe_status attn_cache_append_rotary(const attn_cache *c, const attn_rotary_table *table,
                                               const void *k_new_d, const void *v_new_d, const int32_t *slots_d,
                                               const int32_t *offsets_d, const int32_t *n_keep_d,
                                               const int32_t *path_d, int32_t path_stride, int32_t B, int32_t n_rows,
                                               void *ws_d, size_t ws_bytes, void *stream) {
  moe::CacheView v;
  moe::AppendArgs a;
  moe_status st = moe::cache_view(c, &v);
  if (st == MOE_OK) st = moe::rotary_check(table, c->head_dim);
  if (st != MOE_OK) return st;
  st = moe::append_args(v, moe::AppendCall{k_new_d, v_new_d, slots_d, offsets_d, n_keep_d, path_d, path_stride, B, n_rows,
                                           ws_d, ws_bytes}, v.row, &a);
  if (st != MOE_OK || a.B == 0) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = moe::launch_append_plan(a, s);
  if (e != cudaSuccess) return moe::note_cuda_error(e);
  const bool pdl = moe::prof_quiet(MOE_KERNEL_CACHE_COPY);
  moe::prof_before(MOE_KERNEL_CACHE_COPY, s);
  const dim3 grid(moe::copy_grid(n_rows + B, c->n_layers, a.per_job)), block(moe::COPY_THREADS);
  e = c->dtype == MOE_FP16
          ? moe::launch_dep(pdl, moe::append_rotary_kernel<true>, grid, block, 0, s, a, *table, c->head_dim)
          : moe::launch_dep(pdl, moe::append_rotary_kernel<false>, grid, block, 0, s, a, *table, c->head_dim);
  moe::prof_after(MOE_KERNEL_CACHE_COPY, s);
  return moe::note_cuda_error(e);
}
