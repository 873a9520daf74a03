// Device view of a paged KV cache (cache.h) and the checks every kernel that
// reads its tables makes: slots, lengths and page numbers are device data.
#pragma once
#include "cache.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {

struct CacheView {
  uint16_t *k, *v;
  int32_t *refs, *table, *lens, *status;
  int n_layers, n_pages, page_shift, row;  // row: values of one position (n_kv_heads * head_dim)
  int n_slots, max_pages;
};

constexpr int CACHE_MAX_SEQS = 1024;  // sequences of one call

__device__ __forceinline__ int pages_of(int rows, int page_shift) {
  return (int)(((unsigned)rows + (1u << page_shift) - 1u) >> page_shift);
}

// The page of position block j of a slot, or -1 (status set) if the table names none.
__device__ __forceinline__ int table_page(const CacheView &c, int slot, int j) {
  const int p = c.table[(size_t)slot * c.max_pages + j];
  if ((unsigned)p < (unsigned)c.n_pages) return p;
  set_status(c.status, MOE_ERR_DEVICE_BOUNDS);
  return -1;
}

// A slot's length, or -1 if it does not fit the slot's table.
__device__ __forceinline__ int slot_len(const CacheView &c, int slot) {
  const int L = c.lens[slot];
  return L >= 0 && L <= ((long long)c.max_pages << c.page_shift) ? L : -1;
}

constexpr int COPY_THREADS = 256;     // of a copying CTA

// The last i in [0, n) with start[i] <= v (start ascending, start[0] <= v).
__device__ __forceinline__ int segment_of(const int *start, int n, int v) {
  int s = 0;
#pragma unroll
  for (int step = CACHE_MAX_SEQS / 2; step; step >>= 1)
    if (s + step < n && start[s + step] <= v) s += step;
  return s;
}

// One row (a multiple of 32 16-bit words) of K and V in `layers` layers, by one
// warp; strides in values from layer to layer.  Two layers at a time, so that
// eight 16-byte loads a lane are on their way before the first store.
__device__ __forceinline__ void copy_rows(uint16_t *kd, uint16_t *vd, const uint16_t *ks, const uint16_t *vs, int row,
                                          int layers, size_t to, size_t from) {
  const int lane = threadIdx.x & 31;
  auto at = [](const uint16_t *p, size_t i) { return reinterpret_cast<const uint4 *>(p) + i; };
  auto put = [](uint16_t *p, size_t i, uint4 x) { reinterpret_cast<uint4 *>(p)[i] = x; };
  int l = 0;
  for (; l + 2 <= layers; l += 2) {
#pragma unroll 2
    for (int i = lane; i < row / 8; i += 32) {
      const uint4 k0 = *at(ks, i), v0 = *at(vs, i), k1 = *at(ks + from, i), v1 = *at(vs + from, i);
      put(kd, i, k0);
      put(vd, i, v0);
      put(kd + to, i, k1);
      put(vd + to, i, v1);
    }
    kd += 2 * to, vd += 2 * to, ks += 2 * from, vs += 2 * from;
  }
  if (l < layers)
#pragma unroll 2
    for (int i = lane; i < row / 8; i += 32) {
      const uint4 k0 = *at(ks, i), v0 = *at(vs, i);
      put(kd, i, k0);
      put(vd, i, v0);
    }
}

// A sequence's part of an append, written by the plan and read by the copies.
struct AppendSeg {
  int32_t start;     // its first row in the call's count: copied page rows, then kept rows
  int32_t cow;       // rows to copy from old_page to a page of the sequence's own
  int32_t old_page;
  int32_t slot, len, src;  // len: before the append; src: its first row of k_new
};

struct AppendArgs {
  CacheView c;
  const uint16_t *k_new, *v_new;
  const int32_t *slots, *offsets, *n_keep, *path;
  int path_stride, B, n_rows;
  int32_t *rows;   // [2] rows to copy, 0 if the call changes nothing; jobs handed out (0 at first)
  AppendSeg *seg;  // [B]
  int32_t *pages;  // the pages found
  int per_job;     // layers a warp copies of a row
};

// Host: the view of a cache, after its dimensions and pointers are checked.
moe_status cache_view(const attn_cache *c, CacheView *out);
// Host: the same of any cache with the pool's pointers, whatever its values are; row_words: 16-bit words of a position.
moe_status cache_view_any(const void *k, const void *v, int32_t *refs, int32_t *table, int32_t *lens, int32_t *status,
                          int n_layers, int n_pages, int page_size, int n_kv_heads, int head_dim, int n_slots,
                          int max_pages, int row_words, CacheView *out);

// Host: what an append needs besides its cache and rows, checked, and the plan's launch.
struct AppendCall {
  const void *k_new, *v_new;
  const int32_t *slots, *offsets, *n_keep, *path;
  int path_stride, B, n_rows;
  void *ws;
  size_t ws_bytes;
};
size_t append_ws(int page_size, int B, int n_rows, size_t *pages_at);
// The arguments of an append's kernels; MOE_OK with a->B == 0: nothing to do.
// new_words: 16-bit words of a new row of k_new (and of v_new).
moe_status append_args(const CacheView &c, const AppendCall &call, int new_words, AppendArgs *a);
cudaError_t launch_append_plan(const AppendArgs &a, cudaStream_t s);
// Host: forks and cuts, of any cache.  ks, vs: scales [layers][pages][heads], or null.
size_t fork_ws(int n);
moe_status fork_call(const CacheView &c, const int32_t *src, const int32_t *dst, int n, void *ws, size_t ws_bytes,
                     float *ks, float *vs, int heads, cudaStream_t s);
moe_status trim_call(const CacheView &c, const int32_t *slots, const int32_t *new_lens, int n, cudaStream_t s);

// Warps of a copy at most: eight CTAs for each of 152 SMs.
constexpr int COPY_CTAS = 152 * 8, COPY_WARPS = COPY_CTAS * (COPY_THREADS / 32);

// Layers a warp copies of a row: all of them where the rows alone fill the
// GPU twice, so that a row's place is looked up once; else enough to.  One layer
// always, this rule, all always, us: 24 prompts of up to 500 rows, 10 layers, 89.8,
// 71.2, 71.2; 24 forks into 96 54.1, 46.6, 44.1; four rows 6.8, 6.8, 8.8; one fork
// into four 8.8, 8.8, 12.1.  (Between the two all would be better: 64 x 64 rows 38.0, 38.0, 30.4.)
inline int layers_per_job(long long rows, int n_layers) {
  const long long n = rows * n_layers / (2 * COPY_WARPS);
  return (int)(n < 1 ? 1 : n > n_layers ? n_layers : n);
}

inline int copy_grid(long long rows, int n_layers, int per_job) {
  const long long jobs = rows * ((n_layers + per_job - 1) / per_job);
  const long long g = (jobs + COPY_THREADS / 32 - 1) / (COPY_THREADS / 32);
  return (int)(g < 1 ? 1 : g > COPY_CTAS ? COPY_CTAS : g);
}

}  // namespace moe
