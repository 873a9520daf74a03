// The paged KV cache's bookkeeping and copies (cache.h).
//
// Appending and forking take two kernels each.  One CTA plans the call: it
// checks every sequence, adds up the pages they need, finds that many free
// pages from the lowest on (a scan over the holder counts that stops once it
// has enough) and hands them out.  A grid then copies rows of all layers, one
// warp per (row, layer).  Trimming only touches tables and holder counts.
//
// Each kernel is launched as a programmatic dependent of the one before it in
// the stream, whichever that is, and waits for it before it touches memory: a
// trim and an append back to back, most of whose time is starting kernels, took
// 7.2 us without that.
#include "cache.cuh"

#include "kernels.h"

namespace moe {
namespace {

// Threads of a planning CTA: one a sequence, and 128 where that is enough (its
// barriers and scans are most of a small call: with 512, four rows of one sequence
// 6.9 us for 6.8, one fork into four 9.1 for 8.8, 8 x 64 rows 11.7 for 11.5).  A large
// pool wants more: it is gone over from page 0 on, 2,048 pages a round at 128
// threads, and four rows take 126 us where 280,000 of 312,000 pages are held.
constexpr int PLAN_FEW = 128, PLAN_MANY = CACHE_MAX_SEQS;

// Exclusive prefix sum of one int per thread over the CTA; *total gets the
// sum.  Every thread calls it; red: 33 ints of shared memory.
__device__ __forceinline__ int block_scan(int v, int *red, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();  // an earlier call's readers are done
  if (lane == 31) red[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = lane < (int)(blockDim.x >> 5) ? red[lane] : 0;
    const int own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    red[lane] = w - own;
    if (lane == 31) red[32] = w;
  }
  __syncthreads();
  *total = red[32];
  return red[warp] + s - v;
}

// The `want` lowest pages without holders into list[0 .. want-1]; returns how
// many there are (at least want when it stopped early).  Sixteen pages a
// thread and round.
__device__ __forceinline__ int find_free(const CacheView &c, int want, int *red, int32_t *list) {
  int found = 0;
  for (int p0 = 0; p0 < c.n_pages && found < want; p0 += blockDim.x * 16) {
    const int p = p0 + threadIdx.x * 16;
    uint32_t free16 = 0;
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      if (p + i + 4 <= c.n_pages) {
        const int4 r = *reinterpret_cast<const int4 *>(c.refs + p + i);
        free16 |= ((r.x == 0 ? 1u : 0u) | (r.y == 0 ? 2u : 0u) | (r.z == 0 ? 4u : 0u) | (r.w == 0 ? 8u : 0u)) << i;
      } else {
        for (int j = i; j < i + 4; ++j)
          if (p + j < c.n_pages && c.refs[p + j] == 0) free16 |= 1u << j;
      }
    int total;
    int at = found + block_scan(__popc(free16), red, &total);
    for (uint32_t m = free16; m && at < want; m &= m - 1) list[at++] = p + __ffs(m) - 1;
    found += total;
  }
  return found;
}

// ---------------------------------------------------------------- append

template <int THREADS>
__global__ void __launch_bounds__(THREADS) append_plan_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ int red[33], slot_s[THREADS], first_s[THREADS], block_s[THREADS], bad;
  start_dependent();
  const CacheView &c = a.c;
  const int b = threadIdx.x, in_page = (1 << c.page_shift) - 1;
  const bool in = b < a.B;
  if (b == 0) bad = 0;
  int slot = -1, L = 0, n = 0, lo = 0, have = 0;
  bool ok = true;
  if (in) {
    slot = a.slots ? a.slots[b] : b;
    lo = a.offsets[b];
    const int hi = a.offsets[b + 1];
    ok = slot >= 0 && slot < c.n_slots && lo >= 0 && lo <= hi && hi <= a.n_rows;
    if (ok) {
      L = slot_len(c, slot);
      have = hi - lo;
      n = a.n_keep ? a.n_keep[b] : have;
      ok = L >= 0 && n >= 0 && n <= have && (!a.path || n <= a.path_stride) &&
           (long long)L + n <= ((long long)c.max_pages << c.page_shift);
    }
    slot_s[b] = slot;
  }
  __syncthreads();
  int need = 0, cow = 0, old_page = -1;
  if (in && ok) {
    bool wrong = false;  // all looked at: no load or compare waits for the one before
    if (a.slots)
#pragma unroll 8
      for (int i = 0; i < b; ++i) wrong |= slot_s[i] == slot;
    if (a.path)
#pragma unroll 8
      for (int i = 0; i < n; ++i) wrong |= (unsigned)a.path[(size_t)b * a.path_stride + i] >= (unsigned)have;
    ok = !wrong;
    if (ok && n > 0) {
      need = pages_of(L + n, c.page_shift) - pages_of(L, c.page_shift);
      if (L & in_page) {
        old_page = table_page(c, slot, L >> c.page_shift);
        ok = old_page >= 0;
        if (ok && c.refs[old_page] > 1) {  // other holders: its rows move to a page of its own
          cow = L & in_page;
          ++need;
        }
      }
    }
  }
  if (!ok) bad = 1;
  int total, rows;
  const int first = block_scan(need, red, &total);
  const int start = block_scan(n + cow, red, &rows);
  if (bad) {  // written before the scans' barriers
    if (b == 0) {
      set_status(c.status, MOE_ERR_DEVICE_BOUNDS);
      *a.rows = 0;
    }
    return;
  }
  if (find_free(c, total, red, a.pages) < total) {
    if (b == 0) {
      set_status(c.status, MOE_ERR_OUT_OF_PAGES);
      *a.rows = 0;
    }
    return;
  }
  if (in) {
    first_s[b] = first;
    block_s[b] = cow ? L >> c.page_shift : pages_of(L, c.page_shift);
    a.seg[b] = AppendSeg{start, cow, old_page, slot, L, lo};
    c.lens[slot] = L + n;
    if (cow) atomicSub(&c.refs[old_page], 1);
  }
  if (b == 0) {
    a.rows[0] = rows;
    a.rows[1] = 0;
  }
  __syncthreads();
  for (int k = b; k < total; k += THREADS) {
    const int s = segment_of(first_s, a.B, k), page = a.pages[k];
    c.table[(size_t)slot_s[s] * c.max_pages + block_s[s] + (k - first_s[s])] = page;
    c.refs[page] = 1;
  }
}

__global__ void __launch_bounds__(COPY_THREADS) append_copy_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ int start_s[CACHE_MAX_SEQS];
  start_dependent();
  const CacheView &c = a.c;
  const int rows = *a.rows, in_page = (1 << c.page_shift) - 1;
  if (rows == 0) return;
  for (int b = threadIdx.x; b < a.B; b += COPY_THREADS) start_s[b] = a.seg[b].start;
  __syncthreads();
  const long long warps = (long long)gridDim.x * (COPY_THREADS / 32);
  const int jobs = (c.n_layers + a.per_job - 1) / a.per_job;  // of a row
  const size_t pool = ((size_t)c.n_pages << c.page_shift) * c.row;  // values of a layer
  for (long long job = (long long)blockIdx.x * (COPY_THREADS / 32) + (threadIdx.x >> 5);
       job < (long long)rows * jobs; job += warps) {
    const int group = (int)(job / rows), r = (int)(job - (long long)group * rows);
    const int layer = group * a.per_job, layers = min(a.per_job, c.n_layers - layer);
    const int b = segment_of(start_s, a.B, r);
    const AppendSeg g = a.seg[b];
    int i = r - g.start, at;
    const uint16_t *ks = a.k_new, *vs = a.v_new;
    size_t src, from = (size_t)a.n_rows * c.row;
    if (i < g.cow) {
      at = (g.len & ~in_page) + i;
      src = ((size_t)layer * c.n_pages + g.old_page) * (in_page + 1) + i;
      ks = c.k;
      vs = c.v;
      from = pool;
    } else {
      i -= g.cow;
      at = g.len + i;
      src = (size_t)layer * a.n_rows + g.src + (a.path ? a.path[(size_t)b * a.path_stride + i] : i);
    }
    const int page = c.table[(size_t)g.slot * c.max_pages + (at >> c.page_shift)];
    if ((unsigned)page >= (unsigned)c.n_pages) continue;
    const size_t dst = ((size_t)layer * c.n_pages + page) * (in_page + 1) + (at & in_page);
    copy_rows(c.k + dst * c.row, c.v + dst * c.row, ks + src * c.row, vs + src * c.row, c.row, layers, pool, from);
  }
}

// ------------------------------------------------------------------ fork

struct ForkSeg {
  int32_t start;   // its first row in the call's count of copied rows
  int32_t pstart;  // its first entry in the call's count of shared pages
  int32_t src, dst, old_page, new_page;
};

struct ForkArgs {
  CacheView c;
  const int32_t *src, *dst;
  int n;
  int32_t *rows;  // [2] rows to copy, pages to share; 0 if the call changes nothing
  ForkSeg *seg;   // [n]
  int32_t *pages;
  int per_job;    // layers a warp copies of a row
  float *ks, *vs; // scales [layers][pages][heads] that a copied page brings along, or null
  int heads;
};

template <int THREADS>
__global__ void __launch_bounds__(THREADS) fork_plan_kernel(const __grid_constant__ ForkArgs a) {
  __shared__ int red[33], src_s[THREADS], dst_s[THREADS], look_s[THREADS], full_s[THREADS], bad;
  start_dependent();
  const CacheView &c = a.c;
  const int i = threadIdx.x, in_page = (1 << c.page_shift) - 1;
  const bool in = i < a.n;
  if (i == 0) bad = 0;
  int src = 0, dst = 0, L = 0, old_page = -1;
  bool ok = true;
  if (in) {
    src_s[i] = src = a.src[i];
    dst_s[i] = dst = a.dst[i];
    ok = src >= 0 && src < c.n_slots && dst >= 0 && dst < c.n_slots;
    if (ok) {
      L = slot_len(c, src);
      ok = L >= 0 && c.lens[dst] == 0;
    }
  }
  __syncthreads();
  if (in && ok) {
    bool wrong = false;
#pragma unroll 8
    for (int j = 0; j < a.n; ++j) wrong |= src_s[j] == dst || (j < i && dst_s[j] == dst);
    ok = !wrong;
    if (ok && (L & in_page)) {
      old_page = table_page(c, src, L >> c.page_shift);
      ok = old_page >= 0;
    }
  }
  if (!ok) bad = 1;
  const int tail = in && ok ? L & in_page : 0, full = in && ok ? L >> c.page_shift : 0;
  // The entries to be shared have to name pages: nothing may change otherwise.  A
  // source's are looked at once for its forks in a row: the first 32 by one
  // warp, eight sources' loads at a time, the others by one warp or, of few
  // sources, by all.  (A search for each thread's entries in the sources' prefix sums
  // took 2.2 us of 48 for 24 sources of 25 pages; this takes 0.9.)
  int sources, both, shared;
  const bool looks = full && (i == 0 || src_s[i - 1] != src);
  const int nth = block_scan(looks ? 1 : 0, red, &sources);
  if (looks) {
    look_s[nth] = src;
    full_s[nth] = full;
  }
  __syncthreads();
  bool wrong = false;
  constexpr int WARPS = THREADS / 32, AHEAD = 8;
  const int lane = i & 31;
  auto entry = [&](int k, int j) { return (unsigned)c.table[(size_t)look_s[k] * c.max_pages + j]; };
#pragma unroll 1
  for (int k = i >> 5; k < sources; k += WARPS * AHEAD) {
    unsigned p[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      p[u] = k + u * WARPS < sources && lane < full_s[k + u * WARPS] ? entry(k + u * WARPS, lane) : 0;
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) wrong |= p[u] >= (unsigned)c.n_pages;
  }
  const bool few = sources < WARPS;
#pragma unroll 1
  for (int k = few ? 0 : i >> 5; k < sources; k += few ? 1 : WARPS)
#pragma unroll 4
    for (int j = 32 + (few ? i : lane); j < full_s[k]; j += few ? THREADS : 32)
      wrong |= entry(k, j) >= (unsigned)c.n_pages;
  if (wrong) bad = 1;
  // pages to allocate and rows to copy in one scan: up to 2^10 pages << 20 | 2^10 * 255 rows
  const int at = block_scan(tail ? 1 << 20 | tail : 0, red, &both);
  const int first = at >> 20, start = at & 0xFFFFF, total = both >> 20, rows = both & 0xFFFFF;
  const int pstart = block_scan(full, red, &shared);
  int code = bad ? MOE_ERR_DEVICE_BOUNDS : MOE_OK;  // bad: written before the scans' barriers
  if (!code && find_free(c, total, red, a.pages) < total) code = MOE_ERR_OUT_OF_PAGES;
  if (code) {
    if (i == 0) {
      set_status(c.status, code);
      a.rows[0] = a.rows[1] = 0;
    }
    return;
  }
  __syncthreads();
  if (in) {
    const int page = tail ? a.pages[first] : -1;
    a.seg[i] = ForkSeg{start, pstart, src, dst, old_page, page};
    if (tail) {
      c.table[(size_t)dst * c.max_pages + full] = page;
      c.refs[page] = 1;
    }
    c.lens[dst] = L;
  }
  if (i == 0) {
    a.rows[0] = rows;
    a.rows[1] = shared;
  }
}

__global__ void __launch_bounds__(COPY_THREADS) fork_copy_kernel(const __grid_constant__ ForkArgs a) {
  __shared__ int start_s[CACHE_MAX_SEQS], pstart_s[CACHE_MAX_SEQS];
  start_dependent();
  const CacheView &c = a.c;
  const int rows = a.rows[0], shared = a.rows[1];
  if (rows == 0 && shared == 0) return;
  for (int i = threadIdx.x; i < a.n; i += COPY_THREADS) {
    start_s[i] = a.seg[i].start;
    pstart_s[i] = a.seg[i].pstart;
  }
  __syncthreads();
  for (long long e = (long long)blockIdx.x * COPY_THREADS + threadIdx.x; e < shared;
       e += (long long)gridDim.x * COPY_THREADS) {
    const int s = segment_of(pstart_s, a.n, (int)e), j = (int)e - pstart_s[s];
    const int page = table_page(c, a.seg[s].src, j);
    c.table[(size_t)a.seg[s].dst * c.max_pages + j] = page;
    if (page >= 0) atomicAdd(&c.refs[page], 1);
  }
  if (a.ks)
    for (long long e = (long long)blockIdx.x * COPY_THREADS + threadIdx.x, each = (long long)c.n_layers * a.heads;
         e < a.n * each; e += (long long)gridDim.x * COPY_THREADS) {
      const ForkSeg g = a.seg[e / each];
      if (g.new_page < 0) continue;
      const int layer = (int)(e % each) / a.heads, head = (int)(e % each) % a.heads;
      const size_t base = (size_t)layer * c.n_pages;
      a.ks[(base + g.new_page) * a.heads + head] = a.ks[(base + g.old_page) * a.heads + head];
      a.vs[(base + g.new_page) * a.heads + head] = a.vs[(base + g.old_page) * a.heads + head];
    }
  const long long warps = (long long)gridDim.x * (COPY_THREADS / 32);
  const int jobs = (c.n_layers + a.per_job - 1) / a.per_job;  // of a row
  const size_t pool = ((size_t)c.n_pages << c.page_shift) * c.row;  // values of a layer
  for (long long job = (long long)blockIdx.x * (COPY_THREADS / 32) + (threadIdx.x >> 5);
       job < (long long)rows * jobs; job += warps) {
    const int group = (int)(job / rows), r = (int)(job - (long long)group * rows);
    const int layer = group * a.per_job, layers = min(a.per_job, c.n_layers - layer);
    const ForkSeg g = a.seg[segment_of(start_s, a.n, r)];
    const size_t base = (size_t)layer * c.n_pages, i = r - g.start;
    const size_t src = ((base + g.old_page) << c.page_shift) + i, dst = ((base + g.new_page) << c.page_shift) + i;
    copy_rows(c.k + dst * c.row, c.v + dst * c.row, c.k + src * c.row, c.v + src * c.row, c.row, layers, pool, pool);
  }
}

// ------------------------------------------------------------------ trim

// One CTA per sequence.  All of its pages are looked at before any leaves the
// table, so that a sequence with a bad entry, or a page that nobody holds, stays
// as it was.  A thread keeps the first four it looks at; those of more than 512
// are read again.
__global__ void __launch_bounds__(128) trim_kernel(const __grid_constant__ CacheView c, const int32_t *slots,
                                                   const int32_t *new_lens) {
  start_dependent();
  const int b = blockIdx.x, slot = slots ? slots[b] : b, want = new_lens[b];
  bool ok = slot >= 0 && slot < c.n_slots;
  const int L = ok ? slot_len(c, slot) : -1;
  ok = ok && want >= 0 && want <= L;
  if (ok && slots)  // a slot named twice: only the first counts
    for (int i = threadIdx.x; i < b; i += 128) ok = ok && slots[i] != slot;
  constexpr int KEPT = 4;
  int32_t *table = c.table + (size_t)(ok ? slot : 0) * c.max_pages;
  const int j0 = pages_of(want, c.page_shift) + threadIdx.x, j1 = ok ? pages_of(L, c.page_shift) : 0;
  auto held = [&](int page) { return (unsigned)page < (unsigned)c.n_pages && c.refs[page] > 0; };
  int page[KEPT];
#pragma unroll
  for (int u = 0; u < KEPT; ++u) page[u] = j0 + u * 128 < j1 ? table[j0 + u * 128] : 0;
#pragma unroll
  for (int u = 0; u < KEPT; ++u) ok = (j0 + u * 128 >= j1 || held(page[u])) && ok;
  for (int j = j0 + KEPT * 128; j < j1; j += 128) ok = held(table[j]) && ok;
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) set_status(c.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  auto release = [&](int j, int p) {
    table[j] = -1;
    if (atomicSub(&c.refs[p], 1) <= 0) {  // named by more tables of the call than it has holders
      atomicAdd(&c.refs[p], 1);
      set_status(c.status, MOE_ERR_DEVICE_BOUNDS);
    }
  };
#pragma unroll
  for (int u = 0; u < KEPT; ++u)
    if (j0 + u * 128 < j1) release(j0 + u * 128, page[u]);
  for (int j = j0 + KEPT * 128; j < j1; j += 128) release(j, table[j]);
  if (threadIdx.x == 0) c.lens[slot] = want;
}

}  // namespace

moe_status cache_view_any(const void *k, const void *v, int32_t *refs, int32_t *table, int32_t *lens, int32_t *status,
                          int n_layers, int n_pages, int page_size, int n_kv_heads, int head_dim, int n_slots,
                          int max_pages, int row_words, CacheView *out) {
  if (!k || !v || !refs || !table || !lens || !status || n_layers < 1 || n_pages < 1 || n_slots < 1 || max_pages < 1 ||
      n_kv_heads < 1 || page_size < 1)
    return MOE_ERR_INVALID_ARGUMENT;
  const int ps = page_size, D = head_dim;
  if ((ps & (ps - 1)) || ps < 16 || ps > 256 || (D != 64 && D != 128 && D != 256) || n_kv_heads > 256 ||
      (int64_t)n_pages * ps > INT32_MAX || (int64_t)max_pages * ps > (1 << 30))
    return MOE_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || !aligned16(refs) || !aligned16(table) || !aligned16(lens) || !aligned16(status))
    return MOE_ERR_MISALIGNED;
  out->k = static_cast<uint16_t *>(const_cast<void *>(k));
  out->v = static_cast<uint16_t *>(const_cast<void *>(v));
  out->refs = refs;
  out->table = table;
  out->lens = lens;
  out->status = status;
  out->n_layers = n_layers;
  out->n_pages = n_pages;
  out->page_shift = __builtin_ctz(ps);
  out->row = row_words;
  out->n_slots = n_slots;
  out->max_pages = max_pages;
  return MOE_OK;
}

moe_status cache_view(const attn_cache *c, CacheView *out) {
  if (!c) return MOE_ERR_INVALID_ARGUMENT;
  const moe_status st =
      cache_view_any(c->k_d, c->v_d, c->refs_d, c->table_d, c->lens_d, c->status_d, c->n_layers, c->n_pages,
                     c->page_size, c->n_kv_heads, c->head_dim, c->n_slots, c->max_pages,
                     c->n_kv_heads * c->head_dim, out);
  if (st == MOE_ERR_INVALID_ARGUMENT) return st;
  return c->dtype != MOE_BF16 && c->dtype != MOE_FP16 ? MOE_ERR_UNSUPPORTED : st;
}

// Workspaces: a header of 64 bytes, the segments, the pages found.
size_t append_ws(int page_size, int B, int n_rows, size_t *pages_at) {
  *pages_at = 64 + (size_t)B * sizeof(AppendSeg);
  return *pages_at + ((size_t)n_rows / page_size + 2 * (size_t)B) * 4;
}

moe_status append_args(const CacheView &c, const AppendCall &call, int new_words, AppendArgs *a) {
  if (call.B < 0 || call.n_rows < 0 || (call.path && (!call.n_keep || call.path_stride < 1)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (call.B > CACHE_MAX_SEQS) return MOE_ERR_UNSUPPORTED;
  a->B = call.B;
  if (call.B == 0) return MOE_OK;
  if (!call.offsets || !call.ws || (call.n_rows > 0 && (!call.k_new || !call.v_new))) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned16(call.k_new) || !aligned16(call.v_new) || !aligned16(call.slots) || !aligned16(call.offsets) ||
      !aligned16(call.n_keep) || !aligned16(call.path) || !aligned16(call.ws))
    return MOE_ERR_MISALIGNED;
  const size_t nn = (size_t)c.n_layers * call.n_rows * new_words * 2;
  const size_t np = ((size_t)c.n_layers * c.n_pages << c.page_shift) * c.row * 2;
  if (ranges_meet(call.k_new, nn, c.k, np) || ranges_meet(call.k_new, nn, c.v, np) ||
      ranges_meet(call.v_new, nn, c.k, np) || ranges_meet(call.v_new, nn, c.v, np))
    return MOE_ERR_INVALID_ARGUMENT;
  size_t pages_at;
  if (call.ws_bytes < append_ws(1 << c.page_shift, call.B, call.n_rows, &pages_at)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  a->c = c;
  a->k_new = static_cast<const uint16_t *>(call.k_new);
  a->v_new = static_cast<const uint16_t *>(call.v_new);
  a->slots = call.slots;
  a->offsets = call.offsets;
  a->n_keep = call.n_keep;
  a->path = call.path;
  a->path_stride = call.path_stride;
  a->n_rows = call.n_rows;
  a->rows = static_cast<int32_t *>(call.ws);
  a->seg = ws_ptr<AppendSeg>(call.ws, 64);
  a->pages = ws_ptr<int32_t>(call.ws, pages_at);
  a->per_job = layers_per_job(call.n_rows, c.n_layers);
  return MOE_OK;
}

cudaError_t launch_append_plan(const AppendArgs &a, cudaStream_t s) {
  const bool chain = prof_chain(0);
  return a.B <= PLAN_FEW ? launch_dep(chain, append_plan_kernel<PLAN_FEW>, dim3(1), dim3(PLAN_FEW), 0, s, a)
                         : launch_dep(chain, append_plan_kernel<PLAN_MANY>, dim3(1), dim3(PLAN_MANY), 0, s, a);
}

}  // namespace moe

extern "C" size_t attn_cache_append_workspace_bytes(const attn_cache *c, int32_t B, int32_t n_rows) {
  moe::CacheView v;
  if (moe::cache_view(c, &v) != MOE_OK || B < 1 || B > moe::CACHE_MAX_SEQS || n_rows < 0) return 0;
  size_t at;
  return moe::append_ws(c->page_size, B, n_rows, &at);
}

extern "C" moe_status attn_cache_append(const attn_cache *c, const void *k_new_d, const void *v_new_d,
                                        const int32_t *slots_d, const int32_t *offsets_d, const int32_t *n_keep_d,
                                        const int32_t *path_d, int32_t path_stride, int32_t B, int32_t n_rows,
                                        void *ws_d, size_t ws_bytes, void *stream) {
  moe::CacheView v;
  moe::AppendArgs a;
  moe_status st = moe::cache_view(c, &v);
  if (st != MOE_OK) return st;
  st = moe::append_args(v, moe::AppendCall{k_new_d, v_new_d, slots_d, offsets_d, n_keep_d, path_d, path_stride, B, n_rows,
                                           ws_d, ws_bytes}, v.row, &a);
  if (st != MOE_OK || a.B == 0) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = moe::launch_append_plan(a, s);
  if (e != cudaSuccess) return moe::note_cuda_error(e);
  const bool pdl = moe::prof_quiet(MOE_KERNEL_CACHE_COPY);
  moe::prof_before(MOE_KERNEL_CACHE_COPY, s);
  // Rows of a copied page come on top of the kept ones; the grid, which does not
  // count them (only the device knows them), strides over all.
  e = moe::launch_dep(pdl, moe::append_copy_kernel, dim3(moe::copy_grid(n_rows + B, c->n_layers, a.per_job)),
                      dim3(moe::COPY_THREADS), 0, s, a);
  moe::prof_after(MOE_KERNEL_CACHE_COPY, s);
  return moe::note_cuda_error(e);
}

namespace moe {

size_t fork_ws(int n) { return n < 1 || n > CACHE_MAX_SEQS ? 0 : 64 + (size_t)n * (sizeof(ForkSeg) + 4); }

moe_status fork_call(const CacheView &c, const int32_t *src, const int32_t *dst, int n, void *ws, size_t ws_bytes,
                     float *ks, float *vs, int heads, cudaStream_t s) {
  if (n < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (n > CACHE_MAX_SEQS) return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!src || !dst || !ws) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned16(src) || !aligned16(dst) || !aligned16(ws)) return MOE_ERR_MISALIGNED;
  if (ws_bytes < fork_ws(n)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  ForkArgs a;
  a.c = c;
  a.src = src;
  a.dst = dst;
  a.n = n;
  a.rows = static_cast<int32_t *>(ws);
  a.seg = ws_ptr<ForkSeg>(ws, 64);
  a.pages = ws_ptr<int32_t>(ws, 64 + (size_t)n * sizeof(ForkSeg));
  a.ks = ks;
  a.vs = vs;
  a.heads = heads;
  const long long rows = (long long)n << c.page_shift >> 1;  // half a page a fork on average
  a.per_job = layers_per_job(rows, c.n_layers);
  const bool chain = prof_chain(0);
  cudaError_t e = n <= PLAN_FEW
                      ? launch_dep(chain, fork_plan_kernel<PLAN_FEW>, dim3(1), dim3(PLAN_FEW), 0, s, a)
                      : launch_dep(chain, fork_plan_kernel<PLAN_MANY>, dim3(1), dim3(PLAN_MANY), 0, s, a);
  if (e != cudaSuccess) return note_cuda_error(e);
  const bool pdl = prof_quiet(MOE_KERNEL_CACHE_COPY);
  prof_before(MOE_KERNEL_CACHE_COPY, s);
  e = launch_dep(pdl, fork_copy_kernel, dim3(copy_grid(rows, c.n_layers, a.per_job)), dim3(COPY_THREADS), 0, s, a);
  prof_after(MOE_KERNEL_CACHE_COPY, s);
  return note_cuda_error(e);
}

moe_status trim_call(const CacheView &c, const int32_t *slots, const int32_t *new_lens, int n, cudaStream_t s) {
  if (n < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (n > CACHE_MAX_SEQS) return MOE_ERR_UNSUPPORTED;
  if (n == 0) return MOE_OK;
  if (!new_lens) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned16(slots) || !aligned16(new_lens)) return MOE_ERR_MISALIGNED;
  return note_cuda_error(launch_dep(prof_chain(0), trim_kernel, dim3(n), dim3(128), 0, s, c, slots, new_lens));
}

}  // namespace moe

extern "C" size_t attn_cache_fork_workspace_bytes(const attn_cache *c, int32_t n) {
  moe::CacheView v;
  return moe::cache_view(c, &v) == MOE_OK ? moe::fork_ws(n) : 0;
}

extern "C" moe_status attn_cache_fork(const attn_cache *c, const int32_t *src_d, const int32_t *dst_d, int32_t n,
                                      void *ws_d, size_t ws_bytes, void *stream) {
  moe::CacheView v;
  const moe_status st = moe::cache_view(c, &v);
  return st != MOE_OK ? st
                      : moe::fork_call(v, src_d, dst_d, n, ws_d, ws_bytes, nullptr, nullptr, 0,
                                       static_cast<cudaStream_t>(stream));
}

extern "C" moe_status attn_cache_trim(const attn_cache *c, const int32_t *slots_d, const int32_t *new_lens_d,
                                      int32_t n, void *stream) {
  moe::CacheView v;
  const moe_status st = moe::cache_view(c, &v);
  return st != MOE_OK ? st : moe::trim_call(v, slots_d, new_lens_d, n, static_cast<cudaStream_t>(stream));
}
