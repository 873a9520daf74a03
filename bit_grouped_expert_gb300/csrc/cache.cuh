// Device view of a paged KV cache (cache.h) and the checks every kernel that
// reads its tables makes: slots, lengths and page numbers are device data.
#pragma once
#include "cache.h"
#include "common.cuh"

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

// Host: the view of a cache, after its dimensions and pointers are checked.
moe_status cache_view(const attn_cache *c, CacheView *out);

}  // namespace moe
