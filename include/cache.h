/* cache.h -- C ABI of the paged KV cache in libmoe.so (sm_103a).
 *
 * A page holds the K and V rows of page_size consecutive positions of one
 * sequence, position-major as attn_decode's cache (attn.h): a contiguous cache
 * [L][Hkv][D] is a pool of ceil(L / page_size) pages with an identity table.
 * One page table serves every attention layer.  All bookkeeping lives on the
 * device: a sequence's pages and length change inside the stream, after
 * kernels whose results decide by how much, with no host synchronisation.
 *
 *   holders   refs_d[page] = sequences whose table names the page; 0 = free
 *   allocate  always the lowest free pages, in the order of the call's
 *             sequences, so the same calls give the same tables
 *
 * Conventions as in moe.h, and: device-side data (slots, offsets, lengths,
 * table entries) is checked on the device.  A check that fails sets the
 * cache's status word (MOE_ERR_DEVICE_BOUNDS, or MOE_ERR_OUT_OF_PAGES; the
 * first error stays until the caller zeroes it) and the call it belongs to
 * changes nothing: attn_cache_append and attn_cache_fork take all of their
 * sequences or none, attn_cache_trim each sequence by itself.
 * Calls on one cache must not overlap (one stream, or ordered by events).  A
 * workspace overlaps nothing else.
 */
#ifndef CACHE_H
#define CACHE_H
#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_BF16 = 0, MOE_FP16 = 1 };  /* attn_cache.dtype */

/* Host struct of device pointers; the caller owns every buffer.
 * Supported: page_size 16, 32, 64, 128 or 256, head_dim 64, 128 or 256,
 * 1 <= n_kv_heads <= 256, n_pages * page_size < 2^31, max_pages * page_size
 * <= 2^30.  To start: refs_d, lens_d and status_d zero, table_d -1. */
typedef struct attn_cache {
  void *k_d, *v_d;     /* [n_layers][n_pages][page_size][n_kv_heads][head_dim], bf16 or fp16 */
  int32_t *refs_d;     /* [n_pages]              holders of a page, 0 = free         */
  int32_t *table_d;    /* [n_slots][max_pages]   page of position block j, -1 = none */
  int32_t *lens_d;     /* [n_slots]              cached positions                    */
  int32_t *status_d;   /* [1]                    sticky device status                */
  int32_t n_layers, n_pages, page_size, n_kv_heads, head_dim;
  int32_t n_slots;     /* sequences the tables have room for */
  int32_t max_pages;   /* pages a sequence may have          */
  int32_t dtype;       /* MOE_BF16 or MOE_FP16               */
} attn_cache;

/* Append rows of K and V, of all layers, to B sequences.
 *   k_new_d, v_new_d  [n_layers][n_rows][n_kv_heads][head_dim] (read)
 *   slots_d           int32 [B] sequences, distinct, or NULL: 0 .. B-1
 *   offsets_d         int32 [B+1]: sequence b's rows are offsets[b] .. offsets[b+1]-1
 *   n_keep_d          int32 [B] rows kept, or NULL: all of them (then path_d must be NULL)
 *   path_d            int32 [B][path_stride] or NULL: the i-th kept row of
 *                     sequence b is its row path[b][i] (NULL: its row i).  The
 *                     accepted path and its length from moe_draft_verify fit as they are.
 *   ws_d              workspace of attn_cache_append_workspace_bytes(c, B, n_rows), scratch
 * A kept row goes to the sequence's next position; pages are allocated as
 * needed.  A last page that is partly filled and has other holders is copied
 * to a page of the sequence's own first.  B <= 1024; B == 0 returns MOE_OK
 * with nothing enqueued.
 * Device checks: slots in range and distinct, offsets ascending within
 * n_rows, kept rows within the sequence's rows, room in its table.
 * Errors: MOE_ERR_INVALID_ARGUMENT (null pointers, negative sizes, path_d
 * without n_keep_d, path_stride < 1 with path_d, rows that lie in the pool),
 * MOE_ERR_UNSUPPORTED (the cache's
 * dimensions, B > 1024), MOE_ERR_MISALIGNED, MOE_ERR_WORKSPACE_TOO_SMALL,
 * MOE_ERR_CUDA. */
size_t attn_cache_append_workspace_bytes(const attn_cache *c, int32_t B, int32_t n_rows);
moe_status attn_cache_append(const attn_cache *c, const void *k_new_d, const void *v_new_d, const int32_t *slots_d,
                             const int32_t *offsets_d, const int32_t *n_keep_d, const int32_t *path_d,
                             int32_t path_stride, int32_t B, int32_t n_rows, void *ws_d, size_t ws_bytes,
                             void *stream);

/* Fork n sequences: slot dst[i], empty before, becomes a copy of slot src[i].
 * Full pages are shared (one more holder); a partly filled last page is
 * copied, in all layers, to a page of dst's own.  A src may be named many
 * times; a dst is named once and is no src of the call.  n <= 1024; n == 0
 * returns MOE_OK with nothing enqueued.
 *   src_d, dst_d  int32 [n];  ws_d  attn_cache_fork_workspace_bytes(c, n), scratch
 * Device checks: slots in range, each dst empty, named once and no src, every
 * position block of a src's length in its table.  Errors as for attn_cache_append. */
size_t attn_cache_fork_workspace_bytes(const attn_cache *c, int32_t n);
moe_status attn_cache_fork(const attn_cache *c, const int32_t *src_d, const int32_t *dst_d, int32_t n, void *ws_d,
                           size_t ws_bytes, void *stream);

/* Cut n sequences to new lengths (0 frees a sequence).  Pages wholly behind
 * the new length lose a holder and leave the table.
 *   slots_d     int32 [n], distinct, or NULL: 0 .. n-1
 *   new_lens_d  int32 [n], 0 <= new <= the sequence's length
 * n <= 1024; n == 0 returns MOE_OK with nothing enqueued.  Device checks per
 * sequence: the slot in range (of one named twice the first counts), the new
 * length, and every page to be given up in the table and with a holder.  One
 * that fails is left as it was.  (Holders that are too few for several
 * sequences of one call may be found when these are cut already: the status
 * word is set, the count stays 0.) */
moe_status attn_cache_trim(const attn_cache *c, const int32_t *slots_d, const int32_t *new_lens_d, int32_t n,
                           void *stream);

#ifdef __cplusplus
}
#endif
#endif
