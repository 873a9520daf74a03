/* qcache.h -- C ABI of the 8-bit paged KV cache in libmoe.so (sm_103a), and of
 * attention over it.
 *
 * Pages, tables, holders and checks are those of cache.h; a page's K and V
 * are e4m3 codes, with a scale for each layer, page and KV head:
 *   value = code * scale
 * Appending makes scales that are powers of two: 2^e, e the least whole number
 * from -100 on with |x| <= 448 * 2^e for every finite value the page has taken
 * since its first row.  A scale only grows (cutting rows off leaves it) until the
 * page is begun anew.  Where it grows, the page's earlier codes are rounded to it:
 * exact but for values below 2^-6 of the new scale, whose last bits go.  So a
 * value is off by 2^-4 of itself or half of 2^-9 scales at most, and by one
 * more such half for each time its page's scale grew.  Values that are not
 * finite become the code NaN.  Attention takes any finite scales that are not negative.
 */
#ifndef QCACHE_H
#define QCACHE_H
#include "rotary.h"

#ifdef __cplusplus
extern "C" {
#endif

/* As attn_cache (the same sizes are supported, the same start). */
typedef struct attn_qcache {
  void *k_d, *v_d;              /* e4m3 [n_layers][n_pages][page_size][n_kv_heads][head_dim] */
  float *k_scale_d, *v_scale_d; /* fp32 [n_layers][n_pages][n_kv_heads] */
  int32_t *refs_d;              /* [n_pages] */
  int32_t *table_d;             /* [n_slots][max_pages] */
  int32_t *lens_d;              /* [n_slots] */
  int32_t *status_d;            /* [1] */
  int32_t n_layers, n_pages, page_size, n_kv_heads, head_dim;
  int32_t n_slots, max_pages;
  int32_t reserved;
} attn_qcache;

/* attn_cache_append into the 8-bit cache.
 *   table    K rows are turned by the position they are stored at; NULL: not
 *   dtype    MOE_BF16 or MOE_FP16, of k_new_d and v_new_d (layouts as there)
 * The other arguments, checks and errors are those of attn_cache_append. */
size_t attn_qcache_append_workspace_bytes(const attn_qcache *c, int32_t B, int32_t n_rows);
moe_status attn_qcache_append(const attn_qcache *c, const attn_rotary_table *table, const void *k_new_d,
                              const void *v_new_d, int32_t dtype, const int32_t *slots_d, const int32_t *offsets_d,
                              const int32_t *n_keep_d, const int32_t *path_d, int32_t path_stride, int32_t B,
                              int32_t n_rows, void *ws_d, size_t ws_bytes, void *stream);

/* attn_cache_fork and attn_cache_trim: a copied page brings its scales. */
size_t attn_qcache_fork_workspace_bytes(const attn_qcache *c, int32_t n);
moe_status attn_qcache_fork(const attn_qcache *c, const int32_t *src_d, const int32_t *dst_d, int32_t n, void *ws_d,
                            size_t ws_bytes, void *stream);
moe_status attn_qcache_trim(const attn_qcache *c, const int32_t *slots_d, const int32_t *new_lens_d, int32_t n,
                            void *stream);

/* Attention of the last rows of B sequences, one layer.  Row i of a sequence's
 * n rows is its token at position len - n + i (appended before, with len the
 * cache's length):
 *   o[i,h] = sum_l softmax_l(s) V[l,g],  s_l = scale * (q[i,h] . K[l,g]),  g = h / (Hq / Hkv)
 * over l = 0 .. len - n + i.  A row before position 0 (more rows than the
 * cache holds: padding in front) sees nothing and gets zeros.
 *   layer      the cache's layer
 *   q_d        bf16 or fp16 (dtype) [n_rows][Hq][head_dim] (read)
 *   slots_d    int32 [B] sequences, or NULL: 0 .. B-1 (one may be named twice)
 *   offsets_d  int32 [B+1]: sequence b's rows are offsets[b] .. offsets[b+1]-1
 *   max_rows   upper bound of a sequence's rows, >= 1
 *   scale      0 means 1 / sqrt(head_dim)
 *   ws_d       workspace of attn_qcache_attend_workspace_bytes(c, B, n_rows, max_rows, Hq), scratch
 *   o_d        [n_rows][Hq][head_dim], q's type (written; rows of no sequence are left as they are)
 * Arithmetic: the codes are tensor-core operands as they are, q and the softmax
 * weights times V's scales sums of 8-bit parts that keep all bits of q but for those below 2^-18 of
 * its row's largest value, and 2^-10 of a weight or 2^-23 of the largest product of a weight and its V
 * scale that the row sees; fp32 sums, o rounded once.  Weights below 2^-110 of the row's
 * largest may count as none, and values above 2^80 may pass the range of the sums.
 * What a row does not see cannot change it, codes and scales whatever their bits; a NaN
 * among its scores, or among the values it sees, makes it NaN.  Supported: Hq a multiple of
 * n_kv_heads, at most 128 query heads per KV head, B <= 1024, n_rows * Hq < 2^30.
 * B == 0 or n_rows == 0 returns MOE_OK with nothing enqueued.  Device checks
 * (slots, offsets, lengths, pages) set MOE_ERR_DEVICE_BOUNDS in the cache's status
 * word; the output of that sequence is then not valid.  MOE_ERR_DEVICE_TIMEOUT
 * there: a wait for a copy gave up.  o_d overlaps no input, ws_d nothing else.
 * Errors: MOE_ERR_INVALID_ARGUMENT, MOE_ERR_UNSUPPORTED, MOE_ERR_MISALIGNED,
 * MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA. */
size_t attn_qcache_attend_workspace_bytes(const attn_qcache *c, int32_t B, int32_t n_rows, int32_t max_rows,
                                          int32_t Hq);
moe_status attn_qcache_attend(const attn_qcache *c, int32_t layer, const void *q_d, int32_t dtype,
                              const int32_t *slots_d, const int32_t *offsets_d, int32_t B, int32_t n_rows,
                              int32_t max_rows, int32_t Hq, float scale, void *ws_d, size_t ws_bytes, void *o_d,
                              void *stream);

#ifdef __cplusplus
}
#endif
#endif
