/* rotary.h -- C ABI of rotary positions in libmoe.so (sm_103a): rows of query
 * or key heads turned by their positions, and appending to the paged cache
 * (cache.h) with the new K rows turned on the way.
 *
 * The first `dim` values of a head are dim / 2 pairs, (x[i], x[i + dim/2]) or,
 * interleaved, (x[2i], x[2i+1]).  At position p pair i becomes
 *   (x cos a - y sin a, x sin a + y cos a) * factor,   a = p w[i];
 * the head's other values stay as they are ("RoFormer: Enhanced Transformer
 * with Rotary Position Embedding", Su et al., 2021).
 *
 * Long contexts: w[i] = f (g + (1 - g) / stretch), f = base^(-2i/dim),
 * g = clamp((t - low_turns) / (high_turns - low_turns), 0, 1) with the turns
 * t = original_len f / (2 pi) that the pair makes over the length the model
 * was trained on: pairs that turn often keep their rate, those that turn seldom
 * are slowed ("YaRN: Efficient Context Window Extension of Large Language
 * Models", Peng et al., 2023, section 3.2).  high_turns 0: g = 0, every pair slowed.
 *
 * Arithmetic: a rate is held as the fraction of a turn in 64-bit fixed point, so
 * that position times rate, taken modulo one turn by its overflow, is off by
 * 2^-50 of itself or |p| * 2^-64 turns whatever the position.  What is left beyond the nearest
 * quarter turn keeps 2^-23 of itself in fp32, so that the sines of small angles keep their
 * bits; cos, sin and the products in fp32, rounded once.  A negative position turns backwards, which is also
 * the gradient's way through a rotation.
 *
 * Conventions as in moe.h.
 */
#ifndef ROTARY_H
#define ROTARY_H
#include "cache.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct attn_rotary_config {
  int32_t dim;          /* values of a head that are turned: a multiple of 16, 16 .. 256 */
  int32_t interleaved;  /* pairs: 0 (i, i + dim/2), 1 (2i, 2i + 1) */
  double base;          /* > 0 */
  double stretch;       /* > 0; 1: rates as they are */
  double low_turns, high_turns;  /* 0 <= low < high, or both 0 */
  double original_len;  /* positions; read with high_turns > 0, > 0 then */
  float factor;         /* of cos and sin, finite; usually 1 */
} attn_rotary_config;

/* The rates, on the host; made once, read by every call that turns rows. */
typedef struct attn_rotary_table {
  uint64_t turns[128];  /* of pair i: turns a position, modulo 1, times 2^64 */
  int32_t dim, interleaved;
  float factor;
  int32_t reserved;
} attn_rotary_table;

/* Fill a table (host memory, no GPU needed).  Errors: MOE_ERR_INVALID_ARGUMENT
 * (null pointers, values that are not finite or out of the ranges above),
 * MOE_ERR_UNSUPPORTED (dim). */
moe_status attn_rotary_plan(const attn_rotary_config *cfg, attn_rotary_table *table);

/* Turn n_rows rows of n_heads heads.
 *   x_d          bf16 or fp16 (dtype), row r's heads at x_d + r * x_stride, one after another (read)
 *   positions_d  int32 [n_rows], any value (read)
 *   o_d          the same type, rows o_stride apart (written; nothing between the rows is)
 * o_d may be x_d with the same stride (in place); else the two address ranges, from
 * the first row's first value to the last row's last, lie apart.
 * Strides in values, multiples of 8, at least n_heads * head_dim; head_dim 64,
 * 128 or 256, not below the table's dim; n_heads 1 .. 65536.  n_rows == 0 returns
 * MOE_OK with nothing enqueued.
 * Errors: MOE_ERR_INVALID_ARGUMENT, MOE_ERR_UNSUPPORTED, MOE_ERR_MISALIGNED, MOE_ERR_CUDA. */
moe_status attn_rotary(const attn_rotary_table *table, const void *x_d, int64_t x_stride, int32_t dtype,
                       const int32_t *positions_d, int32_t n_rows, int32_t n_heads, int32_t head_dim, void *o_d,
                       int64_t o_stride, void *stream);

/* attn_cache_append (cache.h) with every kept K row turned by the position it
 * is stored at.  V rows, and rows of a page that is copied, are not turned.
 * Workspace, checks and errors as there; the table's dim is at most head_dim. */
moe_status attn_cache_append_rotary(const attn_cache *c, const attn_rotary_table *table, const void *k_new_d,
                                    const void *v_new_d, const int32_t *slots_d, const int32_t *offsets_d,
                                    const int32_t *n_keep_d, const int32_t *path_d, int32_t path_stride, int32_t B,
                                    int32_t n_rows, void *ws_d, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif
