/* tree.h -- C ABI of attention for drafted tokens over a paged cache, and of
 * the drafts' verification, in libmoe.so (sm_103a).
 *
 * Speculative decoding: a draft proposes a tree of next tokens, the target
 * model evaluates the whole tree in one pass, and the drafts are accepted so
 * that the tokens follow the target's distribution ("Fast Inference from
 * Transformers via Speculative Decoding", Leviathan, Kalman and Matias, 2023;
 * for trees with several tries a node "SpecInfer", Miao et al., 2024).
 *
 * A tree is a range of nodes, offsets[b] .. offsets[b+1]-1 for sequence b, in
 * an order in which parents come first: parent[i] < i counted within the
 * tree, -1 for a root, -2 for a node that is padding (and has no children).  One node per sequence
 * is ordinary decoding, a chain the usual list of drafted tokens.
 */
#ifndef TREE_H
#define TREE_H
#include "cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Attention of B trees over the cache, one layer:
 *   o[i,h] = sum_l softmax_l(s) v[l,g],  s_l = scale * (q[i,h] . k[l,g]),  g = h / (Hq / Hkv)
 * over the cached positions of the node's sequence, the node's ancestors and
 * the node itself.  A row with nothing to see (padding) gets zeros.  The
 * cache is only read: the tree's K and V rows come from k_new_d and v_new_d,
 * and attn_cache_append stores those that are accepted.
 *   layer       the cache's layer
 *   q_d         [n_nodes][Hq][head_dim], the cache's type (read)
 *   k_new_d, v_new_d  [n_nodes][n_kv_heads][head_dim] (read)
 *   slots_d     int32 [B] sequences, or NULL: 0 .. B-1 (one may be named twice)
 *   offsets_d   int32 [B+1] node ranges;  parent_d  int32 [n_nodes]
 *   max_nodes   upper bound of a tree's nodes, 1 .. 256
 *   scale       0 means 1 / sqrt(head_dim)
 *   ws_d        workspace of attn_tree_workspace_bytes(c, B, n_nodes, max_nodes, Hq), scratch
 *   o_d         [n_nodes][Hq][head_dim] (written; rows of no tree are left as they are)
 * Arithmetic: scores and softmax in fp32, the weights rounded to the cache's
 * type for the product with V (fp32 sums), o rounded once.  What a row does
 * not see cannot change it, whatever its bits (rows behind a length, other
 * branches, padding); a NaN among its scores makes it NaN.  Supported: Hq a multiple of n_kv_heads, at most 128
 * query heads per KV head, B <= 1024.  B == 0 or n_nodes == 0 returns MOE_OK
 * with nothing enqueued.  Device checks (slots, offsets, parents, lengths,
 * pages) set MOE_ERR_DEVICE_BOUNDS in the cache's status word; the output of
 * that tree is then not valid.  MOE_ERR_DEVICE_TIMEOUT there: a wait for a
 * copy gave up.  o_d overlaps no input, ws_d nothing else.
 * Errors: MOE_ERR_INVALID_ARGUMENT, MOE_ERR_UNSUPPORTED, MOE_ERR_MISALIGNED,
 * MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_CUDA. */
size_t attn_tree_workspace_bytes(const attn_cache *c, int32_t B, int32_t n_nodes, int32_t max_nodes, int32_t Hq);
moe_status attn_tree(const attn_cache *c, int32_t layer, const void *q_d, const void *k_new_d, const void *v_new_d,
                     const int32_t *slots_d, const int32_t *offsets_d, const int32_t *parent_d, int32_t B,
                     int32_t n_nodes, int32_t max_nodes, int32_t Hq, float scale, void *ws_d, size_t ws_bytes,
                     void *o_d, void *stream);

/* Verification of B drafted trees.  From node 0 (a root, the last sampled
 * token), over the children of the current node c in index order: with
 * R = p[c] and S = 1 at first, child j with token x is taken if
 *   u_accept[j] * S * q[c][x] < R[x],
 * else  R <- max(R - S q[c], 0),  S <- sum R.  A taken child becomes c.  When no
 * child is left the next token is the lowest t with
 *   R[0] + .. + R[t] > u_sample[b] * sum R
 * (from p[c] where R is zero everywhere).  q_d NULL: the drafts are not
 * sampled (looked up, or the draft's likeliest): q[c][x] = 1, and a child not
 * taken leaves R[x] <- 0, S <- S - R[x].  Tests and sums carry 40 bits or more, so
 * the tokens are those of 64-bit arithmetic but for ties closer than that.
 *   p_d          fp32 [n_nodes][V] target distribution after each node (read)
 *   q_d          fp32 [n_nodes][V] draft distribution the node's children were drawn from, or NULL
 *   tokens_d     int32 [n_nodes];  parent_d int32 [n_nodes];  offsets_d int32 [B+1]
 *   u_accept_d   fp32 [n_nodes], u_sample_d fp32 [B], in [0, 1)
 *   path_d       int32 [B][path_stride] (written): the nodes on the accepted path from
 *                node 0, then -1.  path_stride bounds a tree's nodes, 1 .. 1024.
 *   n_path_d     int32 [B] (written) nodes on the path, >= 1 (0 for a tree with no nodes)
 *   next_d       int32 [B] (written) the next token (-1 for a tree with no nodes)
 *   status_d     int32, set to MOE_ERR_DEVICE_BOUNDS (offsets, parents, a token outside
 *                [0, V)) or MOE_ERR_NONFINITE (the mass to draw from is not finite and positive:
 *                NaN or infinity left in R or, of a child not taken, in R[x]; or p[c] zero everywhere);
 *                that tree then has n_path 0 and next -1
 * The written arrays overlap nothing else.
 * Supported: 1 <= V <= 2^20, B <= 65535.  B == 0 returns MOE_OK with nothing enqueued.
 * Errors: MOE_ERR_INVALID_ARGUMENT, MOE_ERR_UNSUPPORTED, MOE_ERR_MISALIGNED, MOE_ERR_CUDA. */
moe_status moe_draft_verify(const float *p_d, const float *q_d, const int32_t *tokens_d, const int32_t *parent_d,
                            const int32_t *offsets_d, const float *u_accept_d, const float *u_sample_d, int32_t B,
                            int32_t n_nodes, int32_t V, int32_t *path_d, int32_t path_stride, int32_t *n_path_d,
                            int32_t *next_d, int32_t *status_d, void *stream);

#ifdef __cplusplus
}
#endif
#endif
