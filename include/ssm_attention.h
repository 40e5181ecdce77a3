/*
 * ssm_attention.h -- the attention blocks of a decoder that mixes them with Mamba2
 * blocks, where such a decoder verifies a draft tree: every node over the sequence's
 * cache and its own ancestors, and the commit of the accepted path into the cache.
 *
 * The cache is paged: k_pages and v_pages are [n_pages][Hkv][page_size][D] (bf16) for
 * one layer; page_table[s][i] is the page of sequence s's rows i*page_size ..; a
 * sequence has cache_len[s] rows (it may have none).  Hq query heads, Hkv key/value
 * heads, query head j reads key/value head j / (Hq / Hkv).
 *
 * Same conventions as ssm_tree.h.  A sequence whose cache_len is negative, above
 * max_cache_len or beyond its page table, or one of whose pages is out of range, sets
 * SSM_STATUS_SEQ_RANGE: the rows that cannot be read count as absent (ssm_tree_attention)
 * or are not written (ssm_kv_commit).
 *
 * The cache may be held in 8 bits (the calls that end in _fp8): e4m3 values, and for each block
 * of `block` tokens of a page and head a scale; a row stands for scale * value.  Rotary
 * positions are given to q and k before any of these calls (ssm_rope, ssm_tree_rope).
 */
#ifndef SSM_ATTENTION_H_
#define SSM_ATTENTION_H_

#include <stddef.h>
#include <stdint.h>

#include "ssm_prompt.h"
#include "ssm_tree.h"

#define SSM_STATUS_SCALE 128 /* a scale of an 8-bit cache outside 2^-100 .. 2^120 */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ssm_tree_attention -- for node v of sequence s and query head j
 *     o = sum_r softmax_r(scale q.k_r) v_r
 * over the rows r of the cache and the K/V rows of v's ancestors and of v itself.  A node
 * is not influenced by the other nodes' rows, whatever they hold.  n_nodes = 1 is the
 * single-token form.
 *   n_nodes     1 .. SSM_MAX_NODES; layout device ssm_node [S][n] (ssm_tree_layout_build; only
 *               `parent` is read; a parent that is not an earlier node makes its node a root and
 *               sets SSM_STATUS_BAD_LAYOUT)
 *   Hq, Hkv     Hkv divides Hq; D 64 or 128
 *   q           device bf16 [S*n][ldq]: Hq*D columns (row s*n + v)
 *   k, v        device bf16 [S*n][ldk], [S*n][ldv]: Hkv*D columns, the nodes' own rows
 *               (q, k, v may be columns of one projection's output)
 *   k_pages, v_pages, page_table  device; page_size a power of two, 8 .. 1024; max_pages = row length
 *               of page_table
 *   cache_len   device int32 [S];  max_cache_len: host bound on them
 *   o           device bf16 [S*n][ldo]: Hq*D columns
 *   workspace   device, 256-byte aligned, >= ssm_tree_attention_workspace_size() bytes
 * Pointers 16-byte aligned, row strides multiples of 8.  Scores, maxima, sums and o are accumulated in fp32;
 * the weights exp(score - maximum) are rounded to bf16 for their product with v (relative error of o 0.0017 to
 * 0.0023, of which its own rounding 0.0017).
 */
int ssm_tree_attention(int32_t n_seq, int32_t n_nodes, int32_t Hq, int32_t Hkv, int32_t D, const ssm_node *layout,
                       const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv,
                       const uint16_t *k_pages, const uint16_t *v_pages, int32_t n_pages, int32_t page_size,
                       const int32_t *page_table, int32_t max_pages, const int32_t *cache_len, int32_t max_cache_len,
                       float scale, uint16_t *o, int64_t ldo, void *workspace, size_t workspace_bytes,
                       int32_t *dev_status, void *stream);

/* Host-only.  Bytes of device workspace ssm_tree_attention needs (at least 256); 0 if the shape is rejected
 * (reason in ssm_last_error()). */
size_t ssm_tree_attention_workspace_size(int32_t n_seq, int32_t n_nodes, int32_t Hq, int32_t Hkv, int32_t D,
                                         int32_t max_cache_len);

/*
 * ssm_kv_commit -- the K and V rows of the accepted path behind the cached rows, all layers in one call:
 * row path[s][i] of sequence s's tree becomes cache row cache_len[s] + i, i < path_len[s].
 *   path, path_len  device int32 [S][max_path], [S] (ssm_accept_path).  A path ends before its first entry
 *                   outside [0, n_nodes) (SSM_STATUS_PATH_RANGE) and before a row without a page
 *                   or past 2^31 - 2 (SSM_STATUS_SEQ_RANGE)
 *   k, v            device bf16 [n_layers][S*n][Hkv*D], dense
 *   k_pages, v_pages  device bf16 [n_layers][n_pages][Hkv][page_size][D], written
 *   len_out         device int32 [S]: cache_len + the rows committed; it may be cache_len
 */
int ssm_kv_commit(int32_t n_layers, int32_t n_seq, int32_t n_nodes, int32_t Hkv, int32_t D, int32_t max_path,
                  const int32_t *path, const int32_t *path_len, const uint16_t *k, const uint16_t *v,
                  uint16_t *k_pages, uint16_t *v_pages, int32_t n_pages, int32_t page_size, const int32_t *page_table,
                  int32_t max_pages, const int32_t *cache_len, int32_t *len_out, int32_t *dev_status, void *stream);

/*
 * ssm_tree_attention_fp8 -- ssm_tree_attention over an 8-bit cache; the nodes' own rows are bf16 as there.
 *   k_pages, v_pages    device e4m3 [n_pages][Hkv][page_size][D]
 *   k_scales, v_scales  device fp32 [n_pages][Hkv][page_size / block], from 2^-100 to 2^120 (those that ssm_kv_commit_fp8
 *                       writes are powers of two).  The rows of a block with any other scale count as absent, where a
 *                       sequence has such rows, and set SSM_STATUS_SCALE
 *   block               a power of two, 8 .. page_size
 * q that is not finite, and values of k that are not, make scores that are NaN.  scale from 2^-40 to 2^40.  The other arguments,
 * workspace and rounding as for ssm_tree_attention: q loses what is below 2^-18 of its row's largest magnitude (with up to 16 query
 * rows of a key/value head, n_nodes * Hq / Hkv, 2^-38: a node's last bits may differ with the number of nodes).  The weights of the
 * nodes' own rows are rounded to bf16.  A cached row's weight is held in fp16 together with its scale of v, to 2^-11 of their product
 * and 2^-31 of the query row's largest such product; the nodes' own rows count there as if their scale were the least among up to 256
 * of the first cached rows, taken as 2^-60 .. 2^60.
 * A row of q * scale whose largest magnitude is below 2^-52, and a block of k below 2^-58, may count as that large.  The sums before
 * the division are fp32: scales of v are to lie within 2^100 of each other (those below 2^-60 count as that here), values of v below
 * 2^100, and the nodes' own below 2^110 times the least scale above.
 */
int ssm_tree_attention_fp8(int32_t n_seq, int32_t n_nodes, int32_t Hq, int32_t Hkv, int32_t D, const ssm_node *layout,
                           const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv,
                           const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scales, const float *v_scales,
                           int32_t n_pages, int32_t page_size, int32_t block, const int32_t *page_table, int32_t max_pages,
                           const int32_t *cache_len, int32_t max_cache_len, float scale, uint16_t *o, int64_t ldo,
                           void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Host-only.  Bytes of device workspace ssm_tree_attention_fp8 needs (at least 256); 0 if the shape is rejected. */
size_t ssm_tree_attention_fp8_workspace_size(int32_t n_seq, int32_t n_nodes, int32_t Hq, int32_t Hkv, int32_t D,
                                             int32_t max_cache_len);

/*
 * ssm_kv_commit_fp8 -- ssm_kv_commit into an 8-bit cache.
 *   k_pages, v_pages    device e4m3 [n_layers][n_pages][Hkv][page_size][D], written
 *   k_scales, v_scales  device fp32 [n_layers][n_pages][Hkv][page_size / block], written
 *   block               a power of two, 8 .. page_size
 * A block's scale is the least power of two, from 2^-100 on, under which the largest finite value of its rows is at most 448 of
 * it.  A block that starts with these rows takes its scale from them; one that holds rows of the sequence already keeps its
 * own, or takes the larger one that the new rows need, and those older rows are then rounded again (a step down by a
 * power of two: only values below 2^-6 of the scale lose anything).  Rows behind the committed ones keep their bits.
 * A value that is not finite becomes NaN.  A scale outside 2^-100 .. 2^120 where such a block has rows sets
 * SSM_STATUS_SCALE; it is replaced, and the older rows keep their bits.  A block is one sequence's: two that share a page have
 * shared rows in whole blocks only, since a block that grows is rounded again.
 */
int ssm_kv_commit_fp8(int32_t n_layers, int32_t n_seq, int32_t n_nodes, int32_t Hkv, int32_t D, int32_t max_path,
                      const int32_t *path, const int32_t *path_len, const uint16_t *k, const uint16_t *v,
                      uint8_t *k_pages, uint8_t *v_pages, float *k_scales, float *v_scales, int32_t n_pages,
                      int32_t page_size, int32_t block, const int32_t *page_table, int32_t max_pages,
                      const int32_t *cache_len, int32_t *len_out, int32_t *dev_status, void *stream);

/*
 * Rotary positions.  Of each head the first `rot` columns are rot/2 pairs; pair i of a row at position p is turned by
 * p * f_i and multiplied by `amplitude`:
 *     a' = amplitude (a cos - b sin),   b' = amplitude (b cos + a sin).
 * The pairs are columns (i, i + rot/2), or with `interleaved` (2i, 2i + 1).  The other columns are copied.
 *
 * ssm_rope_frequencies -- host-only.  f_i in radians a position, base^(-2i/rot), for a context that is to be `factor` times
 * as long as the `original_len` positions of the training:
 *   SSM_ROPE_PLAIN     as they are (factor is not read)
 *   SSM_ROPE_LINEAR    all divided by factor
 *   SSM_ROPE_BASE      the base multiplied by factor^(rot/(rot-2)): the slowest pair is divided by factor, the fastest kept
 *   SSM_ROPE_BY_PARTS  pairs that make `low` turns or fewer over original_len divided by factor, those of `high` turns or more
 *                      kept, those between divided in part (linearly in the turns); 0 <= low < high
 *
 * ssm_rope_turns -- host-only.  The kernels' table of any frequencies: f / (2 pi) in units of 2^-64 of a turn, modulo one.  A
 * position times an entry, modulo 2^64, is exact; what grows with the position is the entry's own rounding alone, 2^-55 of a turn
 * for f up to 1.
 */
#define SSM_ROPE_PLAIN 0
#define SSM_ROPE_LINEAR 1
#define SSM_ROPE_BASE 2
#define SSM_ROPE_BY_PARTS 3
int ssm_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double original_len, double low,
                         double high, double *freq);
int ssm_rope_turns(int32_t n, const double *freq, uint64_t *turns);

/*
 * ssm_rope -- q and k rows at given positions.
 *   Hq, Hkv      heads of q and of k (either may be 0: that tensor is then not read)
 *   D            columns of a head, a multiple of 8, 8 .. 512;  rot even, 2 .. D
 *   turns        device uint64 [rot / 2] (ssm_rope_turns);  amplitude finite
 *   positions    device int32 [n_tok]; a negative one turns backwards
 *   q, k         device bf16 [n_tok][ldq], [n_tok][ldk]: Hq*D and Hkv*D columns
 *   q_out, k_out device bf16, strides ldqo, ldko; each may be its input (it may not overlap it in part)
 * Pointers 16-byte aligned, row strides multiples of 8.  Angles to 2^-25 of a turn up to position 2^29, to 2^-23 at any (f up to 1);
 * products in fp32, rounded once.
 *
 * ssm_tree_rope -- the same for row s*n + v at position cache_len[s] + depth of node v.  A depth outside [0, n_nodes) counts as
 * 0 and sets SSM_STATUS_BAD_LAYOUT, a negative length counts as 0 and sets SSM_STATUS_SEQ_RANGE.
 */
int ssm_rope(int32_t n_tok, int32_t Hq, int32_t Hkv, int32_t D, int32_t rot, int32_t interleaved, const uint64_t *turns,
             float amplitude, const int32_t *positions, const uint16_t *q, int64_t ldq, uint16_t *q_out, int64_t ldqo,
             const uint16_t *k, int64_t ldk, uint16_t *k_out, int64_t ldko, void *stream);
int ssm_tree_rope(int32_t n_seq, int32_t n_nodes, int32_t Hq, int32_t Hkv, int32_t D, int32_t rot, int32_t interleaved,
                  const uint64_t *turns, float amplitude, const ssm_node *layout, const int32_t *cache_len,
                  const uint16_t *q, int64_t ldq, uint16_t *q_out, int64_t ldqo, const uint16_t *k, int64_t ldk,
                  uint16_t *k_out, int64_t ldko, int32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_ATTENTION_H_ */
