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
 */
#ifndef SSM_ATTENTION_H_
#define SSM_ATTENTION_H_

#include <stddef.h>
#include <stdint.h>

#include "ssm_prompt.h"
#include "ssm_tree.h"

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

#ifdef __cplusplus
}
#endif

#endif /* SSM_ATTENTION_H_ */
