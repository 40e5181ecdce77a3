/*
 * ssm_prompt.h -- the state a draft tree is verified from: prompts and single
 * tokens of a Mamba2 layer.
 *
 *   x B C rows of the input projection -> ssm_prompt_conv -> x | B | C
 *   -> ssm_prompt_scan (ragged prompts) or ssm_scan_step (one token a sequence)
 *   -> y, the state h and the conv ring that ssm_tree_verify starts from.
 *
 * The scan is linear attention with a decay for each head: with
 * D_t = softplus(dt_t + dt_bias) and a_t = exp(-D_t exp(A_log)),
 *     h_t = a_t h_{t-1} + D_t x_t (x) B_t,     y_t = C_t h_t + D x_t.
 * H heads of head_dim P; B and C are shared by H / n_groups consecutive heads
 * (n_groups = 1: by all).  Groups are the scan's and the step's only: rows of
 * ssm_prompt_conv, like those of ssm_tree.h, have one group, conv_dim = H*P + 2*N.
 *
 * Same conventions as ssm_tree.h.  The calls work on ONE layer: `layer` picks its
 * parameters, and its part of a cache that holds all L layers of n_slots sequences
 * (h [n_slots][L][H][P][N], ring [n_slots][L][R][conv_dim], ring_head [n_slots][L]:
 * the order of ssm_tree.h's instances).  Sequences are ragged: sequence s has the
 * token rows cu_seqlens[s] .. cu_seqlens[s+1]-1 (it may have none) and the cache
 * slot slots[s] (slots = NULL: s).  Two sequences of a call must not share a slot
 * or a row.
 * A sequence whose rows, slot or length are out of range is skipped (its rows and
 * its slot stay as they were) and sets SSM_STATUS_SEQ_RANGE.
 */
#ifndef SSM_PROMPT_H_
#define SSM_PROMPT_H_

#include <stddef.h>
#include <stdint.h>

#include "ssm_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_STATUS_SEQ_RANGE 32 /* cu_seqlens, a slot, a length or a page out of range */

/*
 * ssm_prompt_conv -- post[t] = SiLU(conv_b + sum_k conv_w[k] row[t-3+k]) over each
 * sequence, the rows before its first being ring positions head-3 .. head-1 (a new
 * sequence: those rows zero).  Afterwards the last min(len, 3) rows stand at ring
 * positions head+len-3 .. head+len-1 (mod R) and ring_head has advanced by len.
 *   n_seq, n_slots, n_tok   sequences, slots of the cache, rows of xBC and out
 *   max_len     bound on a sequence's length (longer ones are skipped); blocks are launched for
 *               max_len tokens of every sequence, so a bound far above the lengths costs time
 *   cu_seqlens  device int32 [n_seq + 1]       slots  device int32 [n_seq] or NULL
 *   xBC         device bf16 [n_tok][ldx], conv_dim columns, ldx a multiple of 8, 16-byte aligned
 *   out         device bf16 [n_tok][ldo], same rules; must not overlap xBC
 *   ring, ring_head   device, updated
 */
int ssm_prompt_conv(const ssm_dims *dims, const ssm_params *prm, int32_t layer, int32_t n_seq, int32_t n_slots,
                    int32_t n_tok, int32_t max_len, const int32_t *cu_seqlens, const int32_t *slots,
                    const uint16_t *xBC, int64_t ldx, uint16_t *ring, int32_t *ring_head, uint16_t *out, int64_t ldo,
                    int32_t *dev_status, void *stream);

/*
 * ssm_prompt_scan -- the recurrence above over ragged sequences, in chunks.
 *   x          device bf16 [n_tok][ldx]: H*P columns      B, C  device bf16 [n_tok][ldb], [n_tok][ldc]:
 *              n_groups*N columns.  16-byte aligned, row strides multiples of 8
 *   dt         device bf16 [n_tok][lddt]: H columns (raw dt)
 *   h_in       device fp32 [n_slots][L][H][P][N], read only, or NULL: all states zero
 *   h_out      device fp32, same shape, written for this layer and these sequences' slots (a sequence
 *              without tokens: its h_in); it may be h_in
 *   y          device bf16 [n_tok][ldy]: H*P columns, 16-byte aligned, ldy a multiple of 8
 *              (it may be x, with ldy = ldx; otherwise it must not overlap an input)
 *   workspace  device, 256-byte aligned, >= ssm_prompt_scan_workspace_size() bytes, as
 *              ssm_tree_verify's
 * max_len as above.  State and sums are fp32; the products of the state update keep x D w to 24 bits;
 * what y reads (the chunk's scores and the state) is rounded to bf16, as y itself is (relative error of
 * y 0.0018, of which its own rounding 0.0017).  ssm_scan_step keeps 32 bits throughout.
 * Only conv-free members of dims and prm are used (n_heads, head_dim, d_state, n_layers; dt_bias, A_log, D).
 */
int ssm_prompt_scan(const ssm_dims *dims, const ssm_params *prm, int32_t layer, int32_t n_groups, int32_t n_seq,
                    int32_t n_slots, int32_t n_tok, int32_t max_len, const int32_t *cu_seqlens, const int32_t *slots,
                    const uint16_t *x, int64_t ldx, const uint16_t *B, int64_t ldb, const uint16_t *C, int64_t ldc,
                    const uint16_t *dt, int64_t lddt, const float *h_in, float *h_out, uint16_t *y, int64_t ldy,
                    void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Host-only.  Bytes of device workspace ssm_prompt_scan needs (at least 256); 0 if the shape is rejected
 * (reason in ssm_last_error()). */
size_t ssm_prompt_scan_workspace_size(const ssm_dims *dims, int32_t n_seq, int32_t n_tok, int32_t max_len,
                                      int32_t n_groups);

/*
 * ssm_scan_step -- the same for one token of each sequence: row s of x, B, C, dt and y belongs to
 * sequence s.  Arguments as for ssm_prompt_scan; h is read and written once.
 */
int ssm_scan_step(const ssm_dims *dims, const ssm_params *prm, int32_t layer, int32_t n_groups, int32_t n_seq,
                  int32_t n_slots, const int32_t *slots, const uint16_t *x, int64_t ldx, const uint16_t *B,
                  int64_t ldb, const uint16_t *C, int64_t ldc, const uint16_t *dt, int64_t lddt, const float *h_in,
                  float *h_out, uint16_t *y, int64_t ldy, int32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_PROMPT_H_ */
