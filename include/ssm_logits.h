/*
 * ssm_logits.h -- what a speculative decoder takes from rows of logits: the target's
 * token at every node (for ssm_accept_path), the alternatives that a draft tree's
 * children are made from, the log probabilities of drafted tokens, and the entropy.
 *
 * Same conventions as ssm_tree.h.
 */
#ifndef SSM_LOGITS_H_
#define SSM_LOGITS_H_

#include <stdint.h>

#include "ssm_tree.h"

#define SSM_STATUS_TOKEN_RANGE 64 /* a token outside [-1, n_vocab) */
#define SSM_MAX_TOP 32            /* alternatives of a row */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ssm_token_scores -- with lse = log sum_j exp(scale x_j) over a row x of logits,
 *     logprob[t][i]     = scale x[tokens[t][i]] - lse
 *     entropy[t]        = lse - sum_j p_j scale x_j,  p_j = exp(scale x_j - lse)
 *     top[t][0 .. k-1]  the indices of the k largest logits, largest first, of equal ones the lowest index first
 *     top_logprob[t][i] = scale x[top[t][i]] - lse
 * in one pass over the logits.
 *   n_rows, n_vocab  rows and columns; n_vocab >= 1
 *   logits           device fp32 (f32 = 1) or bf16 (f32 = 0) [n_rows][ld], ld >= n_vocab, rows of any alignment
 *   scale            1 / temperature, from 2^-100 to 2^100
 *   m, tokens        tokens device int32 [n_rows][m]; -1: none, its logprob is 0; others outside [0, n_vocab): NaN and
 *                    SSM_STATUS_TOKEN_RANGE.  logprob device fp32 [n_rows][m].  m = 0: neither is read or written; m <= 2^31 - 256
 *   entropy          device fp32 [n_rows], or NULL
 *   k, top, top_logprob  0 <= k <= SSM_MAX_TOP, k <= n_vocab; device int32 and fp32 [n_rows][k]; top_logprob may be NULL
 * Logits of minus infinity have probability 0.  A row with a NaN or plus infinity, or with nothing above minus infinity, has NaN for
 * its lse and all that comes from it; its alternatives are in the order of its logits all the same, a NaN behind all others.
 * Sums and differences in fp32, whatever the logits' type.
 */
int ssm_token_scores(int32_t n_rows, int32_t n_vocab, const void *logits, int32_t f32, int64_t ld, float scale, int32_t m,
                     const int32_t *tokens, float *logprob, float *entropy, int32_t k, int32_t *top, float *top_logprob,
                     int32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_LOGITS_H_ */
