/*
 * moe_balance.h -- the training side of the router in libmoe.so: the
 * load-balance loss of a routing decision with its per-expert counts, and
 * the gradient of the router's logits.
 *
 * Conventions as in moe.h: device pointers to dense row-major arrays, sizes
 * checked on the host before anything is launched, work only enqueued on
 * `stream`, nothing allocated, bit-identical results for the same inputs.
 *
 * Tokens and sequences.  The T tokens of a call are rows of one batch that
 * may hold several sequences: sequence s owns tokens seq_offsets[s] ..
 * seq_offsets[s+1]-1 (device array [S+1], non-decreasing, within [0, T]).
 * NULL with S == 1 means that the whole batch is one sequence.  token_mask
 * [T] uint8 or NULL: a token with mask 0 (padding) takes no part.  So do the
 * tokens outside every sequence.  The rows of such tokens are not used: they
 * may hold anything, NaN included.  A seq_offsets array that is not as
 * stated gives wrong results, but no access out of bounds.
 */
#ifndef MOE_BALANCE_H
#define MOE_BALANCE_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_MAX_SEQUENCES 65536 /* S */

/*
 * Balance loss and per-expert counts ("DeepGEMM walkthrough" §2.2's
 * L_aux = alpha E sum_e f_e P_e, taken over each sequence and averaged over
 * the sequences that have a token).  With p_t = softmax(logits[t][.]) and
 * n_s the number of tokens of sequence s that take part:
 *   tokens[s] = n_s, tokens[S] = S+, the number of sequences with n_s > 0
 *   counts[s][e] = #{(t, j) in s : topk_idx[t][j] == e}
 *   probs[s][e]  = (1 / n_s) sum_{t in s} p_t[e]
 *   *loss = alpha / S+ * sum_s E sum_e counts[s][e] / (n_s k) probs[s][e]
 * A sequence without tokens has counts and probs 0 and adds nothing; with
 * S+ == 0 (T == 0, say) the loss is 0.  Entries of topk_idx outside [0, E) are counted
 * nowhere.  A logit of -inf is an expert of probability 0 (a row of nothing
 * else has p = 0 everywhere); other non-finite logits of tokens that take
 * part are a caller error.
 *
 * logits [T][E] fp32 (16-byte aligned), topk_idx [T][k] int32; counts [S][E]
 * int32, probs [S][E] fp32, tokens [S+1] int32 and loss [1] fp32 are
 * written.  Sums in a fixed order, in fp32 or more; what they lose does not
 * grow with T.  Counts are exact.  One sequence over the whole batch
 * without a mask gives moe_router_stats' P and loss up to the rounding of the
 * sums.
 * ws (device, 4-byte aligned) must hold moe_balance_loss_workspace_size(T,
 * E, S) bytes (else MOE_ERR_WORKSPACE); calls that share it must be ordered.
 * Requires 1 <= k <= min(E, MOE_MAX_TOPK), E <= MOE_MAX_EXPERTS,
 * 1 <= S <= MOE_MAX_SEQUENCES, T <= 2^26.
 */
moe_status_t moe_balance_loss(const float *logits, const int32_t *topk_idx,
                              const int32_t *seq_offsets, const uint8_t *token_mask, int T,
                              int E, int k, int S, float alpha, int32_t *counts, float *probs,
                              int32_t *tokens, float *loss, void *ws, size_t ws_bytes,
                              moe_stream_t stream);

/* Bytes of device workspace moe_balance_loss needs for these sizes. */
size_t moe_balance_loss_workspace_size(int T, int E, int S);

/*
 * Gradient of the router's logits: of the gate weights moe_route returned
 * and of the balance loss, in one pass.  For every token that takes part,
 * with p = softmax(logits[t][.]):
 *   d_logits[t][e] =
 *       p[e] (g[e] - sum_i g[i] p[i]),  g[e] = sum_j d_topk_w[t][j] [topk_idx[t][j] == e]
 *     + p[e] (b[e] - sum_i b[i] p[i]),  b[e] = *d_loss alpha E / (S+ n_s)
 *                                              counts[s][e] / (n_s k)
 * With MOE_ROUTE_RENORM (topk_w is the softmax q over the selected logits)
 * the first line is sum_j [topk_idx[t][j] == e] q_j (d_topk_w[t][j] -
 * sum_i d_topk_w[t][i] q_i).  topk_idx and counts are constants of the
 * derivative.  The rows of tokens that take no part are written as zero.
 *
 * d_topk_w [T][k] fp32 or NULL (no gate term; flags must then be 0).
 * counts [S][E] and tokens [S+1] int32 are moe_balance_loss's, or both NULL
 * (no balance term; d_loss must then be NULL and S and seq_offsets only say
 * which tokens take part).  d_loss [1] fp32 or NULL (1).  One of the two
 * terms must be there.  Entries of topk_idx outside [0, E) had no weight and
 * get no gradient.  d_logits [T][E] fp32 must not overlap an input; logits
 * and d_logits are 16-byte aligned.  T == 0 is a no-op.  Limits as for
 * moe_balance_loss.
 */
moe_status_t moe_route_backward(const float *logits, const int32_t *topk_idx,
                                const float *d_topk_w, unsigned flags, const int32_t *counts,
                                const int32_t *tokens, float alpha, const float *d_loss,
                                const int32_t *seq_offsets, const uint8_t *token_mask, int T,
                                int E, int k, int S, float *d_logits, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BALANCE_H */
