/*
 * moeq_route.h -- expert routing with softmax or sigmoid scores, a bias for
 * balance, groups of experts and renormalised weights: the router of layers
 * that moe_route_topk (moeq.h) does not cover (gfx950).
 *
 * The conventions of moeq.h hold: device pointers, caller-owned buffers,
 * asynchronous work on `stream`, no allocation, no synchronization, the same
 * status codes, arguments checked before any HIP call, deterministic results.
 */
#ifndef MOEQ_ROUTE_H
#define MOEQ_ROUTE_H

#include "moeq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* scores */
#define MOEQ_SCORE_SOFTMAX 0   /* s_e = exp(l_e) / sum over all experts of exp(l) */
#define MOEQ_SCORE_SIGMOID 1   /* s_e = 1 / (1 + exp(-l_e))                       */

/* Most groups of experts. */
#define MOEQ_MAX_GROUPS 64

/*
 * moe_route_experts -- per token, with l its logits:
 *   c_e = s_e + bias_e        (the choice: bias moves it, and only it)
 *   groups of E / n_group consecutive experts; a group's value is the sum of the
 *     group_best largest c of its experts (of those there are, if fewer are left
 *     unmasked); the topk_group largest groups stay, ties to the lower group
 *   topk_ids = the k largest c of the groups that stay, ties to the lower expert,
 *     best first
 *   topk_w_j = s of expert j, divided by the k chosen scores' sum (renormalize
 *     != 0), times scale
 * The choice is that of the real numbers c, not of their fp32 roundings: where two
 * of them are too close to be told apart in fp32 they are compared in 64 bits.
 * Without a bias experts are ordered by their logits.
 *
 * A logit (or bias) of -inf masks an expert: it is chosen only after every unmasked
 * expert of the groups that stay, lower experts first (those of other groups
 * included), and has weight 0.  A group without an unmasked expert stays only after
 * all the others.  A token with every expert masked gets the experts 0 .. k - 1 and
 * weights 0.  Other logits and biases are finite (with a NaN or +inf among a token's
 * values its ids stay distinct and inside [0, E), and its outputs mean nothing).
 *
 *   logits   [T, E] fp32 or bf16 (logits_dtype), row stride ld_logits elements
 *   bias     [E] fp32 or NULL
 *   topk_ids [T, k] int32 (out)        topk_w [T, k] fp32 (out)
 * Limits: 0 <= T <= 2^25, 1 <= E <= MOEQ_MAX_EXPERTS, 1 <= n_group <= MOEQ_MAX_GROUPS, E %
 * n_group == 0, 1 <= topk_group <= n_group, group_best 1 or 2, 1 <= k <=
 * min(MOEQ_MAX_TOPK, topk_group * E / n_group), ld_logits >= E, scale finite;
 * every pointer aligned to its elements; outputs do not overlap inputs.
 */
int moe_route_experts(const void* logits, int logits_dtype, int64_t ld_logits, const float* bias,
                      int T, int E, int k, int scoring, int n_group, int topk_group,
                      int group_best, int renormalize, float scale, int32_t* topk_ids,
                      float* topk_w, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOEQ_ROUTE_H */
