/*
 * dgemm_scored.h -- C ABI of the routing by scores.
 *
 * dgemm_route (dgemm_experts.h) ranks a token's experts by their logits.
 * dgemm_route_scored ranks them by a score plus a balance bias, within the best
 * groups of experts, and weights them by the score alone. Its outputs are those of
 * dgemm_route: what the grouped products and dgemm_combine take.
 *
 * The conventions of dgemm_experts.h hold.
 */
#ifndef DGEMM_SCORED_H
#define DGEMM_SCORED_H

#include "dgemm_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most groups of experts of one call. */
#define DGEMM_MAX_EXPERT_GROUPS 32

typedef enum {
    DGEMM_SCORE_SOFTMAX = 0, /* exp(x_e) / sum over the row's experts that may be chosen */
    DGEMM_SCORE_SIGMOID = 1  /* 1 / (1 + exp(-x_e))                                      */
} dgemm_score_t;

typedef enum {
    DGEMM_GROUP_MAX = 0, /* a group's worth: its largest choice value                    */
    DGEMM_GROUP_TOP2 = 1 /* the sum of its two largest (of one, where it has only one)   */
} dgemm_group_score_t;

typedef struct {
    int score;        /* dgemm_score_t                                                   */
    int groups;       /* G: experts e with the same e / (E/G) are a group; divides E;
                       * 1 <= G <= DGEMM_MAX_EXPERT_GROUPS                               */
    int groups_kept;  /* experts are taken from this many groups, 1 <= groups_kept <= G  */
    int group_score;  /* dgemm_group_score_t                                             */
    int renormalize;  /* != 0: a token's weights are divided by their sum                */
    float weight_scale; /* the weights are multiplied by this at the end                 */
} dgemm_scoring_t;

/* Routes T tokens to k of E experts each:
 *   s_e = score of logits[t,e],  c_e = s_e + bias[e]  (the choice value),
 *   the groups_kept groups of most worth are kept, among their experts the k largest
 *   c_e are chosen, largest first; equal values (of groups, of experts): lowest index.
 *   weights[t,j] = weight_scale * s_id, with renormalize weight_scale * s_id / sum_j s_id
 *   (a sum of sigmoid scores below 2^-126 counts as 2^-126); 0 for id -1. Without
 *   renormalize, or beside a chosen logit above -20, a score below 2^-126 may count as 0.
 * The order is that of the values in FP64: where FP32 values are too near to tell, the
 * token is decided again (values that FP64 cannot tell apart are equal). Without a bias,
 * and with all groups kept or groups ranked by their largest value, the order of the logits
 * decides.
 *   logits   [T,E] F32 or BF16. An expert whose logit or bias is -inf or NaN is never
 *            chosen and has no part in the softmax; +inf counts as the largest finite number.
 *   bias     [E] F32 or NULL (all 0).
 *   scoring  in HOST memory, read before the call returns.
 * Groups without an expert that may be chosen are not kept. Fewer than k experts left:
 * id -1, weight 0, row -1. ids, weights, offsets, row_token, slot_row, ws and the limits
 * on T, E and k are those of dgemm_route; ws holds dgemm_route_workspace_size(T, E, k)
 * bytes. k may exceed the experts of the kept groups (the rest of the ids is -1). */
dgemm_status_t dgemm_route_scored(const void* logits, dgemm_dtype_t logits_dtype, int64_t T, int64_t E, int k,
                                  const float* bias, const dgemm_scoring_t* scoring, int32_t* ids, float* weights,
                                  int32_t* offsets, int32_t* row_token, int32_t* slot_row, void* ws, size_t ws_bytes,
                                  dgemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DGEMM_SCORED_H */
