/*
 * moe.h - C ABI of the mixture-of-experts operators of the MI355X (gfx950)
 * library: expert routing with its gradient, the counting sort of the
 * (token, slot) pairs by expert, and the weighted combination of the experts'
 * outputs with its gradients.  Together with mxfp4_quantize's row gather and
 * the grouped GEMMs they are the parts of an MoE layer.
 *
 * The conventions of mxfp8.h hold here too: device pointers, a hipStream_t
 * passed as void*, validation on the host before anything is launched, no
 * allocation, no synchronisation, no fallback, and the same status codes.
 * Results do not depend on the order in which workgroups run.
 */
#ifndef MXFP8_MOE_H
#define MXFP8_MOE_H

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define MOE_FP32 0
#define MOE_BF16 1
#define MOE_FP16 2

/* Flags of moe_route / moe_route_backward. */
#define MOE_ROUTE_SIGMOID 1u     /* scores sigmoid(logit) instead of softmax over the row's experts */
#define MOE_ROUTE_RENORMALIZE 2u /* weights divided by (their sum + 1e-20)                           */

#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_TOP_K 64

/*
 * Expert choice of every row t of logits [tokens][ld]:
 *   score_e  = softmax(logits[t])_e or sigmoid(logits[t][e]);
 *   choice_e = score_e + bias[e] (bias NULL: score_e);
 *   groups > 1: the experts are `groups` runs of experts / groups; a run's
 *     value is the sum of its group_top largest choices (fewer where it has
 *     fewer experts; a choice or a sum of NaN counts as -inf), and only the
 *     experts of the top_groups runs of the largest values can be chosen;
 *   ids[t]     = the top_k experts of the largest choices, largest first;
 *   weights[t] = their scores, renormalized if asked for.
 * Ties go to the lowest index (of group or expert).  The order is that of the
 * scores in 64 bits, not of their 32-bit roundings; without a bias it is the
 * logits' own, that of the runs too where group_top is 1.  The sums, weights and
 * gradients are 32-bit; a weight is within 16 ulp (2e-6) of its exact value (7e-8
 * of it on average), and under softmax |logit - largest| 2^-23 of it more (the
 * rounding of that difference).
 * A logit of -inf has score 0 (a row of nothing else has scores and weights
 * of 0), and a score below fp32's normal range (2^-126) may be given as 0.  NaN
 * or +inf under softmax make the row's weights NaN, under sigmoid a NaN has a
 * NaN score.  A choice of NaN is ordered below every other one, so ids are
 * always top_k different experts.
 *
 * dtype      of the logits: MOE_FP32, MOE_BF16 or MOE_FP16 (aligned to it).
 * experts    1 .. MOE_MAX_EXPERTS; ld >= experts.
 * top_k      1 .. min(experts, MOE_MAX_TOP_K).
 * groups     1 .. min(experts, 64), dividing experts; top_groups 1 .. groups,
 *            top_k <= top_groups * (experts / groups).
 * group_top  1 or 2 (ignored with groups == 1).
 * bias       fp32 [experts] or NULL.
 * weights    fp32 [tokens][top_k]; ids int32 [tokens][top_k].
 * Errors: NULL, SHAPE, MISALIGNED, FLAGS (flags or dtype unknown), LIMIT, HIP.
 */
mxfp8_status moe_route(const void *logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t ld,
                       const float *bias, int32_t top_k, int32_t groups, int32_t top_groups, int32_t group_top,
                       uint32_t flags, float *weights, int32_t *ids, void *stream);

/*
 * Gradient of the logits for the gradient dweights [tokens][top_k] (fp32) of
 * the weights; the choice itself is a constant, so the bias has none.  dlogits
 * [tokens][experts] has the logits' dtype.  ids as moe_route wrote them (an id
 * outside [0, experts) is skipped).
 */
mxfp8_status moe_route_backward(const void *logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t ld,
                                const int32_t *ids, const float *dweights, int32_t top_k, uint32_t flags,
                                void *dlogits, void *stream);

/*
 * Stable counting sort of the slots (t, k), in the order t * top_k + k, by
 * ids[t][k]:
 *   offsets  int32 [experts + 1]: expert e has the sorted rows
 *            offsets[e] .. offsets[e + 1] - 1;
 *   token    int32 [tokens * top_k]: the token of each sorted row;
 *   position int32 [tokens][top_k]: the sorted row of each slot.
 * An id outside [0, experts) belongs to nobody: its position is -1, and the
 * rows from offsets[experts] on have token -1.
 * workspace: moe_dispatch_workspace_bytes(tokens, experts, top_k) bytes of
 * device memory, 4-byte aligned (NULL where that is 0); not kept.
 * tokens * top_k < 2^31; experts 1 .. MOE_MAX_EXPERTS; top_k >= 1.
 * Errors: NULL, SHAPE, MISALIGNED, WORKSPACE, LIMIT, HIP.
 */
size_t moe_dispatch_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k);
mxfp8_status moe_dispatch(const int32_t *ids, int64_t tokens, int64_t experts, int64_t top_k,
                          int32_t *offsets, int32_t *token, int32_t *position,
                          void *workspace, size_t workspace_bytes, void *stream);

/*
 * out[t] = sum_k weights[t][k] * y[position[t][k]], the sum in fp32 in the
 * order of k, rounded once.  A position outside [0, rows) adds nothing.
 * y    [rows][ld_y] of dtype, out [tokens][hidden] of dtype.
 * weights fp32 and position int32, both [tokens][top_k].
 * Errors: NULL, SHAPE, MISALIGNED (to the element), FLAGS (dtype), LIMIT, HIP.
 */
mxfp8_status moe_combine(const void *y, int32_t dtype, int64_t rows, int64_t ld_y, const int32_t *position,
                         const float *weights, int64_t tokens, int64_t top_k, int64_t hidden, void *out,
                         void *stream);

/*
 * Gradients of moe_combine for dout [tokens][ld_dout] of dtype:
 *   dy[r]         = sum over the slots with position r of weights * dout[t]
 *                   (rows without a slot: zeros; one slot, as moe_dispatch
 *                   gives them: rounded once; several: summed in slot order);
 *   dweights[t][k] = <dout[t], y[position[t][k]]> in fp32 (0 for a position
 *                   outside [0, rows)).
 * dy [rows][hidden] or NULL, dweights [tokens][top_k] or NULL: what is NULL is
 * not computed.  workspace: 4 * rows bytes, 4-byte aligned, where dy is not
 * NULL; not kept.
 */
mxfp8_status moe_combine_backward(const void *y, int32_t dtype, int64_t rows, int64_t ld_y, const int32_t *position,
                                  const float *weights, int64_t tokens, int64_t top_k, int64_t hidden,
                                  const void *dout, int64_t ld_dout, void *dy, float *dweights,
                                  void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_MOE_H */
