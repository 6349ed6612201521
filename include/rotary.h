/*
 * rotary.h - C ABI of the rotary positions of the MI355X (gfx950) library.
 *
 * The conventions of mxfp8.h hold here too: device pointers, a hipStream_t
 * passed as void*, validation on the host before anything is launched, no
 * allocation, no synchronisation, no fallback, and the same status codes.
 */
#ifndef MXFP8_ROTARY_H
#define MXFP8_ROTARY_H

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define ROTARY_FP32 0
#define ROTARY_BF16 1
#define ROTARY_FP16 2

/* Flags. */
#define ROTARY_INTERLEAVED 1u /* pairs (2 f, 2 f + 1); else (f, f + pairs)                          */
#define ROTARY_INVERSE 2u     /* by the opposite angle: the gradient of the inputs from the outputs' */

/*
 * Turns the pairs (a, b) of the first 2 * pairs dimensions of every head of q
 * and k by the angle 2 pi positions[i] turns[f]:
 *   (a, b) -> magnitude (a cos - b sin, a sin + b cos),
 * and copies the other dimensions.  The angle is reduced to a part of a turn in
 * 64 bits, the rest is fp32, rounded once.
 *
 * q, k     [tokens][q_heads or k_heads][head_dim] of dtype with strides in
 *          elements (token, head; unit stride along the head), aligned to the
 *          element; k_heads may be 0 (k and k_out NULL).
 * q_out, k_out  dense [tokens][heads][head_dim]; may not overlap the inputs.
 * positions int32 [tokens]; turns fp64 [pairs], 8-byte aligned.
 * head_dim >= 1, 0 <= 2 * pairs <= head_dim, head_dim <= 65536.
 * tokens * (q_heads + k_heads) * head_dim < 2^40, and at most 2^32 - 256 threads,
 * each of which takes two runs of 16 bytes (two elements where pairs, head_dim, the
 * strides or the addresses are no multiples of 16 bytes) of up to eight heads.
 * Errors: NULL, SHAPE, MISALIGNED, FLAGS (dtype or flags unknown), LIMIT, HIP.
 */
mxfp8_status rotary_rotate(const void *q, int64_t q_token, int64_t q_head, int64_t q_heads, const void *k,
                           int64_t k_token, int64_t k_head, int64_t k_heads, int32_t dtype, int64_t tokens,
                           int64_t head_dim, int64_t pairs, const int32_t *positions, const double *turns,
                           float magnitude, uint32_t flags, void *q_out, void *k_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_ROTARY_H */
