/*
 * mxfp4.h - C ABI of the MXFP4 operators of the MI355X (gfx950) library.
 *
 * MXFP4: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign bit), two to a
 * byte (the element of the lower index in the low nibble), and one E8M0 scale
 * per 32 consecutive elements along the reduction direction.  The quantizer
 * takes BF16, the products run on the scaled FP4 matrix instructions with
 * fp32 accumulation and write BF16.
 *
 * The conventions of mxfp8.h hold here too: device pointers, a hipStream_t
 * passed as void*, validation on the host before anything is launched, no
 * allocation, no synchronisation, no fallback, and the same status codes.
 *
 * Numerics (OCP MX):
 *  - shared exponent X = floor(log2 amax) - 2 of a block's amax, clamped to
 *    >= -127; scale byte = X + 127 (0 for an all-zero block);
 *  - code = E2M1(x * 2^-X) rounded to nearest, ties to the even code,
 *    saturated to +-6, sign of zero kept;
 *  - dequantized value = E2M1 value * 2^(byte - 127).
 */
#ifndef MXFP4_H
#define MXFP4_H

#include "mxfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MXFP4_ROWWISE 1u        /* blocks along rows: q_row[rows][cols/2], s_row[rows][cols/32]      */
#define MXFP4_COLWISE 2u        /* blocks along columns, stored transposed:
                                   q_colT[cols][rows/2], s_colT[cols][rows/32]                      */
#define MXFP4_PACKED_SCALES 16u /* s_row / s_colT as packed words, the layout of mxfp8_pack_scales:
                                   s_row  uint32 [cols/128][rows] (cols % 128 == 0),
                                   s_colT uint32 [rows/128][cols] (rows % 128 == 0)                 */

/*
 * x       BF16 [x_rows][ld_x], 16-byte aligned; ld_x >= cols, ld_x % 8 == 0.
 * index   optional DEVICE int32 [rows], 4-byte aligned (ROWWISE alone): output
 *         row r is the copy of x's row index[r]; an index outside
 *         [0, x_rows) gives a row of zeros (codes and scales 0).  NULL: output
 *         row r is x's row r, and x_rows == rows.
 * rows    >= 0; a multiple of 32 with COLWISE (128 with PACKED_SCALES too).
 * cols    >= 0; a multiple of 32 (128 with ROWWISE and PACKED_SCALES).
 * flags   ROWWISE, COLWISE or both, plus PACKED_SCALES optionally.
 * q_row, q_colT  codes, 16-byte aligned; s_row, s_colT scales (4-byte aligned
 *         when packed).  Those of a copy that is not asked for are ignored.
 * Errors: NULL, SHAPE, MISALIGNED, FLAGS, LIMIT, HIP.  Inputs with NaN or Inf
 * are outside the contract (codes unspecified; nothing faults).
 */
mxfp8_status mxfp4_quantize(const void *x, int64_t x_rows, int64_t rows, int64_t cols, int64_t ld_x,
                            const int32_t *index, uint32_t flags,
                            uint8_t *q_row, void *s_row, uint8_t *q_colT, void *s_colT,
                            void *stream);

/*
 * BF16 values of a rowwise (or transposed columnwise) copy.
 * q       codes [rows][cols/2], 16-byte aligned.
 * s       scales: bytes [rows][cols/32], or with PACKED_SCALES words
 *         [cols/128][rows] (4-byte aligned).
 * out     BF16 [rows][ld_out], 16-byte aligned; ld_out >= cols, ld_out % 8 == 0.
 * flags   0 or MXFP4_PACKED_SCALES.
 * A scale byte of 255 (the E8M0 NaN) gives NaN; products beyond the BF16 range
 * give +-inf.
 */
mxfp8_status mxfp4_dequantize(const uint8_t *q, const void *s, int64_t rows, int64_t cols,
                              void *out, int64_t ld_out, uint32_t flags, void *stream);

#define MXFP4_GEMM_ACCUMULATE 1u /* C = bf16( float(C) + sum )                               */
#define MXFP4_GEMM_SWIGLU 8u     /* C[m][n] = bf16( SiLU(g) * u ): B holds 2N rows, gate rows
                                    0..N-1 then up rows N..2N-1 (per expert when grouped)    */

/*
 *   C[m][n] = bf16( sum_k dq(A)[m][k] * dq(B)[n][k] ),  fp32 accumulation.
 *
 * a         codes [M][K/2], 16-byte aligned.
 * a_packed  packed scales of A, uint32 [K/128][M].
 * b         codes [N][K/2] ([2N][K/2] with SWIGLU), 16-byte aligned.
 * b_packed  packed scales of B, uint32 [K/128][rows of B].
 * c         BF16 [M][ldc], 16-byte aligned; ldc >= N, ldc % 8 == 0.
 * M >= 0; N >= 0, N % 32 == 0; K >= 0, K % 128 == 0, K <= 2^22.  K == 0
 * writes zeros (ACCUMULATE: leaves C).  flags: 0 or one of the above.
 * Errors: NULL, SHAPE, MISALIGNED, FLAGS, LIMIT, HIP.
 */
mxfp8_status mxfp4_gemm(const uint8_t *a, const uint32_t *a_packed,
                        const uint8_t *b, const uint32_t *b_packed,
                        void *c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                        uint32_t flags, void *stream);

/*
 *   for g < G, for m in [offsets[g], offsets[g+1]):
 *       C[m][n] = bf16( sum_k dq(A)[m][k] * dq(B_g)[n][k] ).
 *
 * b [G][N][K/2] ([G][2N][K/2] with SWIGLU), b_packed [K/128][G * rows of an
 * expert], offsets DEVICE int32 [G+1] with the meaning and the clamping of
 * mxfp8_grouped_gemm (rows outside every group are not written; invalid
 * offsets make no access leave the buffers), 1 <= G <= 65535.
 */
mxfp8_status mxfp4_grouped_gemm(const uint8_t *a, const uint32_t *a_packed,
                                const uint8_t *b, const uint32_t *b_packed,
                                const int32_t *offsets, int32_t G,
                                void *c, int64_t ldc, int64_t M_total, int64_t N, int64_t K,
                                uint32_t flags, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
