/*
 * mxfp4.h -- C ABI of libmxcast, third part: 4-bit MX data (MXFP4: e2m1
 * elements under the e8m0 block scales of mxcast.h) and the products that read
 * it, and the gated feed-forward block on MX operands of either width, with
 * its gradient and its form for a few rows.
 *
 * Conventions are those of mxcast.h and mxtrain.h: device pointers,
 * caller-owned buffers and stream, no allocation, no synchronisation, no host
 * read of device memory, host validation before any HIP call, asynchronous;
 * outputs must not overlap inputs or each other; the same bits in every call on
 * the same inputs; binary32 sums, one rounding of a bf16 result at the end;
 * padding bytes of a blocked scale layout that is read may hold anything.
 *
 * MXFP4 rule:
 *   amax  = max |x| over a block of 32 (NaN > +Inf > finite);
 *   e     = floor(log2(amax)) - 2, clamped to [-127, 127]; amax = 0 gives
 *           e = -127; the scale byte is e + 127; a block holding a NaN gets
 *           the byte 0xFF and zero codes;
 *   code  = x / 2^e rounded to nearest-even among 0, 0.5, 1, 1.5, 2, 3, 4, 6,
 *           saturated to +-6 (so +-Inf -> +-6); the sign bit of a code is x's.
 * Two codes to a byte, the first of them in its low half.  A block's value is
 * code * 2^(byte - 127); byte 0xFF stands for NaN.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include "mxcast.h"
#include "mxtrain.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Formats of an operand's codes. */
#define MX_FORMAT_E4M3 0 /* MXFP8: a byte an element, (rows, k) bytes          */
#define MX_FORMAT_E2M1 1 /* MXFP4: half a byte an element, (rows, k / 2) bytes */

#define MX_MAX_DECODE_ROWS 64 /* most rows of x that the decode forms take */

/*
 * Cast to MXFP4 along dim0 and dim1 from one read of the input.
 *   x      (batch, rows, cols) of x_type, rows ldx elements apart, matrices
 *          rows * ldx apart; its element's alignment.
 *   q_row  (batch, rows, cols / 2) codes of blocks along each row; 4-byte
 *          aligned.
 *   s_row  e8m0, plain (batch, rows, cols / 32), or with blocked != 0 each
 *          matrix's in the 128 x 4 blocked layout, mx_blocked_bytes(batch,
 *          rows, cols / 32) bytes, every byte written (padding 0); 4-byte
 *          aligned.
 *   q_col  (batch, cols, rows / 2): the cast of each matrix's columns in
 *          blocks of 32 rows, a row for each column; 16-byte aligned.
 *   s_col  plain (batch, cols, rows / 32), or blocked likewise; 4-byte aligned.
 * Either output pair may be NULL (both members); both pairs NULL, a half-NULL
 * pair or x NULL -> MX_ERR_NULL.  cols a multiple of 32; rows any, but a
 * multiple of 32 where q_col is given; cols <= ldx <= 2^31; batch * (rows
 * rounded up to 128) * (cols rounded up to 128) < 2^34; else MX_ERR_SHAPE.
 */
MX_API mx_status mx_cast_mxfp4(const void* x, int32_t x_type, int64_t batch, int64_t rows, int64_t cols, int64_t ldx,
                               uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, int32_t blocked,
                               hipStream_t stream);

/*
 * The values of an MXFP4 cast: x (batch, rows, cols) of x_type, contiguous,
 * 16-byte aligned, from codes q (batch, rows, cols / 2), 4-byte aligned, and
 * scales s, plain or blocked as above.  Exact in both types (where 2^e * code
 * is past binary32's range, above byte 252, it is +-Inf).  Shapes as above.
 */
MX_API mx_status mx_dequantize_mxfp4(const uint8_t* q, const uint8_t* s, int64_t batch, int64_t rows, int64_t cols,
                                     int32_t blocked, void* x, int32_t x_type, hipStream_t stream);

/*
 * Product with MXFP4 weights: C[m][n] = sum over k of A(m, k) * B(n, k).
 *   qa, sa   A's codes in a_format and its (m, k / 32) scales in the blocked
 *            layout, as for mx_gemm_mxfp8; 16-byte aligned.
 *   qb, sb   B's MXFP4 codes (n, k / 2) and blocked scales; 16-byte aligned.
 *   c        (m, n) of c_type, its element's alignment (16-byte, with rows of
 *            whole 16-byte words, is faster).
 * With A in MXFP4 every step of the sum is binary32's.  With A in MXFP8 the
 * matrix instruction adds the products of eight neighbouring k, from a multiple
 * of eight on, with fewer bits, as in mx_gemm_mxfp8: each is cut toward zero to a
 * multiple of 2^-13 times the largest 2^(ea + eb) among those that are not zero
 * (ea, eb the exponents of the codes' fields, before the scales; a subnormal code
 * has its format's lowest), which takes less than that unit from each but the
 * largest.  The groups of eight meet in binary32.  A NaN code or scale gives NaN
 * where it enters.
 * m, n, k >= 0, k % 32 == 0, k <= 2^23, n <= 2^24, n * k < 2^36, m < 2^31 and
 * the tiles of a launch, else MX_ERR_SHAPE; m or n 0 writes nothing; k 0
 * writes zeros.
 */
MX_API mx_status mx_gemm_mxfp4(const uint8_t* qa, const uint8_t* sa, int32_t a_format, const uint8_t* qb,
                               const uint8_t* sb, int64_t m, int64_t n, int64_t k, void* c, int32_t c_type,
                               hipStream_t stream);

/*
 * The same grouped along M, with mx_grouped_gemm_mxfp8's arguments and rules:
 * A's scales in the M-grouped blocked layout, num_groups consecutive (n, k / 2)
 * code matrices and blocked scales of B; rows past the last end are not
 * written.  m + 256 * num_groups < 2^31.
 */
MX_API mx_status mx_grouped_gemm_mxfp4(const uint8_t* qa, const uint8_t* sa, int32_t a_format, const uint8_t* qb,
                                       const uint8_t* sb, const int32_t* group_end_offsets, int32_t num_groups,
                                       int64_t m, int64_t n, int64_t k, void* c, int32_t c_type, hipStream_t stream);

/*
 * Product of a few bf16 rows with MX weights, for decoding:
 *   c[m][n] = sum over k of x[m][k] * W(n, k).
 *   x        bf16 (m, k), rows ldx elements apart; 2-byte aligned.
 *   qw, sw   W's codes in w_format and blocked scales; 16-byte aligned.
 *   c        (m, n) of c_type, contiguous, its element's alignment.
 * x enters as it is; a code times its scale is exact in bf16 but for e4m3
 * values under scale bytes 0 to 2 (rounded to a multiple of 2^-133) and for
 * values of 2^128 and above (e2m1 from byte 253 on, e4m3 from 247), which are
 * +-Inf as in mx_dequantize_mxfp4, also where their product with x is not.
 * 0 <= m <= MX_MAX_DECODE_ROWS, 0 <= n <= 2^27 - 16, k % 32 == 0, 0 <= k <=
 * 2^23, n * k < 2^36, k <= ldx <= 2^28, else MX_ERR_SHAPE; m or n 0 writes
 * nothing; k 0 writes zeros.
 */
MX_API mx_status mx_linear_decode(const void* x, int64_t ldx, const uint8_t* qw, const uint8_t* sw, int32_t w_format,
                                  int64_t m, int64_t n, int64_t k, void* c, int32_t c_type, hipStream_t stream);

/*
 * Gated feed-forward block on MX operands, both projections, the activation
 * and the product in one kernel:
 *   (g, u)[t][j] = sum over k of X(t, k) * (Wg, Wu)(j, k);  y = act(g) * u.
 *   qx, sx   X's codes (rows, k) in x_format and blocked scales (the M-grouped
 *            blocked layout with group_end_offsets); 16-byte aligned.
 *   qw, sw   codes in w_format of num_groups matrices (2 * cols, k), Wg's rows
 *            and then Wu's, and their blocked scales one after another;
 *            16-byte aligned.  Pairs of formats: (E4M3, E4M3), (E4M3, E2M1),
 *            (E2M1, E2M1), x's first; else MX_ERR_SHAPE.
 *   group_end_offsets  NULL: one group, all rows (num_groups must be 1), else
 *            DEVICE int32 [num_groups], cumulative END rows, clamped on the
 *            device as by mx_scales_to_blocked_grouped; rows past the last end
 *            are not written.
 *   act      MX_ACT_SILU or MX_ACT_GELU.
 *   y        bf16 (rows, cols), 16-byte aligned.
 *   q, s     the 8-bit checkpoint of (g, u), as mx_gated_act writes it of a
 *            bf16 h, here of the binary32 sums: codes (rows, 2 * cols), 16-byte
 *            aligned, and plain scales (rows, 2 * cols / 32); or both NULL.
 * Sums as for mx_gemm_mxfp4: with an MXFP8 operand products are cut before they
 * are added, so that a few of the checkpoint's codes (of numbers next to the
 * middle of two) are the neighbour of what exact sums give.
 * rows, cols, k >= 0; cols and k multiples of 32; k <= 2^23, cols <= 2^24, 2 *
 * cols * k < 2^36, rows + 256 * num_groups < 2^31, else MX_ERR_SHAPE.
 */
MX_API mx_status mx_gated_ffn(const uint8_t* qx, const uint8_t* sx, int32_t x_format, const uint8_t* qw,
                              const uint8_t* sw, int32_t w_format, const int32_t* group_end_offsets,
                              int32_t num_groups, int64_t rows, int64_t cols, int64_t k, int32_t act, void* y,
                              uint8_t* q, uint8_t* s, hipStream_t stream);

/*
 * The same of a few bf16 rows (x as for mx_linear_decode): y bf16 (m, cols),
 * 2-byte aligned; 0 <= cols <= 2^27 - 16, 2 * cols * k < 2^36.
 */
MX_API mx_status mx_gated_ffn_decode(const void* x, int64_t ldx, const uint8_t* qw, const uint8_t* sw,
                                     int32_t w_format, int64_t m, int64_t cols, int64_t k, int32_t act, void* y,
                                     hipStream_t stream);

/*
 * Gradient of the block's inside, through its second projection: with D the
 * gradient of the block's output (rows, k) and Wd the second projection's
 * weight (k, cols),
 *   dy[t][j] = sum over i of D(t, i) * Wd(i, j);
 *   dh[:, :cols] = dy * u * act'(g);  dh[:, cols:] = dy * act(g);
 *   y (or NULL) = act(g) * u again,
 * (g, u) the checkpoint's values.  dh is what the weight gradient
 * (mx_wgrad_checkpoint) and, cast, the product with the first projections'
 * weights take.
 *   qd, sd   D's codes along its rows in d_format, (rows, k), and blocked
 *            scales, as qx and sx above.
 *   qw, sw   num_groups matrices (cols, k): Wd cast along the axis that is
 *            summed (the dim1 cast of Wd), and blocked scales.
 *   q, s     as mx_gated_ffn or mx_gated_act wrote them; q 16-byte aligned.
 *   dh       bf16 (rows, 2 * cols); y bf16 (rows, cols); 16-byte aligned.
 * Shapes, formats, groups and act as above (cols * k < 2^36).
 */
MX_API mx_status mx_gated_ffn_backward(const uint8_t* qd, const uint8_t* sd, int32_t d_format, const uint8_t* qw,
                                       const uint8_t* sw, int32_t w_format, const int32_t* group_end_offsets,
                                       int32_t num_groups, int64_t rows, int64_t cols, int64_t k, int32_t act,
                                       const uint8_t* q, const uint8_t* s, void* dh, void* y, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
