/*
 * mxtrain.h -- C ABI of libmxcast, second part: the operators of a training
 * step that stand next to the casts and GEMMs of mxcast.h -- layer norm with
 * its gradients, the MoE router with its balance loss, a gated activation
 * that keeps its input in 8 bits, and a linear layer's weight gradient from
 * an input kept in 8 bits.
 *
 * Conventions are those of mxcast.h: device pointers, caller-owned buffers
 * and stream, no allocation, no synchronisation, no host read of device
 * memory, host validation before any HIP call, asynchronous.  Additionally:
 *  - Rows of an input that has a leading dimension (ld*) start ld elements
 *    apart, ld >= its row length; everything else is contiguous.
 *  - Outputs must not overlap inputs or each other.
 *  - Results are the same bits in every call on the same inputs: sums are
 *    formed in a fixed order, no floating-point atomics.
 *  - Sums, statistics and probabilities are binary32; a value stored as bf16
 *    is rounded once, nearest-even, at the end.
 *
 * An 8-bit activation checkpoint is the dim0 MX cast of a bf16 matrix (rows,
 * cols), cols a multiple of 32, as mx_cast_dim0_dim1 writes it: e4m3 codes
 * (rows, cols) and row-major e8m0 scale bytes (rows, cols / 32).  Any number
 * of rows is accepted here.  Its value is code * 2^(scale - 127); a NaN code
 * or a scale byte 0xFF stands for NaN.
 */
#ifndef MXTRAIN_H
#define MXTRAIN_H

#include "mxcast.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the arguments that come in several. */
#define MX_TYPE_BF16 0
#define MX_TYPE_F32 1

/* Gate functions. */
#define MX_ACT_SILU 0 /* g * s(g), s the logistic function                        */
#define MX_ACT_GELU 1 /* GELU in its tanh form, g * s(2 sqrt(2 / pi) (g + 0.044715 g^3)) */

#define MX_MAX_NORM_COLS 16384 /* longest layer-norm row               */
#define MX_MAX_TOPK 32         /* most experts chosen per row          */

/*
 * Layer norm over the rows of x:
 *   mean = sum x / cols;  var = sum (x - mean)^2 / cols (around the mean
 *   itself, not from a sum of squares);  rstd = 1 / sqrt(var + eps);
 *   y = (x - mean) * rstd * weight + bias.
 *   x       (rows, cols), x_type, rows ldx elements apart.
 *   weight  (cols) of w_type;  bias (cols) of w_type, or NULL for none.
 *   y       (rows, cols) of x_type.
 *   mean, rstd  binary32 (rows), what the backward pass needs.
 *   q, s    both NULL, or (x_type bf16, cols a multiple of 32) the 8-bit
 *           checkpoint of y as stored: codes (rows, cols), 8-byte aligned,
 *           and scales (rows, cols / 32).
 * 0 <= rows < 2^31, 0 <= cols <= MX_MAX_NORM_COLS, cols <= ldx <= 2^31, else
 * MX_ERR_SHAPE (also a bad type, or q on a shape without a checkpoint).
 * With rows or cols 0 nothing is written: mean and rstd of rows without
 * columns are 0 / 0, and the caller's to set.
 * Pointers need their element's alignment (MX_ERR_ALIGN); where x, weight,
 * bias and y are 16-byte aligned and cols and ldx are whole 16-byte words,
 * the kernel moves whole words, which q requires (MX_ERR_ALIGN):
 * mx_layernorm_checkpoint is the form without that.
 */
MX_API mx_status mx_layernorm(const void* x, int64_t ldx, int32_t x_type, const void* weight, const void* bias,
                              int32_t w_type, int64_t rows, int64_t cols, float eps, void* y, float* mean,
                              float* rstd, uint8_t* q, uint8_t* s, hipStream_t stream);

/*
 * mx_layernorm of a bf16 x with its checkpoint, from rows at any pitch and
 * start: x, weight, bias and y need their element's alignment only, q 8 bytes'
 * (MX_ERR_ALIGN).  Rows of whole words take the kernel that mx_layernorm
 * takes and give the same bits; others are read at any element.
 */
MX_API mx_status mx_layernorm_checkpoint(const void* x, int64_t ldx, const void* weight, const void* bias,
                                         int32_t w_type, int64_t rows, int64_t cols, float eps, void* y, float* mean,
                                         float* rstd, uint8_t* q, uint8_t* s, hipStream_t stream);

/*
 * Gradients of mx_layernorm, with xh = (x - mean) * rstd and g = dy * weight:
 *   dx = rstd * (g - mean_row(g) - xh * mean_row(g * xh));
 *   dweight = sum over rows of dy * xh;  dbias = sum over rows of dy.
 *   dy (rows, cols) of x_type, rows lddy elements apart; x, mean, rstd and
 *   weight as in the forward call.
 *   dx       (rows, cols) of x_type.
 *   dweight  binary32 (cols);  dbias binary32 (cols), or NULL.
 *   workspace  mx_layernorm_backward_workspace_bytes(rows, cols) bytes of
 *            device scratch, 16-byte aligned, not used by another call until
 *            this one has run; needs no clearing.
 * With rows 0 the weight gradients are written as zeros.  Two kernels: the
 * first leaves one row of weight-gradient sums per workgroup in the
 * workspace, the second adds them up in a fixed order.
 */
MX_API int64_t mx_layernorm_backward_workspace_bytes(int64_t rows, int64_t cols);
MX_API mx_status mx_layernorm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, int32_t x_type,
                                       const void* weight, int32_t w_type, const float* mean, const float* rstd,
                                       int64_t rows, int64_t cols, void* dx, float* dweight, float* dbias,
                                       void* workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * MoE router.  A row of logits takes part unless valid[row] is 0 or every
 * logit of it is -inf; nothing of a row that does not take part is used.
 *   p = softmax(logits row).
 *   chosen[row][j], j < topk: the experts of the topk largest logits in
 *     descending order, equal logits in ascending expert order, NaN before
 *     +inf; an expert with logit -inf is never chosen: where fewer than topk
 *     remain (and in rows that take no part) the slot holds -1.
 *   gates[row][j] = p[chosen], divided by the row's sum of them if normalize;
 *     0 in slots that hold -1.
 *   lse[row] = log(sum exp(logits)), 0 for a row that takes no part.
 *   counts[e] = slots that hold e;  N = rows that take part;
 *   ends[e] = sum over i <= e of counts[i] rounded up to a multiple of
 *     `align`: the cumulative END offsets that the grouped casts and GEMMs
 *     take, for groups padded to that multiple (32 keeps every 32-row block
 *     of mx_cast_dim0_dim1_grouped_blocked whole).
 *   balance[e] = experts * counts[e] / (topk * N^2), 0 if N is 0;
 *   loss = sum over e of balance[e] * (sum over rows of p[row][e])
 *        = experts * sum_e (counts[e] / (topk N)) * (mean over rows of p).
 * Gradients take the counts as constants: balance[e] is then the derivative
 * of the loss by p[row][e] of any row that takes part.
 *   logits     (rows, experts) of l_type (bf16 or binary32), rows ld apart.
 *   valid      one byte per row, or NULL (every row valid).
 *   chosen     int32 (rows, topk);  gates binary32 (rows, topk);  lse binary32
 *              (rows);  counts, ends int32 (experts);  balance binary32
 *              (experts);  loss one binary32.
 *   workspace  mx_router_workspace_bytes(rows, experts) bytes, as above.
 * 1 <= experts <= MX_MAX_GROUPS (else MX_ERR_GROUPS), 1 <= topk <=
 * min(experts, MX_MAX_TOPK), align >= 1, 0 <= rows, rows * topk + experts *
 * align < 2^31, experts <= ld <= 2^31, else MX_ERR_SHAPE.  With rows 0 counts,
 * ends, balance and loss are written as zeros.
 */
MX_API int64_t mx_router_workspace_bytes(int64_t rows, int64_t experts);
MX_API mx_status mx_router_balance(const void* logits, int64_t ld, int32_t l_type, const uint8_t* valid,
                                   int64_t rows, int32_t experts, int32_t topk, int32_t normalize, int32_t align,
                                   int32_t* chosen, float* gates, float* lse, int32_t* counts, int32_t* ends,
                                   float* balance, float* loss, void* workspace, int64_t workspace_bytes,
                                   hipStream_t stream);

/*
 * The gradient of the logits, from the gates' gradients dgates (binary32
 * (rows, topk), or NULL for none; slots that hold -1 are ignored) and the
 * loss's (one binary32 on the device, or NULL for 0):
 *   dp[e] = dloss * balance[e] + sum over j with chosen[j] = e of d_j, where
 *     d_j = dgates[j], or with normalize (dgates[j] - sum_i dgates[i] *
 *     gates[i]) / (sum of p over the chosen);
 *   dlogits[e] = p[e] * (dp[e] - sum over i of p[i] * dp[i]),
 * p formed again from the logits and lse, and scaled to a sum of 1 where lse is
 * so large that its rounding shows.  Rows whose first slot holds -1 get
 * zeros.  chosen entries outside [0, experts) are ignored; a row's others are
 * distinct, as mx_router_balance leaves them.
 *   dlogits    (rows, experts) of l_type, contiguous.
 */
MX_API mx_status mx_router_balance_backward(const void* logits, int64_t ld, int32_t l_type, const float* lse,
                                            const int32_t* chosen, const float* gates, const float* balance,
                                            const float* dgates, const float* dloss, int64_t rows,
                                            int32_t experts, int32_t topk, int32_t normalize, void* dlogits,
                                            hipStream_t stream);

/*
 * Gated activation with its input kept in 8 bits.  h (rows, 2 * cols) bf16
 * holds the gate in its first cols columns and the factor in the others:
 *   y = act(h[:, :cols]) * h[:, cols:]   (from h itself), bf16 (rows, cols);
 *   q, s  the 8-bit checkpoint of h: codes (rows, 2 * cols), scales (rows,
 *         2 * cols / 32), the bytes mx_cast_dim0_dim1 writes for h; or both
 *         NULL (no checkpoint).
 *   act   MX_ACT_SILU or MX_ACT_GELU.
 * rows >= 0, cols >= 0 a multiple of 32, cols < 2^32, rows * cols <= 2^34,
 * else MX_ERR_SHAPE; h and y 16-byte, q 8-byte aligned, else MX_ERR_ALIGN.
 */
MX_API mx_status mx_gated_act(const void* h, int64_t rows, int64_t cols, int32_t act, void* y, uint8_t* q,
                              uint8_t* s, hipStream_t stream);

/*
 * Its gradient from the checkpoint, with (g, u) the checkpoint's values:
 *   dh[:, :cols] = dy * u * act'(g);  dh[:, cols:] = dy * act(g);
 *   y (or NULL) = act(g) * u again, for a caller that did not keep it.
 * dy, y (rows, cols) and dh (rows, 2 * cols) bf16, 16-byte aligned; q, s as
 * written by the forward call.
 */
MX_API mx_status mx_gated_act_backward(const void* dy, const uint8_t* q, const uint8_t* s, int64_t rows,
                                       int64_t cols, int32_t act, void* dh, void* y, hipStream_t stream);

/*
 * Weight gradient of a linear layer from the 8-bit checkpoint of its input:
 *   dw_g[i][j] = sum over rows t of group g of dy[t][i] * x[t][j],
 *   dy  bf16 (rows, n), rows lddy elements apart;
 *   x   the checkpoint q (rows, k), s (rows, k / 32);
 *   group_end_offsets  NULL: one group, all rows (num_groups must be 1), else
 *       DEVICE int32 [num_groups], cumulative END rows, clamped on the device
 *       as by mx_scales_to_blocked_grouped; rows past the last end belong to
 *       no group; an empty group's gradient is zero.
 *   dw  (num_groups, n, k), binary32 or bf16 by dw_type.
 * Products are formed on the bf16 matrix cores and summed in binary32: a
 * code times its scale is exact in bf16 but for some values under scale bytes
 * 0, 1 and 2, which reach below bf16's smallest step of 2^-133 and are rounded
 * to the nearest multiple of it.  Where the output has too few tiles to fill
 * the GPU the rows are split and the pieces' binary32 sums, kept in the
 * workspace, are added in a fixed order.  Where n is not a multiple of 8 and
 * the product long enough, the workspace also holds a copy of dy in aligned
 * rows, rows * (n rounded up to 8) * 2 bytes, by far the most of it at large
 * sizes (16640 x 8191 x 5120: 340 MB, where n = 8192 needs 67 MB).
 *   workspace  mx_wgrad_checkpoint_workspace_bytes(rows, n, k, num_groups)
 *              bytes, 16-byte aligned (NULL allowed where that is 0).
 * rows, n >= 0, k >= 0 a multiple of 32, rows < 2^31 - 512, n, k and lddy <=
 * 2^22, lddy >= n, else MX_ERR_SHAPE; 1 <= num_groups <= MX_MAX_GROUPS, else
 * MX_ERR_GROUPS.  dy 2-byte aligned (16-byte, with n and lddy multiples of
 * 8, is faster), q 16-byte aligned, dw its element's alignment.
 */
MX_API int64_t mx_wgrad_checkpoint_workspace_bytes(int64_t rows, int64_t n, int64_t k, int32_t num_groups);
MX_API mx_status mx_wgrad_checkpoint(const void* dy, int64_t lddy, const uint8_t* q, const uint8_t* s,
                                     int64_t rows, int64_t n, int64_t k, const int32_t* group_end_offsets,
                                     int32_t num_groups, void* dw, int32_t dw_type, void* workspace,
                                     int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXTRAIN_H */
