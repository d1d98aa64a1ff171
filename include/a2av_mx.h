/*
 * a2av_mx.h -- what stands before an MoE layer's exchange: the root-mean-square
 * norm with the residual's addition, and microscaled rows -- 8 or 4 bits a value
 * with a scale for each 32 -- which travel through the exchange in a half or a
 * quarter of the bytes, and the experts' products on them.
 *
 * A serving layer on W ranks (a2av_moe.h has the other calls):
 *
 *   a2av_norm              h += x; y = norm(h), written as packed rows (and plain, for the router)
 *   a2av_route, a2av_dispatch   row_bytes = a2av_mx_row_bytes(features, format)
 *   a2av_expert_matmul_mx  packed rows times packed weights, in 32 bits
 *   a2av_quantise          the inner activations packed again, for the next product
 *   a2av_combine_weighted  a token's rows summed, onto h
 *
 * A packed row of D values, Dp being D rounded up to 32:
 *
 *   values   A2AV_MXFP8: Dp bytes, e4m3 (largest 448; no infinity).
 *            A2AV_MXFP4: Dp / 2 bytes, e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6, and a sign),
 *            value 2 i in the low half of byte i.
 *   scales   Dp / 32 bytes: s stands for 2^(s - 127), for values 32 b .. 32 b + 31; 255 for NaN.
 *   zeros    up to a multiple of 32 bytes; those of the values past D too.
 *
 * So a row and its scales are one row of the exchange.  What a value stands for is
 * code * scale.  a2av_quantise and a2av_norm choose a block's scale as the smallest
 * (2^-127 at least) that its largest value fits under, and round each value / scale to
 * the nearest code, ties to the even one: nothing is cut off.  A block that holds a
 * NaN or an infinity gets the scale NaN and codes of 0: all of it is NaN.
 *
 * Conventions are those of a2av_moe.h.  Packed buffers are aligned to 16 bytes.
 */
#ifndef A2AV_MX_H_
#define A2AV_MX_H_

#include "a2av_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How rows are held. */
typedef enum {
  A2AV_PLAIN = 0, /* an a2av_dtype_t */
  A2AV_MXFP8 = 1, /* packed, e4m3 */
  A2AV_MXFP4 = 2  /* packed, e2m1 */
} a2av_format_t;

/* Most features of a norm's row, and of a packed one. */
#define A2AV_MAX_NORM_FEATURES 16384
#define A2AV_MAX_MX_FEATURES (1 << 24)

/* a2av_mx_row_bytes -- bytes of a packed row; -1 for a format that is not packed, and
 * for features outside 1 .. A2AV_MAX_MX_FEATURES. */
int64_t a2av_mx_row_bytes(int64_t features, int format);

/*
 * a2av_norm -- root-mean-square norm of the tokens of all W ranks.  For a token's
 * row, in 32 bits:
 *
 *   s = x + residual, rounded to dtype and kept    (without residual: s = x)
 *   y = s / sqrt(mean(s^2) + eps) * weight
 *
 * y is rounded from 32 bits, to dtype or to the codes of a packed row; the scale of a row's
 * block goes by its largest value as it was before the rounding to 32 bits.  The norm is
 * that of the rounded s, which is all that the backward pass needs.  A row of NaN or
 * infinities stays within its own results; squares are summed in 32 bits, so that a row whose
 * squares' sum passes 2^128 counts as one of infinite length (y = 0 where s is finite).
 * Squares below 2^-126 keep fewer bits the smaller they are, and where all of a row's are 0
 * (values below 2^-75) and eps is 0 as well, y is NaN.  Both are for eps to prevent.
 *
 *  features           H, 1 .. A2AV_MAX_NORM_FEATURES.
 *  dtype              a2av_dtype_t of x, residual, sums (and of y, with A2AV_PLAIN).
 *  format             a2av_format_t of y.
 *  eps                >= 0 and finite.
 *  x_ptrs             HOST array of W: [tokens][H].
 *  tokens_per_rank    HOST int64 [W], up to 2^31 - 1 together.
 *  weight_dev         DEVICE float [H], of all ranks.
 *  residual_ptrs      HOST array of W: [tokens][H], or NULL.
 *  sum_ptrs           HOST array of W: s is written here, or NULL.  May be x_ptrs or
 *                     residual_ptrs.
 *  out_ptrs           HOST array of W: y, [tokens][H] or [tokens][a2av_mx_row_bytes(H)].
 *  plain_ptrs         HOST array of W: y rounded to dtype as well (for a router's product),
 *                     with a packed format, or NULL.
 *
 * Device error: A2AV_ERR_TIMEOUT when a copy has not come for about a second: results
 * are not complete.  Host errors: A2AV_ERR_INVALID_ARG, A2AV_ERR_UNSUPPORTED (features or
 * tokens above the limits), A2AV_ERR_CUDA.
 */
int a2av_norm(a2av_handle *h, int64_t features, int dtype, int format, float eps,
              const void *const *x_ptrs, const int64_t *tokens_per_rank, const float *weight_dev,
              const void *const *residual_ptrs, void *const *sum_ptrs, void *const *out_ptrs,
              void *const *plain_ptrs, void *stream);

/* a2av_norm_workspace_bytes -- device workspace of a2av_norm_backward with a weight's
 * gradient for `total_rows` tokens together; -1 for what it would reject. */
int64_t a2av_norm_workspace_bytes(int64_t features, int64_t total_rows);

/*
 * a2av_norm_backward -- its gradients.  With r = 1 / sqrt(mean(s^2) + eps) and
 * g = dy * weight:
 *
 *   d_x = r * (g - s r^2 mean(g s)) + d_sums        (of x, and of the residual as well)
 *   d_weight = sum over all tokens of dy * s * r    (in 32 bits, in a fixed order)
 *
 * A row of infinite length (see a2av_norm) has r = 0: its d_x is d_sums, NaN where s is not finite.
 * Products g s are summed in 32 bits too: a row where that sum alone passes 2^128 gets
 * infinities or NaN.
 *
 *  sum_ptrs           s as the forward call kept it (x, without a residual).
 *  d_out_ptrs         HOST array of W: dy [tokens][H], of dtype.
 *  d_sum_ptrs         HOST array of W: what reaches s from elsewhere, or NULL (0).
 *  d_x_ptrs           HOST array of W: [tokens][H], written.  May be d_out_ptrs or d_sum_ptrs.
 *  d_weight_dev       DEVICE float [H], written, or NULL (not wanted).
 *  workspace          DEVICE scratch, 256-byte aligned, of at least
 *                     a2av_norm_workspace_bytes(H, sum of tokens) where d_weight_dev is given, not
 *                     shared with a call in flight.
 * Errors are those of a2av_norm.
 */
int a2av_norm_backward(a2av_handle *h, int64_t features, int dtype, float eps,
                       const void *const *sum_ptrs, const int64_t *tokens_per_rank,
                       const float *weight_dev, const void *const *d_out_ptrs,
                       const void *const *d_sum_ptrs, void *const *d_x_ptrs, float *d_weight_dev,
                       void *workspace, int64_t workspace_bytes, void *stream);

/*
 * a2av_quantise -- rows of `features` values of dtype to packed rows of `format`, and
 * a2av_dequantise -- back: code * scale, rounded once to dtype.
 *
 *  rows_per_rank      HOST int64 [W], up to 2^31 - 1 together: the rows that the buffers hold.
 *                     Weights [K][Z][D] are K * Z rows.
 *  in_splits_dev      DEVICE int64 [W][W], S as a2av_dispatch writes it, or NULL.  With it
 *                     rank p's rows are those that it has received, the first sum_r S[r][p]
 *                     (read on the device); rows past them are neither read nor written.
 *  x_ptrs / out_ptrs  HOST arrays of W: [rows][features].
 *  packed_ptrs        HOST array of W: [rows][a2av_mx_row_bytes(features, format)].
 *
 * Device error: A2AV_ERR_BAD_SPLITS when an entry of S is negative or a rank has received more
 * rows than its buffers hold: nothing is written.  Host errors are those of a2av_norm.
 */
int a2av_quantise(a2av_handle *h, int64_t features, int dtype, int format,
                  const void *const *x_ptrs, const int64_t *rows_per_rank,
                  const int64_t *in_splits_dev, void *const *packed_ptrs, void *stream);
int a2av_dequantise(a2av_handle *h, int64_t features, int dtype, int format,
                    const void *const *packed_ptrs, const int64_t *rows_per_rank,
                    const int64_t *in_splits_dev, void *const *out_ptrs, void *stream);

/*
 * a2av_expert_matmul_mx -- a2av_expert_matmul on packed rows and weights of one
 * format: the same groups, counts, bias, activation, gate and residual.
 *
 *   z = sum over blocks of scale_x scale_w * (codes_x . codes_w) + b_e,  y as there
 *
 * in 32 bits, rounded once to shape->dtype, which is that of bias, residual and
 * results.  For serving: it keeps nothing for a backward pass.
 *
 *  rows_ptrs          HOST array of W: [rows_per_peer[p]][a2av_mx_row_bytes(D, format)].
 *  weight_ptrs        HOST array of W: [K][Z][a2av_mx_row_bytes(D, format)].
 * A value past D, or a scale of one, must be 0 as a2av_quantise writes it.  Other arguments
 * and errors are those of a2av_expert_matmul; D is A2AV_MAX_MX_FEATURES at most.
 */
int a2av_expert_matmul_mx(a2av_handle *h, const a2av_expert_t *shape, int format,
                          const void *const *rows_ptrs, const int64_t *rows_per_peer,
                          const int64_t *counts_dev, const void *const *weight_ptrs,
                          const void *const *bias_ptrs, const void *const *residual_ptrs,
                          void *const *out_ptrs, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* A2AV_MX_H_ */
