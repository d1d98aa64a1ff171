/*
 * a2av_moe.h -- the operators of an MoE layer around the exchange of a2av.h:
 * the router that makes the dispatch's keys, the experts' products on the rows
 * a dispatch delivers, and the weighted return path that sums a token's rows
 * again; each with its backward pass.
 *
 * A layer on W ranks with E = W * K experts (K per rank), k choices a token:
 *
 *   a2av_route             logits -> keys, weights, counts [W][E]
 *   a2av_dispatch          rows to their experts' ranks (src_row = token, key = expert)
 *   a2av_expert_matmul     each expert's rows times its weights (once or more)
 *   a2av_combine_weighted  y[t] = residual[t] + sum_j weight[t][j] * row of item (t, j)
 *
 * and back: a2av_combine_weighted_backward, a2av_expert_matmul_backward,
 * a2av_combine_weighted with NULL weights (the gradient of the dispatch: a
 * token's gradient is the sum of its items' rows) and a2av_route_backward.
 *
 * Conventions are those of a2av.h: return values, device pointers, streams and
 * the status word.  Every call is asynchronous, allocates nothing and makes no
 * host round trip: how many rows each expert has is read on the device.
 * Buffers are contiguous device memory; a pointer must be aligned to its
 * element, nothing more (16-byte aligned rows take faster kernels).  No output
 * may overlap an input or another output, except where a call says so.
 * Results do not depend on the order in which blocks run.
 */
#ifndef A2AV_MOE_H_
#define A2AV_MOE_H_

#include "a2av.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
typedef enum {
  A2AV_F32 = 0,
  A2AV_BF16 = 1,
  A2AV_F16 = 2
} a2av_dtype_t;

typedef enum {
  A2AV_SCORE_SOFTMAX = 0, /* over all experts of the row */
  A2AV_SCORE_SIGMOID = 1  /* each expert by itself */
} a2av_score_t;

/* Most choices a token has, and most groups its experts form. */
#define A2AV_MAX_TOPK 32
#define A2AV_MAX_ROUTE_GROUPS 32

/* How a2av_route chooses. */
typedef struct {
  int experts;     /* E, 1 .. A2AV_MAX_DISPATCH_KEYS */
  int topk;        /* k, 1 .. min(A2AV_MAX_TOPK, top_groups * E / groups) */
  int dtype;       /* a2av_dtype_t of the logits and of their gradient */
  int score;       /* a2av_score_t */
  int groups;      /* G >= 1 groups of E / G consecutive experts (G divides E) */
  int top_groups;  /* groups kept, 1 .. G */
  int group_top;   /* a group's score is the sum of its 1 or 2 best choices (2: E / G >= 2) */
  int renormalise; /* weights divided by their sum over the token's choices */
  float scale;     /* and multiplied by this */
} a2av_route_t;

/*
 * a2av_route -- routing to experts, for the tokens of all W ranks.
 *
 * For a token's logits x[0..E), in 32 bits:
 *   s = softmax(x), or sigmoid(x) = 1 / (1 + exp(-x))
 *   c = s + bias; for a softmax without bias and with group_top 1, c = x: the
 *       order of a softmax is that of its logits, without its rounding
 *   groups > 1: the top_groups groups of the highest scores stay, c = -inf in the others
 *   key[j]    = the expert of the j-th largest c (ties: the lowest index)
 *   weight[j] = s[key[j]], renormalised (divided by sum_j s[key[j]]) if asked, * scale
 * The bias moves choices only, never weights.  A token's keys and weights are the
 * same, to the bit, whatever other tokens are routed with it.
 *
 * Special values: a NaN choice counts as -inf, so the k keys are always valid
 * and distinct.  A logit of -inf is an expert that is not available: its score
 * is 0.  Where all the scores that a weight is divided by are 0 (every logit,
 * or every chosen one, -inf), the weight is 0.  Other NaN and infinities go
 * through the arithmetic.
 *
 *  logits_ptrs        HOST array of W device pointers: rank r's [tokens_per_rank[r]][E].
 *  tokens_per_rank    HOST int64 [W], 0 .. (2^31 - 1) / k.
 *  bias_dev           DEVICE float [E] or NULL.
 *  key_ptrs           HOST array of W: int32 [tokens][k], written; a2av_dispatch's keys.
 *  weight_ptrs        HOST array of W: float [tokens][k], written.
 *  counts_dev         DEVICE int64 [W][E] or NULL: written with the number of
 *                     rank r's items for expert e.
 *
 * Host errors: A2AV_ERR_INVALID_ARG for NULL or misaligned pointers of ranks that have
 * tokens and for values outside the ranges above; A2AV_ERR_UNSUPPORTED for more
 * experts, choices or groups than the limits, and for more tokens.
 */
int a2av_route(a2av_handle *h, const a2av_route_t *route, const void *const *logits_ptrs,
               const int64_t *tokens_per_rank, const float *bias_dev, int32_t *const *key_ptrs,
               float *const *weight_ptrs, int64_t *counts_dev, void *stream);

/*
 * a2av_route_backward -- the gradient of a2av_route's weights with respect to
 * the logits; the choice itself has none.  With g = scale * d_weight and the
 * sums over a token's choices j:
 *   softmax                 d x_i = s_i * (g_i - sum_j g_j s_j), g_i = 0 for experts not chosen
 *   softmax, renormalised   d x_j = q_j * (g_j - sum g q), q = softmax over the chosen
 *   sigmoid                 d x_j = g_j * s_j (1 - s_j)
 *   sigmoid, renormalised   d x_j = (g_j - sum g q) / (sum s) * s_j (1 - s_j), q = s / sum s
 * and 0 elsewhere.  Rows that a2av_route gives weights of 0 for want of scores get 0.
 *
 *  key_ptrs           as a2av_route wrote them.  A token with a key outside [0, E) gets a
 *                     gradient of 0 and A2AV_ERR_BAD_INDEX is recorded.
 *  d_weight_ptrs      HOST array of W: float [tokens][k].
 *  d_logits_ptrs      HOST array of W: [tokens][E] of the logits' type, written whole.
 * `route`'s groups, top_groups and group_top are checked but not used.
 */
int a2av_route_backward(a2av_handle *h, const a2av_route_t *route, const void *const *logits_ptrs,
                        const int64_t *tokens_per_rank, const int32_t *const *key_ptrs,
                        const float *const *d_weight_ptrs, void *const *d_logits_ptrs,
                        void *stream);

typedef enum {
  A2AV_ACT_NONE = 0,
  A2AV_ACT_RELU = 1,
  A2AV_ACT_GELU = 2, /* z * Phi(z), with the error function */
  A2AV_ACT_SILU = 3  /* z / (1 + exp(-z)) */
} a2av_act_t;

/* The shape of a2av_expert_matmul. */
typedef struct {
  int experts_per_peer; /* K; W * K <= A2AV_MAX_DISPATCH_KEYS */
  int64_t in_features;  /* D >= 1 */
  int64_t out_features; /* N >= 1 */
  int dtype;            /* A2AV_BF16 or A2AV_F16: rows, weights, bias, results */
  int activation;       /* a2av_act_t */
  int gated;            /* 0: Z = N; 1: Z = 2N, act(first half) * second half */
} a2av_expert_t;

/*
 * a2av_expert_matmul -- one product per expert over the rows that a dispatch
 * delivered, with bias, activation and residual in its epilogue:
 *
 *   z = x W_e^T + b_e                                [Z]
 *   y = act(z) + residual, or gated act(z[0..N)) * z[N..2N) + residual
 *
 * Peer p's rows are in the dispatch's order: source rank, then local expert;
 * group (r, e) has counts[r][p * K + e] rows, which follow the group before.
 * One rank with one expert is an ordinary linear layer.  Products are summed
 * in 32 bits; bias, activation and residual are applied in 32 bits and the
 * result is rounded once.  Rows of NaN stay within their own results.  An
 * activation at an infinity, and its slope there, is the limit.
 *
 *  rows_ptrs          HOST array of W: peer p's x, [rows_per_peer[p]][D].  Read only.
 *  rows_per_peer      HOST int64 [W], up to 2^31 - 1 together: the rows each peer's buffers hold.
 *                     Rows past the sum of its groups are neither used nor written.
 *  counts_dev         DEVICE int64 [W][W * K], as a2av_route writes it.
 *  weight_ptrs        HOST array of W: [K][Z][D].
 *  bias_ptrs          HOST array of W: [K][Z], or NULL (no bias).
 *  residual_ptrs      HOST array of W: [rows][N], or NULL.  May be out_ptrs.
 *  out_ptrs           HOST array of W: [rows][N], written.
 *  pre_ptrs           HOST array of W: [rows][Z], written with z rounded to dtype
 *                     (what the backward pass needs of an activation), or NULL.
 *
 * Device errors: A2AV_ERR_BAD_SPLITS when a count is negative or a peer's
 * groups have more rows than rows_per_peer: nothing is written.  A2AV_ERR_TIMEOUT
 * when a copy or a product has not come for about a second: results are not
 * complete.  (A call's own length has no limit.)  Host errors:
 * A2AV_ERR_INVALID_ARG, A2AV_ERR_UNSUPPORTED (W * K or rows above the limits,
 * D, N or Z above 2^24), A2AV_ERR_CUDA.
 */
int a2av_expert_matmul(a2av_handle *h, const a2av_expert_t *shape, const void *const *rows_ptrs,
                       const int64_t *rows_per_peer, const int64_t *counts_dev,
                       const void *const *weight_ptrs, const void *const *bias_ptrs,
                       const void *const *residual_ptrs, void *const *out_ptrs,
                       void *const *pre_ptrs, void *stream);

/*
 * a2av_expert_matmul_workspace_bytes -- device workspace that
 * a2av_expert_matmul_backward needs for W peers of `total_rows` rows together
 * (dz, where there is an activation or a gate, and what the groups have over
 * multiples of 64 rows); -1 for a shape or a count that would be rejected.
 */
int64_t a2av_expert_matmul_workspace_bytes(int world_size, const a2av_expert_t *shape,
                                           int64_t total_rows);

/*
 * a2av_expert_matmul_backward -- the gradients of a2av_expert_matmul.  With
 * dz = dy * act'(z) (gated: dz = [dy * z_2 * act'(z_1), dy * act(z_1)]):
 *
 *   d_rows = dz W_e      d_weights_e = dz_e^T x_e      d_bias_e = sum of dz_e's rows
 *
 * (the residual's gradient is dy itself).  dz is rounded to dtype, which the
 * tensor cores take, before the products (in f16 one above 65504 is infinite);
 * d_bias sums the rounded dz, in 32 bits.
 * An expert without rows gets gradients of 0.
 *
 *  rows_ptrs .. weight_ptrs   as in the forward call.
 *  pre_ptrs           what it saved; may be NULL for A2AV_ACT_NONE without gate.
 *  d_out_ptrs         HOST array of W: dy [rows][N].
 *  d_rows_ptrs        HOST array of W: [rows][D], or NULL (not wanted).
 *  d_weight_ptrs      HOST array of W: [K][Z][D], or NULL.
 *  d_bias_ptrs        HOST array of W: [K][Z], or NULL.
 *  workspace          DEVICE scratch, 256-byte aligned, at least
 *                     a2av_expert_matmul_workspace_bytes(W, shape, sum of rows_per_peer),
 *                     not shared with a call in flight (NULL for no rows at all).
 * Errors are those of the forward call.
 */
int a2av_expert_matmul_backward(a2av_handle *h, const a2av_expert_t *shape,
                                const void *const *rows_ptrs, const int64_t *rows_per_peer,
                                const int64_t *counts_dev, const void *const *weight_ptrs,
                                const void *const *pre_ptrs, const void *const *d_out_ptrs,
                                void *const *d_rows_ptrs, void *const *d_weight_ptrs,
                                void *const *d_bias_ptrs, void *workspace,
                                int64_t workspace_bytes, void *stream);

/*
 * a2av_combine_weighted -- the return path of a2av_dispatch with the routing
 * weights applied and each token's rows summed.  Items are (token t, choice
 * j), token-major: item i = t * k + j.  Item i's row is found as
 * a2av_combine_items finds it, peer = key / keys_per_peer, and
 *
 *   out[t] = residual[t] + sum_j weight[t][j] * row(t, j)
 *
 * summed in 32 bits in the order of j and rounded once.  With NULL weights
 * (all 1) this is the gradient of the dispatch.
 *
 *  keys_per_peer, topk, hidden, dtype   K, k, elements per row, a2av_dtype_t of rows.
 *  peer_ptrs          HOST array of W: peer p's rows [rows_per_peer[p]][hidden].  Read only.
 *  rows_per_peer      HOST int64 [W]: rows the peers' buffers hold; sum_r S[r][p] above
 *                     it is rejected on the device.
 *  in_splits_dev      DEVICE int64 [W][W]: S as the dispatch wrote it.
 *  key_ptrs, sorted_pos_ptrs   HOST arrays of W: int32 / int64 [tokens * k].
 *  weight_ptrs        HOST array of W: float [tokens][k], or NULL.
 *  tokens_per_rank    HOST int64 [W].
 *  residual_ptrs      HOST array of W: [tokens][hidden], or NULL.  May be out_ptrs.
 *  out_ptrs           HOST array of W: [tokens][hidden], written.
 *
 * One kernel, no workspace.  Device errors: an invalid S (a negative entry, or
 * more rows than a peer's buffer holds) records A2AV_ERR_BAD_SPLITS and nothing is
 * written; a token that has an item with a key or a position out of range is
 * not written and A2AV_ERR_BAD_INDEX is recorded, the others are.
 */
int a2av_combine_weighted(a2av_handle *h, int keys_per_peer, int topk, int64_t hidden, int dtype,
                          const void *const *peer_ptrs, const int64_t *rows_per_peer,
                          const int64_t *in_splits_dev, const int32_t *const *key_ptrs,
                          const int64_t *const *sorted_pos_ptrs,
                          const float *const *weight_ptrs, const int64_t *tokens_per_rank,
                          const void *const *residual_ptrs, void *const *out_ptrs, void *stream);

/*
 * a2av_combine_weighted_backward -- its gradients: the row of item (t, j) gets
 * weight[t][j] * dy[t], rounded once, and d_weight[t][j] = sum over the row of
 * dy[t] * row(t, j), in 32 bits.
 *
 *  peer_ptrs          the rows the forward call read; NULL when d_weight_ptrs is NULL.
 *  d_out_ptrs         HOST array of W: dy [tokens][hidden].
 *  d_peer_ptrs        HOST array of W: written in the peers' layout, or NULL.
 *  d_weight_ptrs      HOST array of W: float [tokens][k], written, or NULL.
 * A token with an invalid item is left out whole, as in the forward call.
 */
int a2av_combine_weighted_backward(a2av_handle *h, int keys_per_peer, int topk, int64_t hidden,
                                   int dtype, const void *const *peer_ptrs,
                                   const int64_t *rows_per_peer,
                                   const int64_t *in_splits_dev, const int32_t *const *key_ptrs,
                                   const int64_t *const *sorted_pos_ptrs,
                                   const float *const *weight_ptrs,
                                   const int64_t *tokens_per_rank, const void *const *d_out_ptrs,
                                   void *const *d_peer_ptrs, float *const *d_weight_ptrs,
                                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* A2AV_MOE_H_ */
