/*
 * ep_layer.h -- the rest of a mixture-of-experts layer around ep.h: the
 * router's choice and its gradient, and the experts' products in bf16 with
 * their gradients.  Same library, return codes and conventions as ep.h, which
 * this header includes: device pointers into memory the caller owns, work only
 * enqueued on `stream`, host-detectable errors before any HIP call, nothing
 * allocated, no synchronisation.  Every call may be captured into a HIP graph;
 * calls share no state, so two of them on different streams do not touch each
 * other's memory (each needs a workspace of its own while it runs).  No output
 * may overlap an input, another output or the workspace.
 *
 * Training, a layer runs (R = T * k receive rows):
 *
 *   ep_grouped_linear         router logits (one weight for all rows)
 *   ep_route                  the router's choice and weights
 *   ep_layout, ep_dispatch    token rows to expert rows
 *   ep_grouped_linear         gate and up products, SwiGLU in the epilogue
 *   ep_grouped_linear         down product
 *   ep_combine                the gate-weighted sum back in token order
 *
 * and back:
 *
 *   ep_combine_backward       gradients of the expert rows and routing weights
 *   ep_grouped_linear_wgrad   of the down weight
 *   ep_grouped_linear_dgrad   of the gate and up products, through SwiGLU
 *   ep_grouped_linear_wgrad   of the gate and up weight
 *   ep_grouped_linear_dgrad   of the receive rows
 *   ep_dispatch_backward      of the token rows
 *   ep_route_backward         of the router's logits, whose product has its
 *                             gradients from the same two calls
 */
#ifndef EP_LAYER_H
#define EP_LAYER_H

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of logits, logit gradients, product results and weight gradients */
enum { EP_BF16 = 0, EP_F32 = 1 };

/* score functions of the router */
enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 };

/* activations: of a product's result, and of the rows a product read */
enum { EP_ACT_NONE = 0, EP_ACT_SILU = 1, EP_ACT_GELU = 2, EP_ACT_SWIGLU = 3 };

#define EP_MAX_GROUPS 64

/*
 * Longest side of a weight (N or K), and the bound of N * K: offsets inside
 * an operand's tile and inside one expert's weight are 32-bit byte offsets.
 */
#define EP_LINEAR_MAX_SIDE (1 << 20)
#define EP_LINEAR_MAX_WEIGHT ((1 << 30) - 1)

/*
 * ep_route -- the k experts of each token and their weights, from the
 * router's logits l[t, :]:
 *   s[e] = softmax(l)[e], or 1 / (1 + exp(-l[e]))
 *   c[e] = s[e] + bias[e]                 (bias counts for the choice only)
 *   groups > 1: the experts are `groups` equal runs; a group's rank is the sum
 *     of its group_best largest c, and only the top_groups best groups stay
 *   the k experts of largest c among those that stay, in descending order
 *   w[j] = scale * s[e_j], divided by the sum of the k chosen s if renormalize
 * Equal c (and equal group ranks) go to the lower index.  The comparisons are
 * those of exact scores: without a bias the logits themselves are compared,
 * and sums that float32 cannot tell apart are compared in float64.  The
 * weights are float32; a renormalised weight is formed without passing through
 * scores that underflow, so logits of -200 still share their weight.
 * A NaN counts as larger than any number (c is NaN with its logit or bias).  The
 * weight of a NaN logit is NaN, and so are those divided by a sum with it and
 * every weight of a softmax over a row that holds a NaN or +infinity.  A logit of -infinity has score 0 and weight 0 (a masked
 * expert).  Without a bias it is chosen last, and a row of nothing else gets the
 * lowest indices; with one it is compared by its bias alone.  The chosen indices
 * are distinct and in range whatever the logits hold.
 *   logits     [T, E] of logits_type (EP_BF16 or EP_F32), aligned to its element
 *   bias       float32 [E] or NULL
 *   topk_idx   int32 [T, k],  topk_w float32 [T, k]: as ep_layout and
 *              ep_combine take them
 * Limits: 1 <= E <= EP_MAX_EXPERTS, 1 <= k <= EP_MAX_TOPK, T * k and T * E <=
 * EP_MAX_ENTRIES; groups divides E, 1 <= groups <= EP_MAX_GROUPS, 1 <=
 * top_groups <= groups, k <= top_groups * (E / groups), group_best 1 or 2 and
 * at most E / groups; scale finite.
 * The compute-unit budget does not apply to the calls of this header; a
 * CU-masked stream does.
 */
int ep_route(const void* logits, int logits_type, int T, int E, int score, const float* bias, int groups,
             int top_groups, int group_best, int k, int renormalize, float scale, int32_t* topk_idx, float* topk_w,
             void* stream);

/*
 * ep_route_backward -- the gradient of ep_route's weights to the logits, with
 * dw the gradient of topk_w (ep_combine_backward makes it).  The choice itself
 * has no gradient, the bias none either.  With p[j] = s[e_j], divided by the
 * sum of the chosen s if renormalize, and D = sum_j p[j] * dw[j]:
 *   renormalize, softmax   dl[e_j] = scale * p[j] * (dw[j] - D)
 *   renormalize, sigmoid   dl[e_j] = scale * p[j] * (1 - s[e_j]) * (dw[j] - D)
 *   else, sigmoid          dl[e_j] = scale * s[e_j] * (1 - s[e_j]) * dw[j]
 *   else, softmax          dl[e]   = scale * s[e] * ([e = e_j] dw[j] - D)
 * and zero elsewhere (the last has a gradient for every expert).
 *   logits     [T, E] of logits_type, those that ep_route read
 *   topk_idx   int32 [T, k] from ep_route; an entry outside [0, E) is left out
 *              of every sum, and of an index listed twice both entries count
 *   dw         float32 [T, k]
 *   dlogits    [T, E] of dlogits_type, every value written
 * Float32 throughout, rounded once.  Limits as ep_route.
 */
int ep_route_backward(const void* logits, int logits_type, int T, int E, int score, const int32_t* topk_idx, int k,
                      int renormalize, float scale, const float* dw, void* dlogits, int dlogits_type, void* stream);

/*
 * ep_grouped_linear -- the rows of each expert times that expert's weight,
 * with what follows it:
 *   z[r, n] = sum_i a[r, i] * b[e, n, i] + bias[e, n]      (float32)
 *   y[r, :] = act(z[r, :]) + residual[r, :]                (rounded once)
 *   pre[r, :] = z[r, :] in bf16, for ep_grouped_linear_dgrad
 * for every row r of expert e, offsets[e] <= r < offsets[e + 1].  act:
 *   EP_ACT_NONE    z
 *   EP_ACT_SILU    z / (1 + exp(-z))
 *   EP_ACT_GELU    z * (1 + erf(z / sqrt 2)) / 2
 *   EP_ACT_SWIGLU  silu(z[r, i]) * z[r, N/2 + i], i < N/2: N/2 gate rows, then
 *                  N/2 up rows in b; y has N/2 values a row
 *   a         bf16 [rows, K], K % 8 == 0
 *   offsets   int32 [E + 1] from ep_layout, non-decreasing; they are clamped to
 *             [0, rows], so no value reaches outside the buffers.  NULL with
 *             E == 1: one weight for all rows (a router, a shared expert)
 *   b         bf16 [E, N, K], N % 8 == 0 (swiglu: N % 16 == 0)
 *   bias      float32 [E, N] or NULL
 *   residual  bf16 [rows, N or N/2] or NULL
 *   y         [rows, N or N/2] of y_type; rows that no expert holds (past
 *             offsets[E]) are neither read nor written
 *   pre       bf16 [rows, N] or NULL
 *   workspace ep_grouped_linear_workspace_bytes(...) bytes, 16-byte aligned,
 *             or NULL where that is 0 (it is where there are rows enough for
 *             every compute unit; else sums along K are cut and joined).  At
 *             most 64 MiB, and its contents need not be kept or cleared.
 * a, b, residual, y and pre are 16-byte aligned, bias 4-byte.  Limits: 1 <= E <=
 * EP_MAX_EXPERTS, 0 <= rows <= EP_MAX_ENTRIES, N and K <= EP_LINEAR_MAX_SIDE,
 * N * K <= EP_LINEAR_MAX_WEIGHT, and 2^30 tiles of 128 x 256 results.  rows ==
 * 0 enqueues nothing.  Sums are taken in an order that the sizes fix: equal
 * calls give equal bits.
 */
size_t ep_grouped_linear_workspace_bytes(int64_t rows, int K, int E, int N);
int ep_grouped_linear(const void* a, int64_t rows, int K, const int32_t* offsets, int E, const void* b,
                      const float* bias, int N, int act, const void* residual, void* y, int y_type, void* pre,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * ep_grouped_linear_dgrad -- the gradient of such a product to its rows, and
 * on through the activation that made those rows:
 *   d[r, i] = sum_n dy[r, n] * b[e, n, i]                  (float32)
 *   dx[r, i] = act'(pre[r, i]) * d[r, i]                   (rounded once)
 * EP_ACT_NONE: dx = d.  EP_ACT_SWIGLU: dx and pre have 2 K values a row,
 *   dx[r, i]     = silu'(pre[r, i]) * pre[r, K + i] * d[r, i]
 *   dx[r, K + i] = silu(pre[r, i]) * d[r, i]
 *   dy        bf16 [rows, N]
 *   offsets, b, N, K, E and rows as for ep_grouped_linear
 *   pre       bf16 [rows, K or 2 K], NULL with EP_ACT_NONE: the `pre` of the
 *             product whose result this product read
 *   dx        bf16 [rows, K or 2 K]; rows that no expert holds are neither read
 *             nor written
 *   workspace ep_grouped_linear_dgrad_workspace_bytes(...) bytes
 * The gradient of a residual is dy itself.  Alignment and limits as above.
 */
size_t ep_grouped_linear_dgrad_workspace_bytes(int64_t rows, int K, int E, int N);
int ep_grouped_linear_dgrad(const void* dy, int64_t rows, int N, const int32_t* offsets, int E, const void* b, int K,
                            int act, const void* pre, void* dx, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * ep_grouped_linear_wgrad -- its gradients to the weights and the bias:
 *   db[e, n, i]  = sum of dy[r, n] * a[r, i] over the rows r of expert e
 *   dbias[e, n]  = sum of dy[r, n] over them               (both float32 sums)
 * An expert without rows gets zeros.
 *   dy        bf16 [rows, N],  a bf16 [rows, K]
 *   db        [E, N, K] of db_type
 *   dbias     float32 [E, N] or NULL
 *   workspace ep_grouped_linear_wgrad_workspace_bytes(...) bytes
 * rows == 0 writes zeros (dy and a may be NULL).  Alignment and limits as
 * above.
 */
size_t ep_grouped_linear_wgrad_workspace_bytes(int64_t rows, int K, int E, int N);
int ep_grouped_linear_wgrad(const void* dy, const void* a, int64_t rows, int N, int K, const int32_t* offsets, int E,
                            void* db, int db_type, float* dbias, void* workspace, size_t workspace_bytes,
                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_LAYER_H */
