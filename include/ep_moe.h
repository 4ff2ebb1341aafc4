/*
 * ep_moe.h - the two ends of the dispatch / combine path in an MoE layer: the
 * router in front of it and the experts' products behind it (part of
 * libep.so; conventions, status codes and dtypes as in ep.h).
 *
 *   ep_route              logits -> topk_idx / topk_weights, which
 *                         ep_get_dispatch_layout, ep_dispatch and ep_combine take
 *   ep_balance_loss       load-balance loss, counts per expert and sequence,
 *                         and the loss's gradient for the probabilities
 *   ep_route_backward     gradient of the gates (ep_combine_backward's
 *                         grad_weights) and of the balance loss for the logits,
 *                         in one pass
 *   ep_w4_pack            4-bit weights into the tiles the product reads (once)
 *   ep_expert_product_w4  expert-major rows (ep_dispatch's recv_x and
 *                         recv_scales) times their experts' 4-bit weights,
 *                         plain or with a SwiGLU epilogue; its rows are what
 *                         ep_combine takes
 *
 * A layer's step: ep_route, ep_get_dispatch_layout, ep_dispatch,
 * ep_expert_product_w4 (gate and up, SwiGLU), ep_expert_product_w4 (down),
 * ep_combine.
 *
 * Every result is deterministic: sums have a fixed order.  Nothing is
 * allocated and nothing waits, so every call can be captured in a graph; the
 * counts and offsets stay on the device.
 */
#ifndef EP_MOE_H
#define EP_MOE_H

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a logit becomes a score. */
typedef enum ep_score {
  EP_SCORE_SOFTMAX = 0, /* over the token's experts */
  EP_SCORE_SIGMOID = 1  /* of each logit by itself */
} ep_score_t;

#define EP_MAX_GROUPS 64

typedef struct ep_router {
  int32_t num_tokens;  /* T >= 0; T * L <= 2^32 - 512 with L lanes per token: 8 up to
                          128 experts, 16 up to 256, 32 up to 512, else 64 */
  int32_t num_experts; /* 1 <= E <= EP_MAX_EXPERTS */
  int32_t num_topk;    /* 1 <= k <= min(E, EP_MAX_TOPK) */
  int32_t score;       /* ep_score_t */
  int32_t num_groups;  /* G: E % G == 0, 1 <= G <= EP_MAX_GROUPS; 1: no groups */
  int32_t topk_groups; /* groups kept per token, 1 <= topk_groups <= G,
                          topk_groups * (E / G) >= k */
  int32_t group_topn;  /* a group's score: the sum of its best 1 or 2 experts */
  int32_t normalize;   /* non-zero: a token's weights sum to `scale` */
  float scale;         /* finite factor of the weights */
} ep_router_t;

/*
 * Router: the k best experts of each token and their gates.
 *
 * With s_e the score of logit x_e and b the bias, the selection key of expert
 * e is s_e + b_e.  With G > 1 groups of E / G consecutive experts, a group's
 * key is the sum of its group_topn best keys, and the token keeps its
 * topk_groups best groups.  The slots are the k best keys left, in descending
 * order.  Ties go to the lowest index, of groups and of experts.  The order
 * is that of the keys in 64-bit arithmetic: keys that 32 bits cannot tell
 * apart are compared again in 64.  Without a bias and with group_topn 1 the
 * key is the logit itself, which orders alike.
 *
 *   weight of slot j = scale * s_j            (normalize == 0)
 *                      scale * s_j / sum s_i  (over the token's slots)
 *
 * The bias is no part of the weights (a correction of the load alone).  A
 * logit or bias of -inf is an expert that cannot be selected; a slot that
 * finds no expert is -1 with weight 0, as are all slots of a token that
 * token_mask leaves out (its logits enter no result, whatever they are).  A
 * token with a logit or key that is NaN or +inf gets no slot and sets
 * EP_STATUS_BIT_NONFINITE.
 *
 *   logits_dtype EP_DTYPE_F32 or EP_DTYPE_BF16
 *   logits       [T, E]
 *   bias         [E] fp32 or NULL
 *   token_mask   [T] uint8 or NULL: 0 = the token is not routed
 *   topk_idx     [T, k] int32 out;  topk_weights [T, k] fp32 out
 *   status       device int32, EP_STATUS_BIT_* are OR-ed into it
 */
ep_status_t ep_route(const ep_router_t *router, ep_dtype_t logits_dtype, const void *logits,
                     const float *bias, const uint8_t *token_mask, int32_t *topk_idx,
                     float *topk_weights, int32_t *status, hipStream_t stream);

/* Host only.  Device workspace of ep_balance_loss for num_seqs sequences. */
ep_status_t ep_balance_workspace_bytes(const ep_router_t *router, int32_t num_seqs,
                                       size_t *bytes_host);

/*
 * Load-balance loss over sequences of tokens, and what its gradient needs.
 * Sequence s is the tokens [seq_offsets[s], seq_offsets[s+1]).  A token
 * counts if it has a slot that is not -1; the others (padding) are neither
 * in the counts nor in N_s, their logits are in no sum, and their gradient is 0.
 *
 *   p[t, e]          softmax of the logits, or sigmoid scores over their sum
 *   counts[s, e]     slots of sequence s that hold expert e
 *   seq_tokens[s]    N_s, tokens that count
 *   mean_probs[s, e] P = sum_t p[t, e] / N_s                    (0 if N_s = 0)
 *   f[s, e]          E * counts[s, e] / (k * N_s)
 *   loss             coef / S' * sum_s sum_e f[s, e] P[s, e],  S' sequences with N_s > 0
 *   prob_grad[s, e]  coef * f[s, e] / (S' * N_s) = d loss / d p[t, e]  (0 if N_s = 0)
 *
 * The counts are constants to the gradient, as a count has none.  A score here
 * and in ep_route_backward is exp2(x log2 e) of fp32, off by
 * (1.23 |x| + 3) 2^-24 of itself (x the logit, of a softmax less the row's
 * largest), and 0 below 2^-126; sums over a tile of at most 256 tokens are fp32,
 * those over tiles fp64.
 *
 *   router       num_tokens, num_experts, num_topk and score are used
 *   topk_idx     [T, k] int32; an id outside [-1, E) counts as -1 and sets
 *                EP_STATUS_BIT_ROUTE
 *   seq_offsets  [num_seqs + 1] int32 device, ascending from 0 to T (num_seqs
 *                below 2^21), or NULL (then num_seqs is 1: all tokens).
 *                Offsets that are not that set EP_STATUS_BIT_SEQS, and the
 *                results are meaningless
 *   workspace    ep_balance_workspace_bytes() bytes, 256-byte aligned; used
 *                within the call only, by one call at a time
 *   counts, seq_tokens int32; mean_probs, prob_grad fp32; loss fp32 [1]
 */
ep_status_t ep_balance_loss(const ep_router_t *router, ep_dtype_t logits_dtype,
                            const void *logits, const int32_t *topk_idx,
                            const int32_t *seq_offsets, int32_t num_seqs, float coef,
                            void *workspace, size_t workspace_bytes, int32_t *counts,
                            int32_t *seq_tokens, float *mean_probs, float *prob_grad, float *loss,
                            int32_t *status, hipStream_t stream);

/*
 * Gradient for the logits of the gates and of the balance loss, in one pass:
 *
 *   grad_logits[t, e] = sum_j grad_weights[t, j] d topk_weights[t, j] / d x[t, e]
 *                     + grad_loss sum_e' prob_grad[s(t), e'] d p[t, e'] / d x[t, e]
 *
 * computed in fp32 and rounded once to the logits' type.  The choice of the
 * experts has no gradient, nor has the bias.  Slots of -1 take no part (their
 * grad_weights are not read into any result); a token with no slot gets a row
 * of zeros whatever its logits are.
 * An expert that a token's slots repeat (ep_route makes none; a layout rejects
 * them) counts as often, here as in ep_balance_loss; of three slots and more with
 * the same expert the order of the sum is not fixed.
 *
 *   router        the forward's (score, normalize and scale are used)
 *   topk_idx      [T, k] int32, the forward's; an id outside [-1, E) counts
 *                 as -1 and sets EP_STATUS_BIT_ROUTE
 *   grad_weights  [T, k] fp32, or NULL: no gradient of the gates
 *   prob_grad     [num_seqs, E] fp32 of ep_balance_loss, or NULL: no loss
 *   seq_offsets, num_seqs   as in ep_balance_loss (checked there; a token
 *                 outside every sequence gets no gradient of the loss); not
 *                 used without prob_grad
 *   grad_loss     device fp32 [1] or NULL for 1
 *   grad_logits   [T, E] out, of logits_dtype
 */
ep_status_t ep_route_backward(const ep_router_t *router, ep_dtype_t logits_dtype,
                              const void *logits, const int32_t *topk_idx,
                              const float *grad_weights, const float *prob_grad,
                              const int32_t *seq_offsets, int32_t num_seqs,
                              const float *grad_loss, void *grad_logits, int32_t *status,
                              hipStream_t stream);

/*
 * 4-bit weights of a set of experts: per expert `halves` matrices of
 * out_features x in_features (1, or 2 with swiglu: gate, then up), codes
 * q in 0..15, one bf16 scale and optionally one zero point 0..15 per row and
 * group of `group` consecutive columns:
 *     w[n, c] = scale[n, c / group] * (q[n, c] - zero[n, c / group]),  zero 8 if none
 */
typedef struct ep_w4 {
  int32_t num_experts;  /* >= 1, at most EP_MAX_EXPERTS (a rank's experts, or all) */
  int32_t in_features;  /* K: multiple of `group`, 32 <= K < 2^24 */
  int32_t out_features; /* N: 1 <= N < 2^20 */
  int32_t group;        /* 32, 64 or 128 */
  int32_t swiglu;       /* non-zero: two matrices, the product is silu(gate) * up */
} ep_w4_t;

/* Host only.  Sizes of the packed arrays: w_codes in bytes, w_scales in
 * values (w_zeros has as many). */
ep_status_t ep_w4_packed_sizes(const ep_w4_t *w4, int64_t *code_bytes_host,
                               int64_t *scale_values_host);

/*
 * Lays weights out for the product, once per model.  Rows are padded to 16
 * per matrix and columns to 128; a tile of 16 rows x 128 columns is 1024
 * consecutive bytes, 64 lanes x 4 words, in the order a matrix instruction
 * takes them: lane l, word w hold row l % 16, columns 32 w + 8 (l / 16) + 0..7,
 * column 2 p in bits 4 p..4 p + 3 and column 2 p + 1 in bits 16 + 4 p...
 *     w_codes  [experts, halves, ceil(N / 16), ceil(K / 128), 1024] bytes
 *     w_scales [experts, halves, ceil(N / 16), K / group, 16] bf16;  w_zeros alike, uint8
 * (One piece of 1 KB per wave and load reads at 6.8 to 7.1 TB/s; 16 rows x 64
 * bytes of row-major codes read at 3.7 to 5.6.)
 *
 *   codes   [experts, halves * N, K / 2] uint8, column 2 i in the low half of byte i
 *   scales  [experts, halves * N, K / group] bf16
 *   zeros   the same shape, uint8 0..15 (the high bits are dropped), or NULL
 */
ep_status_t ep_w4_pack(const ep_w4_t *w4, const uint8_t *codes, const uint16_t *scales,
                       const uint8_t *zeros, uint8_t *w_codes, uint16_t *w_scales,
                       uint8_t *w_zeros, hipStream_t stream);

/*
 * The experts' product on expert-major rows: for row r of expert e,
 *     y[r, n] = sum_c x[r, c] * w_e[n, c]
 * summed in fp32, and out[r, n] = bf16(y[r, n]), or with swiglu
 * bf16(silu(y_gate[r, n]) * y_up[r, n]).  Codes and rows enter the matrix
 * instructions exactly, scales are applied in fp32; the output's is the only
 * rounding below fp32.  Rows and scales may be any finite values: y is finite
 * where the sums of groups and of the experts' row are in fp32's range, and
 * each group adds an error of at most (1 + |scale|) 2^-138 at its lower end.
 *
 *   x_dtype       EP_DTYPE_BF16: x bf16 [capacity, K]
 *                 EP_DTYPE_FP8_E4M3: x uint8 [capacity, K] and x_scales fp32
 *                 [capacity, K / 128] (K % 128 == 0), as ep_dispatch writes
 *   w_codes, w_scales, w_zeros (or NULL)   from ep_w4_pack, codes 16-byte aligned
 *   expert_offsets         [num_experts] int32 device: expert e's first row
 *   num_tokens_per_expert  [num_experts] int32 device: its rows.  Both as
 *                 ep_get_dispatch_layout writes them (for one rank's experts,
 *                 a pointer to the rank's first).  Rows are cut off at
 *                 `capacity`, as dispatch's are; an expert whose offset or
 *                 count is negative has none.
 *   capacity      rows of x and out; (capacity / 64 + 1) * num_experts < 2^31 - 1
 *   out           bf16 [capacity, N], apart from x; only the experts' rows are
 *                 written.  A row of x (or a scale of it) that is not
 *                 finite makes its own outputs infinite or NaN, no other's
 */
ep_status_t ep_expert_product_w4(const ep_w4_t *w4, ep_dtype_t x_dtype, const void *x,
                                 const float *x_scales, const uint8_t *w_codes,
                                 const uint16_t *w_scales, const uint8_t *w_zeros,
                                 const int32_t *expert_offsets,
                                 const int32_t *num_tokens_per_expert, int64_t capacity,
                                 uint16_t *out, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_MOE_H */
