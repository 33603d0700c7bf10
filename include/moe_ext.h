/*
 * moe_ext.h -- C ABI of the operators around the sparse Mixture-of-Experts
 * layer of moe.h, in the same library (libmoe.so) and with the same problem
 * struct, status codes and conventions (device pointers, row-major contiguous,
 * 16-byte aligned; the caller owns every buffer; calls only enqueue on `stream`
 * and never synchronize; argument checks run on the host before anything is
 * enqueued, and on any error nothing is written).
 *
 * In addition, an output or workspace buffer of these calls must not overlap
 * any other buffer of the same call: such a call is refused with
 * MOE_ERR_INVALID_ARGUMENT. Calls may run at the same time when neither writes
 * what the other reads or writes; the library keeps no state between them.
 *
 * 8-bit rows. A row of K values is held as codes and scales:
 *   codes  moex_code_pitch(K) bytes, e4m3 (OCP "fn": bias 7, no infinity, 0x7F
 *          and 0xFF are NaN); positions past K hold zero
 *   scales moex_scale_pitch(K) bytes: byte b belongs to values 128 b .. 128 b + 127
 *          and holds e + 127 for the scale 2^e; bytes past the last block hold 0
 * A value is its code times its block's scale. e is the smallest integer with
 * max|v| <= 448 * 2^e over the block, kept in [-120, 120]; codes are rounded to
 * nearest even from the float32 value (moex_add_rmsnorm: from one of more bits). A power of two costs e4m3, a floating
 * format, no relative precision, dividing by it is exact, and the matrix cores
 * apply it while multiplying. A NaN or an infinity becomes a NaN code; an
 * infinity also raises its block's scale to 2^120.
 */
#ifndef MOE_MI355X_MOE_EXT_H_
#define MOE_MI355X_MOE_EXT_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one row's codes and scales for K values (host only). */
static inline size_t moex_code_pitch(int64_t K) { return (size_t)((K + 127) / 128 * 128); }
static inline size_t moex_scale_pitch(int64_t K) { return (size_t)((K + 2047) / 2048 * 16); }

/* Which entry point a workspace size is asked for. */
typedef enum {
  MOEX_STAGE_NORM_BACKWARD = 0,  /* moex_add_rmsnorm_backward */
  MOEX_STAGE_BALANCE = 1,        /* moex_balance_loss */
  MOEX_STAGE_FFN_FP8 = 2,        /* moex_grouped_ffn_fp8 */
  MOEX_STAGE_FORWARD_FP8 = 3,    /* moex_forward_fp8 */
  MOEX_STAGE_TRAIN_BALANCED = 4  /* moe_forward_train + moex_backward_balanced */
} moex_stage_t;

/* Workspace bytes that `stage` needs for problem `p` (host only, nothing is enqueued).
 * A call checks its workspace against the same figure. */
moe_status_t moex_workspace_size(const moe_problem_t* p, int32_t stage, size_t* bytes);

/* Root-mean-square norm in front of the layer, with the residual's addition
 * and an optional output in 8 bits. For every token, over d_model values:
 *   h = x + residual               (rounded to p->dtype; x itself without residual)
 *   r = 1 / sqrt(mean(h^2) + eps)  (float32, from the rounded h)
 *   y = h r gain
 *   x, residual  [T, d_model] of p->dtype; residual may be NULL
 *   gain         [d_model] of p->dtype
 *   h            [T, d_model] of p->dtype: written when residual is given (then
 *                required), NULL without residual
 *   y            [T, d_model] of p->dtype, or NULL
 *   y8, y_scale  8-bit rows of the unrounded y, both or neither
 *   rstd         [T] float32: r, which the backward pass takes, or NULL
 * At least one of y, y8 and rstd is given; eps is finite and not negative;
 * d_model <= 32768 (MOE_ERR_UNSUPPORTED beyond). T, d_model and dtype of p are
 * used; the other fields must form a valid problem. */
moe_status_t moex_add_rmsnorm(const moe_problem_t* p, const void* x, const void* residual, const void* gain, float eps,
                              void* h, void* y, void* y8, void* y_scale, float* rstd, void* stream);

/* Gradients of moex_add_rmsnorm, given dy = dL/dy and dh, the gradient that
 * reaches h along the residual stream (NULL: none). With z = h r, a = dy gain:
 *   dx    = r (a - z mean(a z)) + dh    [T, d_model] of p->dtype, the gradient
 *           of x and, equal to it, of the residual
 *   dgain = sum over tokens of dy z     [d_model] float32
 * h is what the forward call wrote (x without residual), rstd what it returned.
 * Sums are float32 in an order that depends on the problem alone.
 *   ws at least moex_workspace_size(p, MOEX_STAGE_NORM_BACKWARD) bytes */
moe_status_t moex_add_rmsnorm_backward(const moe_problem_t* p, const void* h, const void* gain, const float* rstd,
                                       const void* dy, const void* dh, void* dx, float* dgain, void* ws,
                                       size_t ws_bytes, void* stream);

/* 8-bit rows of x without a norm: x [T, d_model] of p->dtype. */
moe_status_t moex_quantize_rows(const moe_problem_t* p, const void* x, void* x8, void* x_scale, void* stream);

/* Load-balancing loss of a router, its per-expert counts and its gradient.
 * With n the tokens whose token_mask byte is not 0 (all T when token_mask is
 * NULL), p_t = softmax(logits_t) and, over those tokens,
 *   counts_e    = selections of expert e            [E] int32
 *   mean_prob_e = mean over t of p_te               [E] float32
 *   loss        = coef E sum_e counts_e / (n k) mean_prob_e
 *   dlogits_te  = (coef E / n) p_te (f_e - sum_e' f_e' p_te'),  f = counts / (n k)
 * (no gradient through the counts). Rows of masked tokens are not read into any
 * result and get dlogits 0; with n = 0 every output is 0. A logit of -infinity
 * is an expert of probability 0; a row whose logits are all -infinity counts
 * its selections, has probability 0 for every expert and gets dlogits 0.
 *   logits [T, E] float32, topk_idx [T, k] int32 (entries outside [0, E) are
 *   ignored), token_mask [T] bytes or NULL, loss [1] float32, counts and
 *   mean_prob as above, dlogits [T, E] float32 or NULL; coef and coef E finite
 *   ws at least moex_workspace_size(p, MOEX_STAGE_BALANCE) bytes
 * T, E and k of p are used; the other fields must form a valid problem. */
moe_status_t moex_balance_loss(const moe_problem_t* p, const float* logits, const int32_t* topk_idx,
                               const uint8_t* token_mask, float coef, float* loss, int32_t* counts, float* mean_prob,
                               float* dlogits, void* ws, size_t ws_bytes, void* stream);

/* moe_backward with the balance loss of the same router added to the layer's
 * loss: the gradients of moe_backward for dL/dy = dy plus those of
 * moex_balance_loss through the router, and that loss, its counts and mean_prob.
 * counts, mean_prob and dbias may be NULL, loss may not; coef as there. The limits
 * are those of moe_backward.
 *   ws the workspace of the matching moe_forward_train call, of at least
 *      moex_workspace_size(p, MOEX_STAGE_TRAIN_BALANCED) bytes */
moe_status_t moex_backward_balanced(const moe_problem_t* p, const void* x, const void* w_router, const void* W1,
                                    const void* W2, const void* dy, const uint8_t* token_mask, float coef, void* dx,
                                    void* dw_router, float* dbias, void* dW1, void* dW2, float* loss, int32_t* counts,
                                    float* mean_prob, void* ws, size_t ws_bytes, void* stream);

/* Expert weights in 8 bits, laid out once for the matrix cores. W1 [E, d_model,
 * d_expert] and W2 [E, d_expert, d_model] bf16 as the layer takes them. For a
 * weight of K contraction rows and N columns, with KB = moex_code_pitch(K) / 128:
 *   codes  [E][N / 32][KB][4][2][32][16]: byte b of (q, h, n) is the code of
 *          column 32 g + n at contraction position 128 kb + 32 q + 16 h + b
 *   scales [E][N / 32][KB][32]: one byte per column and block of 128 positions
 * (blocks of the 8-bit row format along the contraction; positions past K hold
 * zero codes). W1q, W1s, W2q, W2s hold moex_weight_bytes / moex_weight_scale_bytes
 * of (E, d_model, d_expert) and (E, d_expert, d_model). bf16 problems only;
 * MOE_ERR_UNSUPPORTED also when an expert's weight reaches 2^37 values. */
static inline size_t moex_weight_bytes(int64_t E, int64_t K, int64_t N) { return (size_t)(E * N) * moex_code_pitch(K); }
static inline size_t moex_weight_scale_bytes(int64_t E, int64_t K, int64_t N) {
  return (size_t)(E * N) * (moex_code_pitch(K) / 128);
}
moe_status_t moex_quantize_experts(const moe_problem_t* p, const void* W1, const void* W2, void* W1q, void* W1s,
                                   void* W2q, void* W2s, void* stream);

/* The expert FFNs with rows, hidden activations and weights in 8 bits: for
 * every expert e and row r in [offsets[e], offsets[e+1])
 *   H[r]      = 8-bit rows of GELU_tanh(X[r] W1[e])
 *   y_perm[r] = H[r] W2[e]                     [T*k, d_model] bf16
 * with X[r] row perm[r] of the T 8-bit rows x8 (perm [T*k] int32 in [0, T)), or
 * row r of T*k of them when perm is NULL. Sums are float32; a matrix instruction
 * cuts the products it adds at once some 2^-12 below the largest (measured: 1.6e-5
 * of a product in the root mean square on normal data). Hidden values within that of
 * the border of two codes take either; y_perm is off by 0.0018 to 0.0020 of itself in
 * the root mean square, 0.0017 of it the rounding to bf16.
 *   x8, x_scale  as moex_add_rmsnorm or moex_quantize_rows write them
 *   offsets      [E + 1] int32, non-decreasing, offsets[0] = 0, offsets[E] <= T*k
 *   rows of y_perm outside [0, offsets[E]) are left untouched
 *   ws at least moex_workspace_size(p, MOEX_STAGE_FFN_FP8) bytes
 * bf16 problems only; MOE_ERR_UNSUPPORTED also when the codes of x8, or those of
 * one expert's weight, reach 2 GiB, a width 2^22, or T*k rows of a width 2^42
 * values (in pieces of 32 rows of an expert and 64 columns, 2^31 of them). */
moe_status_t moex_grouped_ffn_fp8(const moe_problem_t* p, const void* x8, const void* x_scale, const int32_t* perm,
                                  const int32_t* offsets, const void* W1q, const void* W1s, const void* W2q,
                                  const void* W2s, void* y_perm, void* ws, size_t ws_bytes, void* stream);

/* The whole layer with 8-bit experts: moe_forward's routing of x (bf16), the
 * experts on the 8-bit rows, and the gate-weighted combine. x8 and x_scale are
 * the 8-bit rows of x (moex_add_rmsnorm writes both forms in one pass), or both
 * NULL: then the call makes them from x.
 *   ws at least moex_workspace_size(p, MOEX_STAGE_FORWARD_FP8) bytes */
moe_status_t moex_forward_fp8(const moe_problem_t* p, const void* x, const void* x8, const void* x_scale,
                              const void* w_router, const float* router_bias, const void* W1q, const void* W1s,
                              const void* W2q, const void* W2s, void* y, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_MOE_EXT_H_ */
