/*
 * moe_train.h -- C ABI of what trains the surroundings of the sparse
 * Mixture-of-Experts layer of moe.h: the layer's stages one by one with their
 * gradients, for experts of the caller's own; a dense projection beside the
 * routed experts; and the optimizer's step. Same library (libmoe.so), problem
 * struct, status codes and conventions (device pointers, row-major contiguous,
 * 16-byte aligned; the caller owns every buffer; calls only enqueue on `stream`
 * and never synchronize; argument checks run on the host before anything is
 * enqueued, and on any error nothing is written). As in moe_ext.h, an output or
 * workspace must not overlap any other buffer of the same call, and calls may
 * run at the same time when neither writes what the other reads or writes.
 */
#ifndef MOE_MI355X_MOE_TRAIN_H_
#define MOE_MI355X_MOE_TRAIN_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which entry point a workspace size is asked for. */
typedef enum {
  MOET_STAGE_DISPATCH = 0,        /* moet_dispatch */
  MOET_STAGE_LINEAR = 1,          /* moet_linear */
  MOET_STAGE_LINEAR_BACKWARD = 2  /* moet_linear_backward */
} moet_stage_t;

/* Workspace bytes that `stage` needs for problem `p` (host only, nothing is enqueued).
 * Any valid problem has a size, also one that the entry point itself does not support. */
moe_status_t moet_workspace_size(const moe_problem_t* p, int32_t stage, size_t* bytes);

/* ---- Rows sorted by expert and back, with weights, and the gradients.
 *
 * A selection (t, j) is entry j of token t's row of topk_idx; one whose entry is
 * outside [0, E) is dropped. Rows are ordered by expert, then by selection, so a
 * token that names an expert twice has two rows there. `inv` holds each
 * selection's row and -1 for a dropped one; entries outside [0, T*k) are taken
 * as dropped everywhere. Weights, gates and their gradients are float32 [T, k];
 * those of dropped selections are not read, and their gradient is 0. Rows of
 * T*k-row arrays that no selection names are neither read nor written. Products
 * and sums are float32 in an order that depends on the problem alone, rounded
 * once. T, d_model, E, k and dtype (float32 or bfloat16) of p are used; the other
 * field must form a valid problem. */

/* Dispatch: counts, offsets, perm and inv as moe_permute gives them, and
 *   x_perm[inv[t, j]] = weight[t, j] x[t]     (x[t] itself without weight)
 *   topk_idx [T, k] int32, weight [T, k] or NULL, x [T, d_model]
 *   counts [E], offsets [E + 1], perm [T*k], inv [T*k] int32: entries of perm
 *   from offsets[E] on are left untouched
 *   x_perm [T*k, d_model]
 *   ws at least moet_workspace_size(p, MOET_STAGE_DISPATCH) bytes */
moe_status_t moet_dispatch(const moe_problem_t* p, const int32_t* topk_idx, const float* weight, const void* x,
                           int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* x_perm, void* ws,
                           size_t ws_bytes, void* stream);

/* Its gradients, given dx_perm = dL/dx_perm:
 *   dx[t]         = residual[t] + sum over j of weight[t, j] dx_perm[inv[t, j]]
 *   dweight[t, j] = <x[t], dx_perm[inv[t, j]]>
 * residual [T, d_model] (what reaches x on other ways) or NULL; weight as in the
 * forward call; x and dweight both or neither. */
moe_status_t moet_dispatch_backward(const moe_problem_t* p, const void* dx_perm, const int32_t* inv, const void* x,
                                    const float* weight, const void* residual, void* dx, float* dweight,
                                    void* stream);

/* Combine: y[t] = residual[t] + sum over j of gate[t, j] y_perm[inv[t, j]], with
 * a residual [T, d_model] or NULL, and gates or NULL (all 1: for rows that were
 * weighted on the way to the experts). */
moe_status_t moet_combine(const moe_problem_t* p, const void* y_perm, const int32_t* inv, const float* gate,
                          const void* residual, void* y, void* stream);

/* Its gradients, given dy = dL/dy (which is the residual's own):
 *   dy_perm[inv[t, j]] = gate[t, j] dy[t]
 *   dgate[t, j]        = <dy[t], y_perm[inv[t, j]]>
 * gate as in the forward call; y_perm and dgate both or neither. Entries of inv
 * that name a row are distinct, as moet_dispatch gives them. */
moe_status_t moet_combine_backward(const moe_problem_t* p, const void* dy, const int32_t* inv, const void* y_perm,
                                   const float* gate, void* dy_perm, float* dgate, void* stream);

/* Gradient of moe_route's gates (softmax over all E logits, at the selected
 * experts; none through the choice): with q_t = softmax(logits_t) and dp_te the
 * sum of dgate[t, j] over the selections j of expert e,
 *   dlogits_te = q_te (dp_te - sum over e' of q_te' dp_te') + add_te
 *   logits [T, E] float32; topk_idx, dgate [T, k]; add [T, E] float32 (another
 *   loss's gradient of the logits) or NULL; dlogits [T, E] float32
 * A logit of -infinity is an expert of probability 0; a row of nothing else has
 * probability 0 for every expert. */
moe_status_t moet_gate_backward(const moe_problem_t* p, const float* logits, const int32_t* topk_idx,
                                const float* dgate, const float* add, float* dlogits, void* stream);

/* ---- A dense projection (a dense expert's, beside the routed ones), with K =
 * d_model and N = d_expert of p:
 *   u = x W + bias,  y = residual + act(u)
 *   x [T, K], W [K, N], bias [N] or NULL, residual [T, N] or NULL, y [T, N], all
 *   bfloat16; u [T, N] bfloat16 or NULL: u rounded, which the backward pass takes
 * y is made from u before it is rounded. Sums are float32. T, K, N are used; the
 * other fields must form a valid problem. bf16 problems only; MOE_ERR_UNSUPPORTED
 * also when x, W or the rows of y reach 2 GiB, or K or N 2^22 (256 rows of either
 * are reached with one 32-bit offset). moet_linear_backward has the same limits.
 *   ws at least moet_workspace_size(p, MOET_STAGE_LINEAR) bytes */
typedef enum {
  MOET_ACT_NONE = 0,
  MOET_ACT_GELU = 1, /* the tanh form, as the layer's experts */
  MOET_ACT_SILU = 2, /* u / (1 + e^-u) */
  MOET_ACT_RELU = 3  /* max(u, 0), slope 0 at 0 */
} moet_act_t;
moe_status_t moet_linear(const moe_problem_t* p, const void* x, const void* W, const void* bias, int32_t act,
                         const void* residual, void* u, void* y, void* ws, size_t ws_bytes, void* stream);

/* Its gradients, given dy = dL/dy (which is the residual's own): with dU = dy act'(u),
 *   dx = dU W^T [T, K],  dW = x^T dU [K, N],  dbias = sum over rows of dU [N]
 * all bfloat16, each may be NULL but not all; sums are float32. dU is rounded to
 * bfloat16 between the products (without activation it is dy). u as the forward call wrote it;
 * it may be NULL with MOET_ACT_NONE.
 *   ws at least moet_workspace_size(p, MOET_STAGE_LINEAR_BACKWARD) bytes */
moe_status_t moet_linear_backward(const moe_problem_t* p, const void* x, const void* W, const void* u, int32_t act,
                                  const void* dy, void* dx, void* dW, void* dbias, void* ws, size_t ws_bytes,
                                  void* stream);

/* ---- The optimizer's step over a list of tensors.
 *
 * Moments in 8 bits: 128 consecutive values of a tensor share a scale 2^e, e the
 * smallest integer with max <= top 2^e, kept in [-120, 120] and held as the byte
 * e + 127; m is held as e4m3 codes (top 448), v as e5m2 codes (top 57344, one
 * byte with the range that a square needs). They are rounded stochastically, or
 * the small part that a step changes of v would be lost at every step: with s
 * the spacing of codes at |x| and r the element's 16-bit random number, |x|
 * becomes s floor(|x| / s + r / 65536); a v that is not 0 is never rounded to 0,
 * since an update divides by its root. Element i of tensor j at step t draws, in 32-bit arithmetic,
 *   mix((lo32(i) + mix(seed + mix(0x9E3779B9 t + j))) ^ (0x9E3779B9 hi32(i)))
 *   mix(x): x ^= x >> 16; x *= 0x7FEB352D; x ^= x >> 15; x *= 0x846CA68B; x ^= x >> 16
 * whose low half is m's number and whose high half v's. What is not finite, or above
 * top 2^120, becomes a NaN code; max is that of the values that are not NaN. */
typedef struct {
  void* param;        /* [n] of param_dtype, updated */
  const void* grad;   /* [n] of grad_dtype */
  float* master;      /* [n], updated: the parameter in 32 bits that a bfloat16 one is rounded from; NULL for float32 */
  void* m;            /* [n] float32, or e4m3 codes */
  void* v;            /* [n] float32, or e5m2 codes */
  void* m_scale;      /* ceil(n / 128) bytes, or NULL: moments in 32 bits */
  void* v_scale;      /* the same; both or neither */
  int64_t n;          /* values; 0 leaves the tensor out, its pointers unread */
  int32_t param_dtype; /* a moe_dtype_t */
  int32_t grad_dtype;
  double lr_factor;    /* the tensor's own factor of lr */
  double weight_decay; /* decoupled: the parameter loses lr weight_decay of itself */
} moet_tensor_t;

typedef struct {
  double lr, beta1, beta2, eps;
  uint32_t seed; /* of the stochastic rounding */
} moet_adamw_t;

#define MOET_MAX_TENSORS 1024                 /* of one call */
#define MOET_GRAD_NORM_WS_BYTES 8704          /* workspace of moet_grad_norm */

/* One AdamW step, with t = counter[0] + 1 and g = grad grad_scale:
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   param -= lr lr_scale lr_factor (m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps) + weight_decay param)
 * from the moments before they are rounded, which are taken in 64 bits; the move is made
 * from their float32 values, so one whose v is past float32 moves by its decay alone.
 *   tensors  HOST array of count <= MOET_MAX_TENSORS entries, read during the call only
 *   opt      HOST pointer: finite lr >= 0, beta1 and beta2 in [0, 1), 1e-15 <= eps <= 1e15
 *   counter  [2] int32: steps taken, and 0, which the call uses. It is advanced by one
 *   lr_scale [1] float32 or NULL: a factor of lr that may change between replays of a captured step
 *   grad_scale [1] float32 or NULL; when it is NaN the step is left out: nothing is written
 * Lists of more than 48 tensors take a launch for every 48. MOE_ERR_UNSUPPORTED when
 * the list reaches 2^41 values. */
moe_status_t moet_adamw(const moet_tensor_t* tensors, int32_t count, const moet_adamw_t* opt, int32_t* counter,
                        const float* lr_scale, const float* grad_scale, void* stream);

/* Norm of all gradients of a list as one vector, and the factor that clips it:
 *   norm  [1] float32 = sqrt(sum of squares), added in 64 bits in a fixed order
 *   scale [1] float32 = min(1, max_norm / norm), NaN when a gradient is not finite
 *         (moet_adamw then leaves the step out); may be NULL
 * The factor is taken from the norm in 64 bits: a norm past float32 is written as
 * infinity and still has its factor. grad, grad_dtype and n of the tensors are used.
 * max_norm > 0, infinity included: norm and guard without clipping.
 *   ws  MOET_GRAD_NORM_WS_BYTES */
moe_status_t moet_grad_norm(const moet_tensor_t* tensors, int32_t count, double max_norm, float* norm, float* scale,
                            void* ws, size_t ws_bytes, void* stream);

/* Both in one call and with a launch less: moet_grad_norm, and moet_adamw with its
 * scale; norm and scale [1] float32 are written, scale may be NULL. */
moe_status_t moet_adamw_clipped(const moet_tensor_t* tensors, int32_t count, const moet_adamw_t* opt, int32_t* counter,
                                const float* lr_scale, double max_norm, float* norm, float* scale, void* ws,
                                size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_MOE_TRAIN_H_ */
