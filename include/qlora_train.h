/*
 * qlora_train.h -- C ABI of the operators that a training step of adapters needs beside its
 * linears (qlora.h): block norms with their gate and residual scale, the token
 * log-probabilities and the paired preference loss over a vocabulary, and the global gradient
 * norm with clipping.
 *
 * The conventions of qlora.h hold: row-major, device pointers unless stated otherwise, BF16 as
 * uint16_t bit patterns, a status per call, arguments checked before any launch, work enqueued
 * on `stream` without synchronization, no device memory allocated, and workspaces whose first
 * QLORA_WS_COUNTER_BYTES bytes are zero before their first use and left zero by every call (one
 * workspace serves calls of any kind; calls that share one must not overlap in time).  Every
 * call may be captured in a HIP graph.  Tensors need the alignment of their elements only, but for
 * the optimizer's buffers (qlora_adamw_step_clipped).  Sums are taken in a fixed order: the same
 * inputs give the same bits.
 */
#ifndef QLORA_NF4_TRAIN_H
#define QLORA_NF4_TRAIN_H

#include "qlora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the tensors that may have either. */
enum qlora_type { QLORA_BF16 = 0, QLORA_F32 = 1 };

/* The widest row of the norms. */
#define QLORA_NORM_MAX_WIDTH 8192

/* The boundary between two blocks of a residual stream, as one pass over its M rows of d:
 *     n  = y                        without post_norm,
 *          y / rms(y) * w_post      with it;   rms(v) = sqrt(mean(v^2) + eps)
 *     x' = res_scale * x + g n      the residual stream after the block
 *     h  = x' / rms(x') * w_pre     the next block's input
 * x' is rounded once to the stream's type; h is formed from x' before that rounding.
 * A row's sum of squares is FP32: exact to rounding while it and its mean lie within 1e-37 .. 1e38
 * (elements of about 1e-18 to 1e17 at any width); above that a row norms to zeros.
 *   x, x_out: [M, d] of `type` (QLORA_BF16 or QLORA_F32); x_out may be x, or NULL (not written).
 *   y: BF16 [M, d], the block's output, or NULL: the block adds nothing (then no post_norm,
 *      w_post or gate).  h: BF16 [M, d], or NULL: no norm before a next block.
 *   w_post, w_pre: BF16 [d], or NULL for ones.
 *   gate: BF16 [ceil(M / gate_rows), d], row m of the stream taking row m / gate_rows: one gate
 *      for all tokens (gate_rows = M), one per sequence of gate_rows tokens, or one per token
 *      (gate_rows = 1); NULL for ones.
 * No workspace.  Errors: INVALID_ARG (null or misaligned pointer, M outside [1, 2^24), both
 * outputs NULL, a weight or gate without its norm or block, gate_rows < 1 with a gate, res_scale
 * or eps not finite, eps < 0), BAD_SHAPE (d outside [1, QLORA_NORM_MAX_WIDTH]), UNSUPPORTED
 * (unknown type), HIP. */
int qlora_norm_residual_fwd(const void *x, const uint16_t *y, int64_t M, int64_t d, int type, int post_norm,
                            const uint16_t *w_post, const uint16_t *gate, int64_t gate_rows, const uint16_t *w_pre,
                            float res_scale, float eps, void *x_out, uint16_t *h, hipStream_t stream);

/* Its backward.  Given dh (BF16 [M, d], the gradient of h, or NULL: h was not used) and dx_out
 * ([M, d] of `type`, the gradient that reaches x' from later blocks, or NULL: none), with x_out
 * the stored x':
 *     a  = dh w_pre,  r_x = 1 / rms(x'),  r_y = 1 / rms(y),
 *     t  = dx_out + r_x a - x' r_x^3 mean(a x')                          the gradient of x'
 *     dx = res_scale t       dw_pre = sum over rows of dh x' r_x         dgate = sum of t n over a
 *     b  = t g w_post        dw_post = sum over rows of t g y r_y              gate row's rows
 *     dy = r_y b - y r_y^3 mean(b y)      (t g without post_norm)
 * dx: [M, d] of `type`, may be dx_out.  dy: BF16 [M, d].  dw_post, dw_pre: BF16 [d].  dgate: BF16,
 * the gate's shape.  Sums in FP32, rounded once.  Each output may be NULL (not computed);
 * outputs are overwritten.  x_out may be NULL without dh.
 * ws: qlora_norm_residual_workspace_size() bytes (gate_rows = 0 without a gate).
 * Errors: as the forward; INVALID_ARG also where dh and dx_out are both NULL, every output is
 * NULL, or an output has no operand (dy, dw_post or dgate without y, dw_post without post_norm,
 * dgate without a gate, dw_pre without dh); WORKSPACE. */
int qlora_norm_residual_workspace_size(int64_t M, int64_t d, int64_t gate_rows, size_t *ws_bytes);
int qlora_norm_residual_bwd(const void *x_out, const uint16_t *y, const uint16_t *dh, const void *dx_out, int64_t M,
                            int64_t d, int type, int post_norm, const uint16_t *w_post, const uint16_t *gate,
                            int64_t gate_rows, const uint16_t *w_pre, float res_scale, float eps, void *dx,
                            uint16_t *dy, uint16_t *dw_post, uint16_t *dgate, uint16_t *dw_pre, void *ws,
                            size_t ws_bytes, hipStream_t stream);

/* Log-probability of each row's label: logps[t] = x_t[label_t] - log sum_v exp(x_t[v]).
 *   logits: [rows, V] of `type`.  labels: int64 [rows]; a label outside [0, V) (-100, say)
 *   leaves its row out: its logits are not read and its logps is 0.  logps: FP32 [rows].
 * A logit of -inf has probability 0; NaN, +inf or a row of -inf alone gives NaN.
 * ws: qlora_logps_workspace_size() bytes.
 * Errors: INVALID_ARG (null or misaligned pointer, rows outside [1, 2^24)), BAD_SHAPE (V outside
 * [1, 2^22]), UNSUPPORTED (unknown type), WORKSPACE, HIP. */
int qlora_logps_workspace_size(int64_t rows, int64_t V, size_t *ws_bytes);
int qlora_token_logps(const void *logits, const int64_t *labels, int64_t rows, int64_t V, int type, float *logps,
                      void *ws, size_t ws_bytes, hipStream_t stream);

/* Preference loss of `pairs` pairs of answers (paired log ratios against a reference model)
 * and the gradient of the logits.  Sequences of S tokens: the chosen answers 0 .. pairs - 1,
 * then their rejected ones.
 *   logps  = token log-probabilities as qlora_token_logps, [2 pairs, S]
 *   D_i    = sum of logps - ref_logps over the tokens of sequence i that are counted
 *   z_p    = beta (D_p - D_{pairs + p})
 *   loss   = mean over p of (1 - e) softplus(-z_p) + e softplus(z_p),    e = label_smoothing
 *   dlogits[i, t, v] = c_i ([v = label] - softmax(logits[i, t])[v]), 0 for tokens left out,
 *     c_p = -c_{pairs + p} = grad_scale (beta / pairs) (sigmoid(z_p) + e - 1)
 *   logits [2 pairs, S, V] of `type`; labels int64 [2 pairs, S] (see qlora_token_logps; already
 *   shifted: row t's logits predict labels[t]); ref_logps FP32 [2 pairs, S], as
 *   qlora_token_logps gives them for the reference model, or NULL for zeros (read only where
 *   the label counts).  Log ratios are summed in FP64 token by token, so nothing is lost to
 *   the cancellation of two long sums.
 *   loss FP32 [1], log_ratios FP32 [2 pairs] (D), logps FP32 [2 pairs, S]: all written.
 *   dlogits: [2 pairs, S, V] of `type`, may be logits itself (then overwritten), or NULL: no
 *   gradient.  A sequence without counted tokens has D = 0 and no gradient.
 * Each counted token's gradient reads its pair's 2 S log ratios (16 S bytes): from S of about
 * V / 4 on that is more than its logits (BF16).
 * ws: qlora_preference_workspace_size() bytes.
 * Errors: INVALID_ARG (null or misaligned pointer, pairs outside [1, 2^22), 2 pairs S outside
 * [1, 2^24), beta, label_smoothing or grad_scale not finite, label_smoothing outside [0, 1],
 * dlogits overlapping logits in part), BAD_SHAPE (V), UNSUPPORTED (type), WORKSPACE, HIP. */
int qlora_preference_workspace_size(int64_t pairs, int64_t S, int64_t V, size_t *ws_bytes);
int qlora_preference_loss(const void *logits, const int64_t *labels, const float *ref_logps, int64_t pairs,
                          int64_t S, int64_t V, int type, float beta, float label_smoothing, float grad_scale,
                          float *loss, float *log_ratios, float *logps, void *dlogits, void *ws, size_t ws_bytes,
                          hipStream_t stream);

/* A list of gradient tensors, laid out once for the steps that follow: a table in the caller's
 * device memory.  The tensors' values may change between calls; their addresses and sizes may
 * not.  The struct is plain data of the caller's. */
typedef struct qlora_gradlist {
  void *table;
  int64_t chunks; /* entries of the table */
} qlora_gradlist_t;

/* Bytes of the table of `count` tensors of numel[i] elements.  Host only.
 * Errors: INVALID_ARG (count or a size negative, null pointer), BAD_SHAPE (over 2^38 elements or
 * so: 2^24 table entries). */
int qlora_gradlist_size(int count, const int64_t *numel, size_t *table_bytes);

/* Fill the table (16-byte aligned device memory of qlora_gradlist_size() bytes; may be NULL when
 * that is 0) and *list, on `stream`.
 *   grads[i]: device pointer to numel[i] elements of types[i] (QLORA_BF16 or QLORA_F32).
 *   out, out_types: where qlora_grad_clip writes tensor i, and in which type; out NULL (out_types
 *   ignored), or out[i] == grads[i] with the same type: in place.  The arrays are host memory,
 *   read before the call returns; an empty tensor's pointers may be NULL.  Otherwise no out
 *   tensor overlaps a gradient or another out tensor.
 * Errors: INVALID_ARG (null or misaligned pointer, count or a size negative, in place with
 * another type), BAD_SHAPE, UNSUPPORTED (unknown type), WORKSPACE (table too small), HIP. */
int qlora_gradlist_init(int count, const void *const *grads, const int32_t *types, const int64_t *numel,
                        void *const *out, const int32_t *out_types, void *table, size_t table_bytes,
                        qlora_gradlist_t *list, hipStream_t stream);

/* norm[0] = sqrt of the sum of the squares of all elements (FP32 [1]; squares and sums in FP64,
 * so neither overflows nor vanishes on the way).  An empty list gives 0.
 * ws: qlora_grad_workspace_size() bytes.  Errors: INVALID_ARG, WORKSPACE, HIP. */
int qlora_grad_workspace_size(const qlora_gradlist_t *list, size_t *ws_bytes);
int qlora_grad_norm(const qlora_gradlist_t *list, float *norm, void *ws, size_t ws_bytes, hipStream_t stream);

/* The norm as above, then out = c grad for every tensor, c = min(1, max_norm / (norm + 1e-6)) in
 * FP32, each product rounded once to the output's type.  Tensors clipped in place are not
 * touched when c is 1.  A norm of NaN makes every output NaN; an infinite one gives c = 0.
 * Errors: as qlora_grad_norm, INVALID_ARG also for max_norm not finite or negative. */
int qlora_grad_clip(const qlora_gradlist_t *list, float max_norm, float *norm, void *ws, size_t ws_bytes,
                    hipStream_t stream);

/* qlora_adamw_step on gradients clipped as they are read: grad is multiplied by
 * min(1, max_norm / (norm[0] + 1e-6)) in FP32 (no rounding to BF16 in between, nothing written).
 * As there, master, m and v are 16-byte aligned, grad and param 8-byte aligned: a slice of a flat
 * state starts at a multiple of four parameters.
 * norm: device FP32 [1], as qlora_grad_norm gives it.  When it is not finite the whole step
 * is skipped: master, m, v and param keep their values.
 * Errors: as qlora_adamw_step; INVALID_ARG also for norm NULL or max_norm not finite or negative. */
int qlora_adamw_step_clipped(float *master, float *m, float *v, const uint16_t *grad, uint16_t *param, int64_t n,
                             int64_t step, float lr, float beta1, float beta2, float eps, float weight_decay,
                             const float *norm, float max_norm, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_NF4_TRAIN_H */
