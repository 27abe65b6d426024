/*
 * qlora_adapters.h -- C ABI of the frozen linear with many low-rank adapters (each row of the
 * batch names its own), of the dropout on the adapters' input, and of dropout on its own.
 *
 * The conventions of qlora.h hold: row-major, device pointers unless stated otherwise, BF16 as
 * uint16_t bit patterns, a status per call, arguments checked before any launch, work enqueued
 * on `stream` without synchronization, no device memory allocated, and workspaces whose first
 * QLORA_WS_COUNTER_BYTES bytes are zero before their first use and left zero by every call (one
 * workspace serves calls of any kind; calls that share one must not overlap in time, and graphs
 * captured with one must not run at once).  Outputs overlap no input unless stated otherwise.
 * Every call may be captured in a HIP graph.  Sums are taken in a fixed order: the same inputs
 * give the same bits.
 *
 * Dropout masks come from a counter-based generator and are never stored: Philox4x32 with ten
 * rounds ("Parallel random numbers: as easy as 1, 2, 3", Salmon et al. 2011).  `rng` is device
 * memory that holds two 64-bit words, seed and offset, read when the kernels run (so a captured
 * graph takes whatever they hold at each replay).  Element e of a tensor, counted from its start
 * row by row, is kept when
 *     h(e) >= t,   t = floor(p 65536 + 1/2),
 * where h(e) is half e % 8 (low halves first) of the four words that the generator gives for
 * the counter (e / 8, offset) under the key `seed`; kept elements are multiplied by
 * 65536 / (65536 - t), dropped ones are zero whatever they held.  Calls with the same seed and
 * offset drop the same places: give each use an offset of its own, and the backward that of its
 * forward.
 */
#ifndef QLORA_NF4_ADAPTERS_H
#define QLORA_NF4_ADAPTERS_H

#include "qlora.h"
#include "qlora_train.h" /* enum qlora_type */

#ifdef __cplusplus
extern "C" {
#endif

#define QLORA_MAX_ADAPTERS 4096

/* The adapters of one linear [d_out, d_in], laid out once for the calls that follow: a table in
 * the caller's device memory, written on the stream that qlora_adapters_init is given: calls on
 * another stream wait for that first, and the table stays until the last call, or replay of a
 * captured one, has run.  The tensors' values may change between calls; their addresses and
 * ranks may not.  The struct is plain data of the caller's. */
typedef struct qlora_adapters {
  void *table;
  int64_t d_out, d_in;
  int32_t count;
  int32_t max_rank;
  int32_t whole; /* 1: every rank is a multiple of 8 */
  int32_t grads; /* 1: every adapter has its gradients */
} qlora_adapters_t;

/* Bytes of the table of `count` adapters.  Host only.  Errors: INVALID_ARG (null output, count
 * outside [1, QLORA_MAX_ADAPTERS]). */
int qlora_adapters_size(int count, size_t *table_bytes);

/* Fill the table (16-byte aligned device memory of qlora_adapters_size() bytes) and *set, on
 * `stream`.  For i < count (host arrays, read before the call returns):
 *   A[i] [r[i], d_in], B[i] [d_out, r[i]]: device BF16 adapters, 16-byte aligned (B[i] by its
 *   elements only where r[i] is no multiple of 8); alpha[i]: the branch is scaled by alpha / r.
 *   dA, dB: device BF16 of the same shapes that qlora_adapters_bwd writes, aligned by their
 *   elements; both NULL for a set that is never trained.  They overlap neither each other nor any
 *   operand of the calls (not checked here).
 * Errors: INVALID_ARG (null or misaligned pointer, count, r outside [1, 128], alpha not finite),
 * BAD_SHAPE (as qlora.h), WORKSPACE (table NULL or too small), HIP. */
int qlora_adapters_init(int count, const uint16_t *const *A, const uint16_t *const *B, const int32_t *r,
                        const float *alpha, uint16_t *const *dA, uint16_t *const *dB, int64_t d_out, int64_t d_in,
                        void *table, size_t table_bytes, qlora_adapters_t *set, hipStream_t stream);

/* Columns of T (below): the set's largest rank, rounded up to a multiple of 8. */
int qlora_adapters_t_width(const qlora_adapters_t *set, int64_t *width);

/* Workspace bytes of qlora_adapters_fwd (QLORA_OP_FWD) or qlora_adapters_bwd (QLORA_OP_BWD).
 * Host only.  Errors: INVALID_ARG, BAD_SHAPE, UNSUPPORTED. */
int qlora_adapters_workspace_size(int op, int64_t M, const qlora_adapters_t *set, int dq_format, size_t *ws_bytes);

/* Y[m] = X[m] w_hat^T + s_a T[m] B_a^T,   T[m] = drop(X[m]) A_a^T,   a = ids[m], s_a = alpha_a / r_a
 * ("QLoRA -- Fine-Tuning a 65B Model on One GPU", "Prerequisite: LoRA's low-rank update": the
 * base is shared and frozen, an adapter is a small pair of matrices beside it).  w_hat is the
 * BF16 weight that qlora_dequantize gives; sums and T are FP32, Y is rounded once.
 *   X [M, d_in], Y [M, d_out]: device BF16, 16-byte aligned.
 *   ids: device int32 [M], the adapter of each row, in any order; a number outside [0, count)
 *        (-1, say) leaves its row with the base product only.  NULL: adapter 0 for all rows.
 *   dropout: p in [0, 1); 0 drops nothing and rng is not read.  It applies to the adapters'
 *        input only, to X as a [M, d_in] tensor.  rng: device uint64[2], 8-byte aligned.
 *   T_save: device FP32 [M, t_width], 16-byte aligned, receives T for the backward (zeros past a
 *        row's rank and for rows without an adapter); may be NULL.
 * A row's result depends on its own adapter only: values of others that are not finite stay
 * with the rows that name them.  Infinite operands give the infinities and NaN that the formulas
 * give, here and in the backward (a T or G past BF16's largest, 3.39e38, counts as infinite).
 * ws: qlora_adapters_workspace_size(QLORA_OP_FWD) bytes.
 * Errors: INVALID_ARG (null or misaligned pointer, Y or T_save overlapping X, ids, rng or each other,
 * M outside [1, 2^23], dropout outside [0, 1) or so near 1 that t would be 65536), BAD_SHAPE (also where
 * the weight's shape is not the set's), UNSUPPORTED, WORKSPACE, HIP. */
int qlora_adapters_fwd(const qlora_nf4dq_t *Wq, const qlora_adapters_t *set, const uint16_t *X, int64_t M,
                       const int32_t *ids, float dropout, const uint64_t *rng, uint16_t *Y, float *T_save, void *ws,
                       size_t ws_bytes, hipStream_t stream);

/* Its backward ("QLoRA -- Fine-Tuning a 65B Model on One GPU", "Where the gradients actually
 * go").  With G[m] = dY[m] B_a (FP32), k the mask and c its scale:
 *   dX[m] = dY[m] w_hat + s_a c k[m] * (G[m] A_a)           [M, d_in] BF16, or NULL: not computed
 *   dA_a  = s_a sum over the rows of a of G[m]^T drop(X[m])     [r_a, d_in]
 *   dB_a  = s_a sum over the rows of a of dY[m]^T T[m]          [d_out, r_a]
 * dA and dB go to the set's gradient tensors and are overwritten (zeros where no row names the
 * adapter).  dY [M, d_out], X [M, d_in], dX: device BF16, 16-byte aligned.  T_saved: the
 * forward's, or NULL to recompute it.  dropout and rng as in the forward.
 * ws: qlora_adapters_workspace_size(QLORA_OP_BWD) bytes.
 * Errors: as the forward, INVALID_ARG also for a set without gradients and for dX overlapping X, dY,
 * T_saved, ids or rng. */
int qlora_adapters_bwd(const qlora_nf4dq_t *Wq, const qlora_adapters_t *set, const uint16_t *X, const uint16_t *dY,
                       int64_t M, const int32_t *ids, float dropout, const uint64_t *rng, const float *T_saved,
                       uint16_t *dX, void *ws, size_t ws_bytes, hipStream_t stream);

/* out = residual + drop(x) over n elements (residual NULL: drop(x)).  The gradient of x is
 * qlora_dropout of out's gradient with the same p, rng and n, without the residual.
 *   x of x_type; residual and out of out_type (QLORA_BF16 or QLORA_F32), aligned by their
 *   elements.  out may be residual, and x where the types agree; otherwise they do not overlap.
 *   One FP32 fused multiply-add an element, rounded once to out_type.  n == 0 is a no-op.
 * No workspace.  Errors: INVALID_ARG (n negative or over 2^40, null or misaligned pointer,
 * dropout as above, partial overlap, out over rng), UNSUPPORTED (unknown type), HIP. */
int qlora_dropout(const void *x, int x_type, int64_t n, float dropout, const uint64_t *rng, const void *residual,
                  void *out, int out_type, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_NF4_ADAPTERS_H */
