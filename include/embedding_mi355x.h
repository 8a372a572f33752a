/*
 * embedding_mi355x.h -- C ABI of an embedding table's three operations on
 * AMD Instinct MI355X (gfx950): the lookup of rows by token, its gradient, and
 * the Adam/AdamW step of the rows that tokens name, which takes that gradient
 * without writing it.  Exported by the library that adam_mi355x.h describes,
 * whose status codes, threading rules and adam_last_error() hold here too.
 *
 * Definitions, for a table of `rows` x `cols` and `tokens` tokens x_0, x_1, ..
 *   lookup:    out_i = scale * table[x_i]
 *   gradient:  d_r = scale * sum of grad_i over all i with x_i = r
 *   step:      adam_step's update of p, m, v (and the AMSGrad maximum) with
 *              g = d_r, for every row r that at least one token names; other
 *              rows and their state stay as they are (no decay of the moments
 *              or of the params: a step for sparse gradients)
 * A token outside [0, rows) is padding: its row of out is zero, and its row of
 * grad is not read.
 *
 * Numerics.  Sums are held in fp32, in an order that depends on the sizes and
 * the tokens only, so that a call repeated gives the same bits; the order is
 * not the tokens' own.  scale is applied to the whole sum, rounded once, and
 * a bf16 result is that fp32 value (plus the fp32 or bf16 value it is added to, in
 * another rounding) rounded to nearest even.  The step performs adam_step's
 * operations in its order; no moment is rounded for storage.
 */
#ifndef EMBEDDING_MI355X_H
#define EMBEDDING_MI355X_H

#include <stdint.h>

#include "adam_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

enum embedding_token_dtype { EMBEDDING_TOKENS_I32 = 0, EMBEDDING_TOKENS_I64 = 1 };

typedef struct {
    int64_t rows, cols;   /* of the table; each < 2^31 */
    int64_t tokens;       /* how many; < 2^31 */
    int64_t table_stride; /* elements from a row of the table (or of its gradient) to the next, >= cols */
    int64_t value_stride; /* elements from a token's row of out (>= cols) or grad (>= 0) to the next */
    int32_t table_dtype;  /* enum adam_grad_dtype: of the table, or of its gradient */
    int32_t value_dtype;  /* enum adam_grad_dtype: of out, or of grad */
    int32_t token_dtype;  /* enum embedding_token_dtype */
    float scale;          /* finite */
} embedding_shape;

/*
 * embedding_lookup: out's rows from the table, enqueued on hip_stream with no
 * allocation, copy or synchronization (it can be recorded into a graph).
 *   table, tokens: device memory, read only; out: device memory, which meets
 *   neither; each aligned to its element.
 * Errors (no work enqueued): EINVAL (NULL pointer where there is something to
 * do, a size or stride outside its domain or reaching beyond 2^60 elements,
 * an unknown dtype, a scale that is not finite, out meeting table or tokens),
 * EALIGN; EDEVICE if a launch fails.
 */
int embedding_lookup(const embedding_shape *shape, const void *table, const void *tokens, void *out, void *hip_stream);

/*
 * Bytes of device workspace that embedding_gradient and embedding_adam_step
 * take for these sizes (may be 0).  Pure host function; < 0 (EINVAL) for
 * sizes outside their domain.
 */
int64_t embedding_gradient_workspace_bytes(int64_t tokens, int64_t rows, int64_t cols);

/*
 * embedding_gradient: the whole table_grad, rows that no token names as zeros;
 * or with accumulate != 0 added to it, rows that no token names untouched.
 * Enqueued on hip_stream with no allocation, copy or synchronization (it can
 * be recorded into a graph).
 *   grad: device memory of value_dtype, row i at i * value_stride; tokens:
 *   device memory; both read only.  table_grad: device memory of table_dtype.
 *   workspace: device memory, 256-byte aligned, of at least
 *   embedding_gradient_workspace_bytes (NULL will do for 0), written by the
 *   call.  Calls that share one must be ordered on the device, and so must the
 *   replays of graphs that recorded one.
 *   table_grad and workspace meet nothing else of the call.
 * Errors (no work enqueued): as embedding_lookup, and EINVAL for a workspace too small.
 */
int embedding_gradient(const embedding_shape *shape, const void *grad, const void *tokens, void *table_grad,
                       int32_t accumulate, void *workspace, int64_t workspace_bytes, void *hip_stream);

/*
 * embedding_adam_step: the step on the rows that tokens name, over state
 * buffers the caller owns: those of adam_step_noalloc for the one tensor of
 * rows * cols elements with fp32 storage, so that both kinds of step may be
 * taken on them by turns.  Enqueued on hip_stream with no allocation, copy or synchronization;
 * recorded into a graph it repeats the call as recorded (same t and hyperparameters).
 *   shape: table_dtype ADAM_GRAD_F32, table_stride == cols, rows * cols < 2^32.
 *   layout: storage ADAM_STORE_F32, grad_dtype == shape->value_dtype; options
 *   may hold ADAM_OPT_AMSGRAD.
 *   table: device float, updated in place; grad, tokens, workspace: as for
 *   embedding_gradient.
 *   state: as adam_step_noalloc's, ADAM_BUF_M_F32, ADAM_BUF_V_F32 and with
 *   AMSGrad ADAM_BUF_VMAX_F32 being read, each buffer aligned to 16 bytes, as table is.
 *   hp: as adam_step's; its only flag here is ADAM_F_DECOUPLED_WD.  t counts the
 *   caller's steps, whichever rows they named.
 * Errors (no work enqueued): as embedding_gradient and adam_step_noalloc; EMODE for a
 * layout of another storage or gradient type.
 */
int embedding_adam_step(const embedding_shape *shape, float *table, const void *grad, const void *tokens,
                        void *const *state, const adam_hparams *hp, const adam_layout *layout, void *workspace,
                        int64_t workspace_bytes, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* EMBEDDING_MI355X_H */
