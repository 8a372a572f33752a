/*
 * muon_mi355x.h -- C ABI of the Muon parameter step for AMD Instinct MI355X
 * (gfx950): momentum kept in fp32, bf16 or 8 bits, orthogonalised by
 * Newton-Schulz products, applied to fp32 params; and of the
 * orthogonalisation on its own.  Exported by the library that
 * adam_mi355x.h describes, whose status codes, threading rules and
 * adam_last_error() hold here too.  Matrices go through muon_step, the other
 * params (biases, norms, embeddings) through adam_step.
 *
 * Numerics.  The momentum is Adam's first moment, laid out and decoded as
 * adam_mi355x.h defines it (fp32, each operation rounded once; g widened
 * exactly from bf16):
 *   m = fma(beta, m_old, (1-beta)*g)
 *   u = fma(beta, m, (1-beta)*g) with MUON_F_NESTEROV, else m
 * from the stored m_old; u takes the new m before it is rounded for storage.
 * 8-bit storage: per 2048-element block of the flattened matrix the scale is
 * A = max |m| (a block with A < 2^-112 stores zero codes and scale 0); codes
 * are int8 in [-127, 127], |m| * fl(127 * fl(1/A)) rounded to nearest even, or
 * stochastically with the draws adam_step takes for its first moment (whose
 * encoder multiplies by fl(127/A): next to a rounding border the two may
 * differ by a code).
 *   X_0 = u / (|u|_F + eps), transposed if it has more rows than columns
 *   X_k = (a_k I + b_k A + c_k A^2) X_(k-1),  A = X_(k-1) X_(k-1)^T,  k = 1..steps
 *   p = fma(-lr*s, O, p*(1 - lr*wd)),  O = X_steps, transposed back
 * with s by enum muon_scale.  The norm is summed in fp64.  The products run
 * on the fp16 matrix units with fp32 sums: each factor is held as two fp16
 * values (high part and remainder, 22 bits; X and A scaled by 2^10, the
 * polynomial by 2^8, remainders by 2^11 besides) and three of the four partial
 * products are summed, so that O is about as far from the exact result as a
 * computation in fp32 is (at most some six times as far, where that one loses
 * almost nothing).  Entries of X below 2^-24, as one entry or column with nearly
 * all of the norm leaves the others, have an error of 2^-46 instead of 22 bits,
 * and below 2^-33 those of X_0 from a bf16 matrix one of 2^-40; the
 * iterations may grow either by the product of the |a_k|.
 * Iterations of larger matrices may be taken two or three at a time, as one
 * polynomial in the first one's A.  A bf16 output is the fp32 result rounded
 * once, to nearest even.
 * A matrix whose u is all zero gives O = 0; one with a NaN or an infinity
 * gives NaN in all of O (and in the params; the stored momentum of that
 * matrix is then unspecified).  Other matrices of the call are not affected.
 *
 * Range.  Coefficients are those of a polynomial that keeps singular values
 * below about 1.2 (as the default 3.4445, -4.7750, 2.0315 does).  If it does
 * not, and an entry of X or A reaches 64 or one of the polynomial's 256, that
 * matrix's result is NaN.
 */
#ifndef MUON_MI355X_H
#define MUON_MI355X_H

#include <stdint.h>

#include "adam_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct muon_state muon_state; /* opaque; owns the momentum and the workspace */

enum muon_storage {
    MUON_STORE_BF16 = 1, /* m: bf16 (round to nearest even) */
    MUON_STORE_Q8 = 2,   /* m: int8 [-127,127], fp32 scale per block */
    MUON_STORE_F32 = 3   /* m: fp32 */
};

enum muon_flags {
    MUON_F_NESTEROV = 1u,
    MUON_F_STOCHASTIC = 2u /* 8-bit storage only: Philox stochastic rounding */
};

enum muon_scale {
    MUON_SCALE_NONE = 0,     /* s = 1 */
    MUON_SCALE_SPECTRAL = 1, /* s = sqrt(max(1, rows / cols)) */
    MUON_SCALE_RMS = 2       /* s = 0.2 sqrt(max(rows, cols)): updates of about AdamW's size */
};

#define MUON_MAX_STEPS 16 /* iterations per call */

typedef struct {
    int32_t storage;    /* enum muon_storage */
    int32_t grad_dtype; /* enum adam_grad_dtype */
    int32_t block_size; /* must be ADAM_BLOCK_SIZE */
    uint32_t options;   /* must be 0 */
} muon_layout;

/* The Newton-Schulz iteration. */
typedef struct {
    int32_t steps;             /* 1 .. MUON_MAX_STEPS */
    float eps;                 /* > 0, finite: added to the norm */
    const float *coefficients; /* host, 3 * steps values a_1, b_1, c_1, a_2, .., each in [-64, 64];
                                  NULL: the default triple in every iteration */
} muon_iteration;

typedef struct {
    float lr;           /* >= 0, finite */
    float momentum;     /* beta, in [0, 1) */
    float weight_decay; /* >= 0, finite; decoupled */
    int32_t scale;      /* enum muon_scale */
    int64_t t;          /* 1-based step number (stochastic rounding's counter) */
    uint32_t flags;     /* enum muon_flags */
    uint32_t reserved;  /* must be 0 */
    uint64_t seed;      /* Philox key for stochastic rounding */
    muon_iteration iteration;
} muon_hparams;

/*
 * Bytes of momentum for a list of rows[k] x cols[k] matrices:
 *   sum_k pad16(rows*cols) * e + blocks * s, (e, s) = (4, 0) for F32, (2, 0)
 *   for BF16, (1, 4) for Q8.
 * muon_state_workspace_bytes: the device workspace that a state of this list
 * holds beside it (the factors of the products, for a part of the list at a
 * time: 16 bytes per element of the largest part and 8, 16 or 20, as iterations
 * are taken one, two or three at a time, per element of its square factors,
 * dimensions rounded up to tiles, and up to 64 MB for the parts of split
 * products; 4 bytes per element of matrices of up to 64 x 768, which
 * take no factors in memory).
 * Pure host functions.  Return < 0 (an adam_status) on bad arguments:
 * n_tensors < 0, rows or cols NULL with n_tensors > 0, a dimension < 0 or
 * >= 2^21, rows*cols >= 2^32, layout NULL or invalid.
 */
int64_t muon_state_bytes(int32_t n_tensors, const int64_t *rows, const int64_t *cols, const muon_layout *layout);
int64_t muon_state_workspace_bytes(int32_t n_tensors, const int64_t *rows, const int64_t *cols,
                                   const muon_layout *layout);

/*
 * Creates a state for n_tensors matrices (zero dimensions allowed, n_tensors
 * may be 0) on the current HIP device, with m = 0.  Work is enqueued on
 * hip_stream and the call returns after it completes.  On success *out owns
 * the state (free with muon_state_destroy).
 * Errors: EINVAL (as muon_state_bytes, or out NULL), ENOMEM, EDEVICE.
 */
int muon_state_create(muon_state **out, int32_t n_tensors, const int64_t *rows, const int64_t *cols,
                      const muon_layout *layout, void *hip_stream);

/*
 * One step over every matrix of the state, enqueued on hip_stream.
 *   params[k]: device float[rows*cols], row-major and contiguous, updated in place;
 *   grads[k]:  device float or bf16 (uint16), the same shape, read only;
 *   both arrays are host arrays of n_tensors device pointers, each 16-byte
 *   aligned (NULL allowed only for empty matrices), distinct for distinct k.
 *   expect: the layout the caller believes the state has (EMODE if it differs).
 * Calls on one state share its workspace: they are ordered on the device
 * (one stream, or the caller synchronizes).
 * Errors (no work enqueued): EINVAL (NULL argument, a hyperparameter outside
 * its domain, unknown flag bits, reserved != 0, STOCHASTIC without 8-bit
 * storage, two tensors with one param pointer, call from a device other than
 * the state's, hip_stream in HIP graph capture, as in adam_step), EMODE,
 * EALIGN; EDEVICE if a launch fails.
 */
int muon_step(muon_state *s, float *const *params, const void *const *grads, const muon_hparams *hp,
              const muon_layout *expect, void *hip_stream);

/*
 * The state's buffers, as adam_state_buffer_bytes, adam_state_read and
 * adam_state_write: ADAM_BUF_M_CODES and ADAM_BUF_M_SCALE (Q8),
 * ADAM_BUF_M_BF16 (BF16), ADAM_BUF_M_F32 (F32).
 * muon_state_momentum: the momentum's values, each matrix's segment padded
 * to 16 entries (padding 0), in device memory dst, 16-byte aligned: float
 * for F32 and Q8 storage (codes times their scale), bf16 for BF16; nbytes
 * must be exactly that size.  Asynchronous on hip_stream.
 * Errors: EINVAL (for muon_state_momentum also a call from a device other than
 * the state's), EALIGN, EDEVICE.
 */
int64_t muon_state_buffer_bytes(const muon_state *s, int32_t which);
int muon_state_read(muon_state *s, int32_t which, void *dst, int64_t nbytes, void *hip_stream);
int muon_state_write(muon_state *s, int32_t which, const void *src, int64_t nbytes, void *hip_stream);
int muon_state_momentum(muon_state *s, void *dst, int64_t nbytes, void *hip_stream);

/*
 * Checkpoint / resume, as adam_state_save and adam_state_load: the same
 * stream layout with magic "MEAMMUON", version 1, header of 40 + 24*n bytes
 * (i64 rows[n], i64 cols[n], i64 draw_index[n] after the fixed part) and the
 * state's buffers as records.
 */
int64_t muon_state_serialized_bytes(const muon_state *s);
int muon_state_save(muon_state *s, void *dst, int64_t nbytes, void *hip_stream);
int muon_state_load(muon_state **out, const void *src, int64_t nbytes, void *hip_stream);

/* Draw indices, as adam_state_set_draw_index and adam_state_get_draw_index. */
int muon_state_set_draw_index(muon_state *s, const int64_t *first_index, void *hip_stream);
int32_t muon_state_get_draw_index(const muon_state *s, int64_t *first_index, int32_t max_tensors);

/* Layout, tensor count (returned) and the first min(n_tensors, max_tensors)
   shapes (rows and cols may be NULL when max_tensors is 0). */
int32_t muon_state_describe(const muon_state *s, muon_layout *layout, int64_t *rows, int64_t *cols,
                            int32_t max_tensors);

/* Frees the state (after synchronizing the device, so no stream of the process
   may be capturing).  NULL is ignored. */
void muon_state_destroy(muon_state *s);

/*
 * muon_orthogonalize: out_i = O(x_i) for a batch of rows x cols matrices,
 * enqueued on hip_stream with no allocation, copy or synchronization (it can
 * be recorded into a graph; a replay repeats the call as recorded).
 *   x, out: device memory of x_dtype and out_dtype (enum adam_grad_dtype);
 *     element (i, r, c) at i*batch_stride + r*row_stride + c elements, strides
 *     >= 0, row_stride >= cols; aligned to the element; the last element's
 *     index is below 2^60.  out's matrices lie one after the other
 *     (batch_stride at least a matrix's extent) or side by side (all of them
 *     within a row_stride, as the heads of a fused weight are), and not
 *     between x's first and last element, except that out may be x itself
 *     with the same strides and type.
 *   workspace: device memory, 256-byte aligned, of at least
 *     muon_orthogonalize_workspace_bytes(batch, rows, cols), which may be 0
 *     (then NULL will do); written by the call, so neither x nor out lies in
 *     those bytes.  Calls that share one must be ordered on the device; so must
 *     the replays of graphs that recorded one.
 * Errors (no work enqueued): EINVAL (NULL pointer with a non-empty batch, a
 * dimension < 0 or >= 2^21, rows*cols >= 2^32, batch >= 2^31, a stride
 * outside its domain, out overlapping itself or x, unknown dtype, an iteration
 * outside its domain, workspace too small or overlapping x or out), EALIGN;
 * EDEVICE if a launch fails.
 */
typedef struct {
    int64_t batch, rows, cols;
    int64_t x_batch_stride, x_row_stride;     /* elements */
    int64_t out_batch_stride, out_row_stride; /* elements */
    int32_t x_dtype, out_dtype;               /* enum adam_grad_dtype */
} muon_matrices;

int64_t muon_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols);
int muon_orthogonalize(const muon_matrices *mats, const void *x, void *out, const muon_iteration *iteration,
                       void *workspace, int64_t workspace_bytes, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_MI355X_H */
