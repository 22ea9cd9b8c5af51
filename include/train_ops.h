/*
 * train_ops.h -- C ABI of the operators in front of the optimizer step, on
 * one GB300 (sm_103a): the embedding lookup with scaling, its gradient by
 * sorted tokens, and the global gradient norm over many tensors with
 * clipping.  They are part of the library of lamb.h and share its return
 * codes and lamb_last_error().
 *
 *   train_embed        out[i, :] = round(scale * table[ids[i] - first_row, :])
 *   train_embed_grad   grad[v, :] = round(old + scale * sum over the i with
 *                      ids[i] = first_row + v of grad_out[i, :])
 *   train_clip_*       G = ||g / S|| over all tensors;
 *                      c = max_norm / G if max_norm > 0 and G > max_norm, else 1;
 *                      out = round(c / S * g); inf/NaN anywhere: nothing written,
 *                      or NaN everywhere (train_clip_set_poison)
 *
 * With them a language model's training step runs around lamb_step: the
 * lookup starts the forward pass, the gradient by sorted tokens ends the
 * backward pass in the grad buffer that the step reads, and the clip takes
 * grads summed in fp32 (or in 16 bits) to the 16-bit grads of the step.  A clip
 * into other tensors that a step reads needs train_clip_set_poison, or the step
 * does not learn of an overflow.
 *
 * Element types.  Every matrix and tensor is bf16, fp16 or fp32
 * (TRAIN_BF16, TRAIN_FP16, TRAIN_FP32), and input and output types need not
 * match.  All arithmetic is fp32 or wider, with one rounding (to nearest
 * even) when a result is stored.  Pointers need only the alignment of their
 * element type; 16-byte aligned rows and tensors run fastest.
 *
 * Memory and streams.  The caller owns every buffer.  Calls enqueue their
 * work on the given stream (a cudaStream_t; NULL: the legacy default stream)
 * of the current device and return without waiting; buffers must stay valid,
 * and inputs unchanged, until the stream has passed them.  Outputs must not
 * overlap inputs, except where noted.  No call but train_clip_create and
 * train_clip_destroy allocates, frees or waits, so the calls can be captured
 * into a CUDA graph.
 *
 * Results do not depend on timing: every sum has a fixed order on a given
 * GPU model, and two calls on the same inputs give the same bits.
 */
#ifndef TRAIN_OPS_GB300_H
#define TRAIN_OPS_GB300_H

#include <stdint.h>

#include "lamb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types (the first two are LAMB_GRAD_BF16 and LAMB_GRAD_FP16). */
#define TRAIN_BF16 0
#define TRAIN_FP16 1
#define TRAIN_FP32 2

/* Types of token ids. */
#define TRAIN_INT32 0
#define TRAIN_INT64 1

/*
 * Embedding lookup: out[i, :] = round(scale * table[ids[i] - first_row, :]).
 *
 *   table        n_rows x dim, rows table_stride elements apart, read only
 *   ids          n_ids token ids (TRAIN_INT32 or TRAIN_INT64), consecutive
 *   first_row    the token id of the table's first row (>= 0; the last row's
 *                is at most 2^63 - 1): a table may hold a slice of the
 *                vocabulary.  A token outside
 *                [first_row, first_row + n_rows), negative ones among them,
 *                gives a row of zeros, so that the slices' results add up
 *   out          n_ids x dim, rows out_stride elements apart
 *
 * Strides are at least dim.  n_rows, dim and n_ids are at most 2^31 - 1; any
 * may be 0.
 */
LAMB_API int train_embed(const void* table, int32_t table_dtype, int64_t n_rows, int64_t dim,
                         int64_t table_stride, const void* ids, int32_t ids_dtype,
                         int64_t n_ids, int64_t first_row, float scale, void* out,
                         int32_t out_dtype, int64_t out_stride, void* stream);

/* Bytes of workspace that train_embed_grad needs for these sizes. */
LAMB_API int train_embed_grad_workspace(int64_t n_ids, int64_t n_rows, int64_t dim,
                                        int64_t* bytes);

/*
 * Gradient of the lookup with respect to the table.  The tokens are sorted on
 * the GPU, and each row's grads are summed in fp32 in an order that only the
 * ids fix; no atomic sum is used.
 *
 *   grad_out     n_ids x dim, rows grad_out_stride elements apart
 *   ids, first_row, scale   as in train_embed; tokens outside the slice add
 *                nothing
 *   padding_id   a token that adds nothing either (negative: none)
 *   accumulate   0: grad = round(scale * sum), rows that no token names
 *                become zero, and what was there is not read;
 *                1: grad = round(grad + scale * sum), rows that no token
 *                names are neither read nor written
 *   grad         n_rows x dim, rows grad_stride elements apart
 *   workspace    device memory, 16-byte aligned, of at least
 *                train_embed_grad_workspace bytes; its contents before the
 *                call do not matter, and it is free again when the stream has
 *                passed the call
 * n_ids * dim and n_rows * dim are at most 2^40.
 */
LAMB_API int train_embed_grad(const void* grad_out, int32_t grad_out_dtype,
                              int64_t grad_out_stride, const void* ids, int32_t ids_dtype,
                              int64_t n_ids, int64_t first_row, int64_t padding_id, float scale,
                              int32_t accumulate, void* grad, int32_t grad_dtype,
                              int64_t n_rows, int64_t dim, int64_t grad_stride, void* workspace,
                              int64_t workspace_bytes, void* stream);

/*
 * Global gradient norm and clipping over a fixed list of tensors.
 *
 * A handle is made once for the list and used every step; it owns a work
 * table and a small scratch area on the device.  It is bound to the device
 * current at its creation and to the stream given there; its calls enqueue
 * on that stream, and must not be made from two host threads at once.
 */
typedef struct train_clip_handle train_clip_handle;

/*
 *   sizes[i], dtypes[i], grads[i]   tensor i: elements (>= 0), type, device
 *                pointer; consecutive elements
 *   outs         NULL: clipping works in place.  Else outs[i] receives tensor
 *                i's clipped grads in out_dtypes[i]; each is grads[i] itself
 *                (then of the same type) or overlaps none of the grads
 * Tensors that overlap, one that is listed twice among them, are refused.
 * The arrays are host arrays, read before the call returns.  The call
 * waits for the upload of its work table.
 */
LAMB_API int train_clip_create(train_clip_handle** out, int32_t n_tensors, const int64_t* sizes,
                               const int32_t* dtypes, void* const* grads, void* const* outs,
                               const int32_t* out_dtypes, void* stream);

/*
 * What clipping leaves in the outputs when a grad is inf or NaN.  poison 0, as a
 * handle is made: nothing is written, they keep what they held.  1: every output
 * becomes NaN, those in place too.
 *
 * A step that reads outputs in other tensors needs 1 (or must wait for stats[2]):
 * lamb_step looks for inf and NaN in the grads that it is given, and would find
 * the clipped grads of the step before, finite, and apply them again.  With NaN
 * there it skips, and its loss scaler backs off.  The same holds in place for
 * grads spread over ranks without the split step: what train_clip_finish knows
 * of another rank's overflow, this rank's grads do not show.
 *
 * The call only sets the handle; calls made later use it (and so does a graph
 * that they are captured into).
 */
LAMB_API int train_clip_set_poison(train_clip_handle* h, int32_t poison);

/*
 * The norm alone.  stats (device, 3 floats) receives
 *   stats[0]  G = ||g / S||, +inf if a grad is inf or NaN
 *   stats[1]  the factor c / S that clipping multiplies the grads by (here
 *             1 / S), 0 if a grad is inf or NaN
 *   stats[2]  1 if a grad is inf or NaN, else 0
 * Squares are summed in fp32 a few at a time and in fp64 beyond; G and the
 * factor are formed in fp64 and rounded once.  loss_scale S is finite, > 0, and
 * 1 / S is finite in fp32.
 */
LAMB_API int train_clip_norm(train_clip_handle* h, float loss_scale, float* stats);

/* The norm, then out = round(c / S * g) for every tensor; max_norm <= 0 (or
 * a norm of at most max_norm) leaves c = 1.  If a grad is inf or NaN nothing
 * is written but stats, or NaN to every output (train_clip_set_poison).  In
 * place with c / S = 1 nothing needs writing.
 *
 * The outputs are divided by S, so a step that reads them takes loss_scale 1.
 * While lamb_step's dynamic loss scaler is on it divides by its own scale
 * whatever it is told: then clip with loss_scale 1 and max_norm times that scale
 * (lamb_result's next_loss_scale before the backward pass), which leaves the
 * scale in the outputs for the step to take off; stats[0] carries it too. */
LAMB_API int train_clip_grads(train_clip_handle* h, float max_norm, float loss_scale,
                              float* stats);

/*
 * The same in two halves, for grads that are spread over ranks:
 * train_clip_partial writes this rank's {sum g^2, 1 if a grad is inf or NaN}
 * (of the grads as given) to exchange (device, 2 doubles, 8-byte aligned);
 * the caller sums that over the ranks on the handle's stream; and
 * train_clip_finish forms G, c and the decision to write from the sums, as
 * train_clip_grads does.  lamb_split_norms' norm_exchange has the same layout.
 */
LAMB_API int train_clip_partial(train_clip_handle* h, double* exchange);
LAMB_API int train_clip_finish(train_clip_handle* h, const double* exchange, float max_norm,
                               float loss_scale, float* stats);

/* Free what the handle owns (after waiting for its stream).  NULL is a no-op. */
LAMB_API int train_clip_destroy(train_clip_handle* h);

#ifdef __cplusplus
}
#endif
#endif
