/*
 * lopt_train.h -- C ABI of the training operators in liblopt.so.
 *
 * lopt_step() (lopt.h) reads one contiguous fp32 gradient per parameter.
 * The operators here stand between a model's matrix products and those
 * gradients:
 *
 *   embedding      lookup of table rows with a scale, and the table's
 *                  gradient, summed token by token in a fixed order
 *   layer norm     forward, with the residual sum before it if wanted, and
 *                  backward with the gradients of weight and bias
 *   distillation   the loss of a row of logits against a teacher's top
 *                  logits, and its gradient, in one pass over the row
 *
 * Conventions
 *   - Return LOPT_OK or a negative LOPT_E_* code, as in lopt.h.  Arguments
 *     are checked on the host before anything is launched.
 *   - Every pointer is a device pointer on the current device, owned by the
 *     caller; work is enqueued on `stream` (a cudaStream_t) and nothing is
 *     allocated, synchronised or kept after the call.  Calls may be captured
 *     in a CUDA graph.
 *   - A matrix [rows x cols] has contiguous rows; `*_stride` is the distance
 *     between rows in elements.  Inputs may have any stride >= 0 (0: one row
 *     for all); outputs have a stride >= cols.
 *   - Element types: LOPT_F32, LOPT_F16, LOPT_BF16.  Arithmetic, sums and
 *     statistics are fp32; every output is rounded once, to its own type.
 *   - Outputs must not overlap inputs or each other (LOPT_E_ALIAS), except
 *     where "in place" is allowed below: then both must start at the same
 *     address with the same stride.
 *   - The same inputs give the same bits: sums run in a fixed order.
 */
#ifndef LOPT_TRAIN_H
#define LOPT_TRAIN_H

#include <stdint.h>

#include "lopt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- types ------------------------------------------------------------- */
#define LOPT_F32   0
#define LOPT_F16   1
#define LOPT_BF16  2

#define LOPT_I32   0   /* index types */
#define LOPT_I64   1

/* An index was not below the number of rows or columns (found on the device;
 * see `status` below). */
#define LOPT_E_INDEX -10

#define LOPT_MAX_TOP 1024   /* longest list of a teacher's top logits */

/*
 * Indices.  A negative index stands for "none": padding, an unused slot.
 * An index at or above the limit is an error that only the device can see:
 * it is treated as "none", and the kernels set bit 0 of *status (a device
 * int32 the caller zeroes and reads when it likes; NULL: not reported).  Bit 1
 * says that a bounded wait (1 s) inside lopt_distill() ran out: rows whose
 * loss is then NaN are not whole, neither is their gradient.
 */

/*
 * A status word of the library's own, one per device, for callers that keep
 * none: zero before the first call, at the same address as long as the
 * device's context lives.  lopt_status_word() gives its address on the current
 * device, to any thread, also while a stream is being captured.
 * lopt_status_take() waits for the current device, gives the bits set since
 * the last time and clears them.
 */
int lopt_status_word(int32_t** word);
int lopt_status_take(int32_t* flags);

/*
 * out[i] = scale * table[index[i]],  i < n;  zeros where the index is none.
 *   table  [rows x cols] of table_type;  index  [n];  out  [n x cols].
 */
int lopt_embed_forward(const void* table, int table_type, int64_t rows, int64_t cols, int64_t table_stride,
                       const void* index, int index_type, int64_t n, float scale,
                       void* out, int out_type, int64_t out_stride, int32_t* status, void* stream);

/*
 * The gradient of the table:
 *   grad[v] = scale * sum over i with index[i] == v, i ascending, of grad_out[i].
 * grad is contiguous fp32 [rows x cols], as lopt_step() reads it.  With
 * accumulate = 0 every row is written (zeros where no token has it); with 1
 * the sums are added to what grad holds, and rows without tokens are left.
 * The tokens are sorted by id and the sorted list is cut into pieces of equal
 * length, whose sums are then added in order: the same index list and sizes
 * give the same bits, but where a row's sum is cut depends on the other ids too.
 * workspace: lopt_embed_workspace() bytes, 256-byte aligned, any contents.
 */
int lopt_embed_workspace(int64_t n, int64_t rows, int64_t cols, int64_t* bytes);
int lopt_embed_backward(const void* grad_out, int type, int64_t grad_out_stride,
                        const void* index, int index_type, int64_t n, int64_t rows, int64_t cols, float scale,
                        int accumulate, float* grad, void* workspace, int64_t workspace_bytes,
                        int32_t* status, void* stream);

/*
 * Layer norm over the columns of s = x, or of s = x + residual:
 *   mean = sum(s) / cols,  rstd = 1 / sqrt(sum((s - mean)^2) / cols + eps),
 *   y = (s - mean) * rstd * weight + bias.
 * residual (and then summed, which receives s rounded to `type`) may be
 * NULL, and bias.  mean and rstd are fp32 [rows].  weight and bias are
 * [cols] of weight_type: LOPT_F32 or `type`.  The statistics and y come from
 * the unrounded s.  In place: y or summed on x or on residual.
 */
int lopt_layernorm_forward(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride,
                           const void* residual, int64_t residual_stride,
                           const void* weight, const void* bias, int weight_type, float eps,
                           void* y, int64_t y_stride, void* summed, int64_t summed_stride,
                           float* mean, float* rstd, void* stream);

/*
 * Its backward pass, for x the s of the forward pass, xhat = (x - mean) * rstd
 * and g = grad_out * weight:
 *   grad_x = rstd * (g - sum(g) / cols - xhat * sum(g * xhat) / cols) [+ grad_residual]
 *   grad_weight = sum over rows of grad_out * xhat,  grad_bias = sum over rows of grad_out.
 * grad_residual (the gradient that reaches s past the norm) and grad_bias
 * may be NULL.  grad_weight and grad_bias are fp32 [cols]; accumulate adds
 * to what they hold.  In place: grad_x on grad_out, x or grad_residual.
 * workspace: lopt_layernorm_workspace() bytes, 256-byte aligned, any contents.
 */
int lopt_layernorm_workspace(int64_t rows, int64_t cols, int64_t* bytes);
int lopt_layernorm_backward(const void* grad_out, int type, int64_t rows, int64_t cols, int64_t grad_out_stride,
                            const void* x, int64_t x_stride, const float* mean, const float* rstd,
                            const void* weight, int weight_type,
                            const void* grad_residual, int64_t grad_residual_stride,
                            void* grad_x, int64_t grad_x_stride, float* grad_weight, float* grad_bias,
                            int accumulate, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Distillation from a teacher's top logits.  Row r has logits z over all
 * cols classes, and `top` slots with the teacher's logit t_k for class i_k; a
 * slot counts if its index is not none and t_k > -inf.  With temperature T,
 *   p = softmax over the slots that count of t / T,   q = softmax of z / T,
 *   loss[r] = w * T^2 * sum_k p_k * (log p_k - log q[i_k]),
 *   grad[r][j] = w * T * (q[j] - sum over k with i_k == j of p_k),
 * w = row_weight[r] (NULL: 1).  A row with w == 0, or with no slot that
 * counts, has loss 0 and gradient 0, whatever its logits hold.  One slot
 * with any finite t_k is the cross entropy with class i_k.  grad (type of the
 * logits) may be NULL: the loss alone.  In place: grad on logits.
 * top_type: LOPT_F32 or `type`.  1 <= top <= LOPT_MAX_TOP, 1e-30 <= T <= 1e3.
 * The loss is off by about 2^-20 w T^2 (1 + log cols), from the logarithms, and
 * 2^-22 w T times the differences t_k - max t and z - max z that it weighs.
 */
int lopt_distill(const void* logits, int type, int64_t rows, int64_t cols, int64_t logits_stride,
                 const void* top_logits, int top_type, int64_t top_logits_stride,
                 const void* top_index, int index_type, int64_t top_index_stride, int64_t top,
                 float temperature, const float* row_weight,
                 float* loss, void* grad, int64_t grad_stride, int32_t* status, void* stream);

/*
 * Self-test of the bounded waits: lopt_distill() whose waits run out after
 * limit_ns (0 to 10^9) instead of 1 s.  Nothing hangs or faults: rows that it
 * did not finish have a NaN loss, and bit 1 of *status is set.
 */
int lopt_selftest_distill(int64_t limit_ns, const void* logits, int type, int64_t rows, int64_t cols,
                          int64_t logits_stride, const void* top_logits, int top_type, int64_t top_logits_stride,
                          const void* top_index, int index_type, int64_t top_index_stride, int64_t top,
                          float temperature, const float* row_weight, float* loss, void* grad, int64_t grad_stride,
                          int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOPT_TRAIN_H */
