/*
 * lopt_lm.h -- C ABI of the language model operators in liblopt.so.
 *
 * Beside the training operators of lopt_train.h, whose conventions and types
 * hold here too:
 *
 *   block norm            the norm of a block's output, its gate and residual
 *                         scale, the sum with the residual stream and the norm
 *                         before the next block; forward and backward
 *   linear cross entropy  of hidden states against the output table, without
 *                         keeping the logits; forward and backward
 *   AdamW                 one step over a list of tensors, moments in 32 or 8
 *                         bits, gradients clipped by their global norm
 */
#ifndef LOPT_LM_H
#define LOPT_LM_H

#include <stdint.h>

#include "lopt_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Block norm.  With rms(v) = 1 / sqrt(sum(v^2) / cols + eps) of a row:
 *   summed = residual + scale * sigmoid(gate) * (h * rms(h) * w_post)
 *   y = summed * rms(summed) * w_pre
 * gate may be NULL (no sigmoid factor).  w_post and w_pre are [cols] of
 * weight_type: LOPT_F32 or `type`.  rstd_post and rstd_pre receive rms(h) and
 * rms(summed), fp32 [rows].  y and the statistics come from the unrounded sum.
 * Sums of squares are fp32: a row whose sum is above its range counts as infinite.
 * In place: y or summed on h, residual or gate.
 */
int lopt_block_norm_forward(const void* h, int type, int64_t rows, int64_t cols, int64_t h_stride,
                            const void* residual, int64_t residual_stride, const void* gate, int64_t gate_stride,
                            const void* w_post, const void* w_pre, int weight_type, float scale, float eps,
                            void* y, int64_t y_stride, void* summed, int64_t summed_stride,
                            float* rstd_post, float* rstd_pre, void* stream);

/*
 * Its backward pass.  With xhat = summed * rstd_pre, hhat = h * rstd_post,
 * g = grad_y * w_pre, open = sigmoid(gate):
 *   grad_residual = rstd_pre * (g - xhat * sum(g * xhat) / cols) [+ grad_summed]
 *   dz = scale * open * grad_residual,  q = dz * w_post
 *   grad_h = rstd_post * (q - hhat * sum(q * hhat) / cols)
 *   grad_gate = q * hhat * (1 - open)
 *   grad_w_post = sum over rows of dz * hhat,  grad_w_pre = sum over rows of grad_y * xhat.
 * grad_summed (the gradient that reaches the sum past the norm) may be NULL;
 * gate and grad_gate are both given or both NULL.  grad_w_* are fp32 [cols];
 * accumulate adds to what they hold.  In place: grad_h, grad_residual and
 * grad_gate on grad_y, h, summed, gate or grad_summed.
 * workspace: lopt_block_norm_workspace() bytes, 256-byte aligned, any contents.
 */
int lopt_block_norm_workspace(int64_t rows, int64_t cols, int64_t* bytes);
int lopt_block_norm_backward(const void* grad_y, int type, int64_t rows, int64_t cols, int64_t grad_y_stride,
                             const void* h, int64_t h_stride, const void* summed, int64_t summed_stride,
                             const void* gate, int64_t gate_stride, const float* rstd_post, const float* rstd_pre,
                             const void* w_post, const void* w_pre, int weight_type, float scale,
                             const void* grad_summed, int64_t grad_summed_stride,
                             void* grad_h, int64_t grad_h_stride, void* grad_residual, int64_t grad_residual_stride,
                             void* grad_gate, int64_t grad_gate_stride, float* grad_w_post, float* grad_w_pre,
                             int accumulate, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Linear cross entropy.  x: [rows x cols] hidden states, weight: [classes x
 * cols], the output table, both of `type` (LOPT_F16 or LOPT_BF16); target: an
 * index per row, none where it is negative (padding; see lopt_train.h for those
 * at or above `classes`).  With logits z = x weight^T, which are never stored:
 *   lse[r] = log sum exp z[r],   loss[r] = row_weight[r] * (lse[r] - z[r][target[r]])
 * row_weight may be NULL (1).  A row without a target or with weight 0 has loss
 * 0; its lse is that of its logits, whatever they are.  loss and lse: fp32 [rows].
 * Products are exact, sums fp32.
 *
 * Backward, for the sum of the rows' losses, with lse as the forward pass gave it:
 *   G[r][j] = row_weight[r] * (exp(z[r][j] - lse[r]) - [j == target[r]])
 *   grad_x = G weight,   grad_weight = G^T x
 * Rows that do not count give zeros and add nothing, whatever they hold.  grad_x
 * (of `type`) or grad_weight may be NULL.  grad_weight is of LOPT_F32, which
 * accumulate = 1 adds to, or of `type`.  For the products G is the sum of 16-bit
 * parts, the first rounded relative to 2^-15 of the largest row_weight at least: two or
 * three for an fp32 grad_weight; for one of `type` and for grad_x two, or one, beside
 * which the targets' entries are fp32.
 *
 * Bit 1 of *status: a bounded wait (1 s) ran out; losses, lse and grad_x are then
 * NaN and grad_weight is not valid.
 * workspace: lopt_linear_ce_workspace() bytes for the direction, 256-byte aligned,
 * any contents; aligned = 1 where the rows of x and weight start on 16-byte
 * boundaries (others are copied first), grad_weight_type LOPT_F32 or other.  LOPT_F32's
 * size does for the other types too, and either does without grad_weight.
 * rows and classes up to 2^22, cols up to 2^16.
 */
int lopt_linear_ce_workspace(int64_t rows, int64_t classes, int64_t cols, int aligned, int backward,
                             int grad_weight_type, int64_t* bytes);
int lopt_linear_ce_forward(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, const void* weight,
                           int64_t classes, int64_t weight_stride, const void* target, int index_type,
                           const float* row_weight, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                           int32_t* status, void* stream);
int lopt_linear_ce_backward(const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride, const void* weight,
                            int64_t classes, int64_t weight_stride, const void* target, int index_type,
                            const float* row_weight, const float* lse, void* grad_x, int64_t grad_x_stride,
                            void* grad_weight, int grad_weight_type, int64_t grad_weight_stride, int accumulate,
                            void* workspace, int64_t workspace_bytes, int32_t* status, void* stream);

/*
 * Self-test of the bounded waits: lopt_linear_ce_forward() whose waits run out
 * after limit_ns (0 to 10^9) instead of 1 s.  Nothing hangs or faults: if one did, all
 * losses and lse of the launch (32,768 rows or fewer) are NaN, and bit 1 of *status is set.
 */
int lopt_selftest_linear_ce(int64_t limit_ns, const void* x, int type, int64_t rows, int64_t cols, int64_t x_stride,
                            const void* weight, int64_t classes, int64_t weight_stride, const void* target,
                            int index_type, const float* row_weight, float* loss, float* lse, void* workspace,
                            int64_t workspace_bytes, int32_t* status, void* stream);

/*
 * AdamW.  For every element of every tensor, in fp32, each operation rounded
 * once (no fused multiply-add), with g the gradient times the clip factor:
 *   m = beta1 * m + (1 - beta1) * g
 *   v = beta2 * v + ((1 - beta2) * g) * g
 *   param = param * (1 - lr * weight_decay)                  where decay is set
 *   param = param - (lr / (1 - beta1^t)) * (m / (sqrt(v) * (1 / sqrt(1 - beta2^t)) + eps))
 *   copy = param, rounded
 *
 * 8-bit moments: a tensor is cut into blocks of LOPT_ADAMW_BLOCK consecutive
 * elements (the last may be shorter) with one fp32 scale each for m and v.  A
 * code q of m (int8) stands for sign(q) * q^2 * m_scale, a code of v (uint8)
 * for (q^2 * v_scale)^2: it holds the root of v.  After the step scale is the
 * block's largest |m| (or root of v) over 127^2 (255^2), and a value between
 * two codes takes the upper one with the chance that makes the mean of what the
 * codes stand for right, of m and of the root of v: repeated steps do not lose
 * changes smaller than the distance of two codes.  (v itself, the root's square, is
 * then above its value on average, by the variance of that rounding: some 3 % for a
 * root of 5e-4 of its block's largest, some 50 % for one of 1e-5.)  A block whose largest value is at most 1e-30 is
 * stored as zeros.  The chance is decided by bits of
 *   h = mix((i ^ key) & 0xffffffff), with i >> 32 times 0x85ebca6b, modulo 2^32, XORed into key,
 *   key = mix(seed ^ (index + 1) * 0x9e3779b9 modulo 2^32),
 * mix the final mixing of MurmurHash3 (32 bits), i the element, index the
 * tensor's place in the list: the upper half of h for m, the lower for v.
 * Non-finite gradients make the moments of their block NaN; max_norm guards
 * against that.
 *
 * max_norm > 0 (infinity allowed): the norm of all gradients together is
 * computed first (squares summed to about 2^-45 of their sum) and written to
 * *norm; the clip factor is min(1, max_norm / (norm + 1e-6)), rounded once.  If
 * the norm is not finite the step changes nothing, and *norm tells.
 * max_norm = 0: no clipping, norm and workspace are not used.
 */
#define LOPT_ADAMW_BLOCK 256

typedef struct {
  float* param;         /* n elements */
  const void* grad;     /* n of grad_type */
  void* m;              /* n float, or int8 codes */
  void* v;              /* n float, or uint8 codes */
  float* m_scale;       /* 8-bit moments: one per block; else NULL */
  float* v_scale;
  void* copy;           /* n of copy_type, or NULL */
  int64_t n;
  int32_t grad_type;    /* LOPT_F32, LOPT_F16, LOPT_BF16 */
  int32_t copy_type;    /* LOPT_F16, LOPT_BF16 */
  int32_t moments;      /* 32 or 8: bits */
  int32_t decay;        /* 1: weight decay applies */
} lopt_adamw_tensor;

/* LOPT_OK if the list is sound; LOPT_E_ALIAS if two of its arrays overlap (the
 * step itself checks each tensor on its own, not tensors against each other). */
int lopt_adamw_check(const lopt_adamw_tensor* tensors, int32_t n);
int lopt_adamw_workspace(int64_t* bytes);
int lopt_adamw_step(const lopt_adamw_tensor* tensors, int32_t n, int64_t t, double lr, double beta1, double beta2,
                    double eps, double weight_decay, double max_norm, uint32_t seed, float* norm,
                    void* workspace, int64_t workspace_bytes, void* stream);
/* The moments as fp32 values: m[i] and v[i] receive tensor i's (host arrays of
 * device pointers, outputs that overlap nothing). */
int lopt_adamw_moments(const lopt_adamw_tensor* tensors, int32_t n, float* const* m, float* const* v, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOPT_LM_H */
