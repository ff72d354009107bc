/*
 * conv_bwd_train.h -- C ABI of the training-step operators that surround a
 * backward-data pass: matrix products grouped by expert with ragged sizes
 * (forward, data gradient, weight gradient), the global gradient norm with
 * clipping, and the clipped policy loss with a KL term (forward, backward).
 *
 * They chain as one step of a policy-tuned expert model: the loss gives
 * dlogits, the expert products carry it to the rows and to the filters, the
 * clip scales the gradients that come out.
 *
 * Conventions are those of conv_bwd_data.h: every call returns a
 * conv_bwd_status and throws nothing; tensors are row-major device memory
 * that the caller owns; a run call validates its arguments on the host,
 * enqueues on `stream` (a cudaStream_t; NULL = legacy default stream),
 * allocates nothing and never synchronises, so it can be captured in a CUDA
 * graph.  A plan owns its workspace and a device status word, allocated by
 * create on the device current then (which must be current in every run, else
 * CONV_BWD_ERR_INVALID_ARG); without a device create succeeds and run returns
 * CONV_BWD_ERR_CUDA.  Runs of
 * one plan share that workspace and must not overlap on the GPU; use one plan
 * per stream.  Device-side problems (an index out of range, a bounded wait
 * that ran out) are recorded in the status word and read with get_status;
 * kernels never trap.  Results do not depend on the order in which blocks run:
 * the same call on the same inputs gives the same bits.
 */
#ifndef CONV_BWD_TRAIN_H
#define CONV_BWD_TRAIN_H

#include <stdint.h>

#include "conv_bwd_data.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- expert products ------------------------------------------------------
 *
 * x [rows][K] holds rows sorted by expert: expert e owns rows
 * [offsets[e], offsets[e+1]); offsets is a device array of experts + 1 int32
 * (a router's output; the host never reads it).  w [experts][N][K] holds one
 * filter per expert in the K-contiguous layout of a 1x1 KYXC filter.
 *
 *   forward: y[i][n]     = sum_k x[i][k]  * w[e][n][k]          i in expert e
 *   data:    dx[i][k]    = sum_n dy[i][n] * w[e][n][k]
 *   weight:  dw[e][n][k] (+)= sum_{i in e} dy[i][n] * x[i][k]
 *
 * y and dx are fully overwritten: rows of no expert (before offsets[0], from
 * offsets[experts]) become +0.  dw is fp32 for either dtype (gradients are
 * accumulated over micro-batches); an expert without rows gets zeros, or
 * stays as it is when accumulating.  Rows of one expert never reach another
 * expert's results, NaN or infinity included.  One expert is a plain
 * linear layer.
 *
 * Offsets must be non-decreasing within [0, rows].  Others are recorded as a
 * DEVICE_FAULT and read as their running maximum clamped to that range.
 *
 * ld* are row strides in elements (>= the row's width; 0 means dense).
 * bf16 products are accumulated in fp32 and rounded once. */
typedef struct {
    int64_t experts, K, N;
    int32_t dtype; /* conv_bwd_dtype of x, w, y, dy, dx */
} conv_bwd_experts_desc;

typedef struct conv_bwd_experts_plan_s *conv_bwd_experts_plan;

typedef enum { CONV_BWD_EXPERTS_FORWARD = 0, CONV_BWD_EXPERTS_DATA = 1, CONV_BWD_EXPERTS_WEIGHT = 2 } conv_bwd_experts_dir;

/* Errors: INVALID_ARG (a size < 1, unknown dtype), UNSUPPORTED (experts >
 * 1024, K or N > 2^20, experts*K*N > 2^40), CUDA (allocation failed). */
conv_bwd_status conv_bwd_experts_create(const conv_bwd_experts_desc *desc, conv_bwd_experts_plan *out);
conv_bwd_status conv_bwd_experts_destroy(conv_bwd_experts_plan plan);

/* rows = 0 is valid (nothing is read; forward and data write nothing, weight
 * writes zeros or, accumulating, nothing).
 * Errors: INVALID_ARG (NULL pointer, rows < 0, ld smaller than the row,
 * output overlapping an input), MISALIGNED (a pointer not aligned to its
 * element), UNSUPPORTED (rows or output tiles > 2^31 - 2^16),
 * CUDA. */
conv_bwd_status conv_bwd_experts_forward(conv_bwd_experts_plan plan, int64_t rows, const void *x, int64_t ldx,
                                         const void *w, const int32_t *offsets, void *y, int64_t ldy, void *stream);
conv_bwd_status conv_bwd_experts_data(conv_bwd_experts_plan plan, int64_t rows, const void *dy, int64_t lddy,
                                      const void *w, const int32_t *offsets, void *dx, int64_t lddx, void *stream);
conv_bwd_status conv_bwd_experts_weight(conv_bwd_experts_plan plan, int64_t rows, const void *dy, int64_t lddy,
                                        const void *x, int64_t ldx, const int32_t *offsets, float *dw,
                                        int32_t accumulate, void *stream);

/* Synchronise `stream`, read and clear the plan's status word, as
 * conv_bwd_data_get_status.  After a wait that ran out this also makes the
 * plan's workspace ready for the next run. */
conv_bwd_status conv_bwd_experts_get_status(conv_bwd_experts_plan plan, void *stream, int32_t *detail);

/* ---- global gradient norm and clipping --------------------------------------
 *
 *   norm = sqrt(sum over all tensors and elements of g^2)
 *   coef = min(1, max_norm / (norm + 1e-6))
 *   out_i = g_i * coef            (computed in fp32, rounded once)
 *
 * over `count` tensors of `sizes[i]` elements (0 allowed) and `dtypes[i]`
 * (conv_bwd_dtype).  norm and coef are device floats.  The sum does not
 * overflow or underflow where the norm is a normal fp32 number.  A NaN makes
 * norm, coef and every output NaN; an infinity makes norm infinite and coef 0
 * (outputs 0, and NaN where the gradient was infinite); so a caller sees a
 * broken step in norm.
 *
 * Errors of create: INVALID_ARG (count < 0, size < 0, unknown dtype, NULL
 * arrays with count > 0), UNSUPPORTED (count > 65536, more than 2^40 elements,
 * tensors of 2^38 elements or more), CUDA. */
typedef struct conv_bwd_clip_plan_s *conv_bwd_clip_plan;
conv_bwd_status conv_bwd_clip_create(int32_t count, const int64_t *sizes, const int32_t *dtypes,
                                     conv_bwd_clip_plan *out);
conv_bwd_status conv_bwd_clip_destroy(conv_bwd_clip_plan plan);

/* grads is a host array of `count` device pointers (NULL allowed where the
 * size is 0), aligned to their element; no other alignment is needed.
 * Errors: INVALID_ARG (NULL), MISALIGNED, CUDA. */
conv_bwd_status conv_bwd_clip_norm(conv_bwd_clip_plan plan, const void *const *grads, float *norm, void *stream);

/* Norm, coef and the scaled gradients.  out[i] may be grads[i] (in place) or
 * memory that overlaps no gradient and no other output; INVALID_ARG for an
 * output that overlaps its own gradient otherwise, a NaN or negative
 * max_norm, or NULL arguments. */
conv_bwd_status conv_bwd_clip_run(conv_bwd_clip_plan plan, const void *const *grads, void *const *out, float max_norm,
                                  float *norm, float *coef, void *stream);

conv_bwd_status conv_bwd_clip_get_status(conv_bwd_clip_plan plan, void *stream, int32_t *detail);

/* ---- clipped policy loss with a KL term -------------------------------------
 *
 * Per token t with logits row z_t [vocab], chosen token a_t:
 *   logp = scale*z_t[a_t] - lse,   lse = log sum_v exp(scale*z_t[v])
 *   r    = exp(logp - old_logp)                  (1 where old_logp is NULL)
 *   d    = ref_logp - logp
 *   l    = -min(r*A, clamp(r, 1 - clip_low, 1 + clip_high)*A) + kl*(exp(d) - d - 1)
 *   loss = sum_t weight_t * l_t
 *   coef = dloss/dlogp = weight * (-[r*A <= clamp(r)*A] r*A + kl*(1 - exp(d)))
 *   dlogits[v] = grad * coef * scale * ([v == a] - exp(scale*z[v] - lse))
 *
 * The KL term is the non-negative estimate of KL(policy || reference) from
 * the chosen token; it is left out where ref_logp is NULL or kl is 0.  With
 * old_logp NULL the ratio is 1 and its gradient that of r (the first step
 * after sampling).  A token with weight 0 or a_t < 0 is masked: its row is not
 * read, it adds nothing, its logp, lse and coef are 0 and its dlogits row is
 * +0.  A row whose logits are all -inf has no distribution: its lse is -inf
 * and its logp, loss and gradient are NaN; single -inf logits are vocabulary
 * entries with probability 0.  a_t >= vocab is recorded as a DEVICE_FAULT and
 * treated as masked.  All arithmetic is fp32 (the loss is summed in fp64);
 * dlogits are rounded once to the logits' type.
 *
 * logits [tokens][ld]; ld >= vocab in elements, any alignment (0 = dense). */
typedef struct {
    int64_t vocab;
    int32_t dtype;                            /* conv_bwd_dtype of logits and dlogits */
    float clip_low, clip_high, kl, scale;     /* 0 <= clip_low <= 1, clip_high >= 0, kl >= 0, scale > 0, finite */
} conv_bwd_policy_desc;

typedef struct conv_bwd_policy_plan_s *conv_bwd_policy_plan;
/* Errors: INVALID_ARG (vocab < 1, unknown dtype, a parameter out of its
 * range), UNSUPPORTED (vocab > 2^30), CUDA. */
conv_bwd_status conv_bwd_policy_create(const conv_bwd_policy_desc *desc, conv_bwd_policy_plan *out);
conv_bwd_status conv_bwd_policy_destroy(conv_bwd_policy_plan plan);

/* loss [1], logp, lse, coef [tokens], all fp32, fully written.  tokens = 0
 * writes loss = 0.
 * Errors: INVALID_ARG (NULL, tokens < 0, ld < vocab), MISALIGNED,
 * UNSUPPORTED (tokens >= 2^31), CUDA. */
conv_bwd_status conv_bwd_policy_forward(conv_bwd_policy_plan plan, int64_t tokens, const void *logits, int64_t ld,
                                        const int32_t *actions, const float *advantage, const float *weight,
                                        const float *old_logp, const float *ref_logp, float *loss, float *logp,
                                        float *lse, float *coef, void *stream);

/* dlogits from the forward's lse and coef; grad is a device float (the
 * upstream gradient of loss; NULL = 1).  dlogits [tokens][ldd] may be logits
 * itself (with ldd = ld). */
conv_bwd_status conv_bwd_policy_backward(conv_bwd_policy_plan plan, int64_t tokens, const void *logits, int64_t ld,
                                         const int32_t *actions, const float *lse, const float *coef,
                                         const float *grad, void *dlogits, int64_t ldd, void *stream);

/* Forward and backward (grad = 1) in one launch that reads the logits from
 * memory once. */
conv_bwd_status conv_bwd_policy_forward_backward(conv_bwd_policy_plan plan, int64_t tokens, const void *logits,
                                                 int64_t ld, const int32_t *actions, const float *advantage,
                                                 const float *weight, const float *old_logp, const float *ref_logp,
                                                 float *loss, float *logp, void *dlogits, int64_t ldd, void *stream);

conv_bwd_status conv_bwd_policy_get_status(conv_bwd_policy_plan plan, void *stream, int32_t *detail);

#ifdef __cplusplus
}
#endif

#endif /* CONV_BWD_TRAIN_H */
