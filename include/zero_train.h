/*
 * zero_train.h -- C ABI of the training operators beside the ZeRO step
 * (zero_step.h): AdamW over many separate tensors with 32-bit or 8-bit
 * moments, the global gradient norm with its clipping factor, and the linear
 * layer whose gradients the steps consume.
 *
 * The general rules of zero_step.h hold: 0 or a negative ZERO_E* code, a
 * rejected call has no side effects, device memory is the caller's, kernels
 * are enqueued on the caller's stream and the call returns at once, counts
 * and strides are in elements.  All of these operators may be captured in a
 * CUDA graph once their first call on the device has been made.
 */
#ifndef ZERO_TRAIN_H
#define ZERO_TRAIN_H

#include "zero_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of gradients, parameters and layers. */
#define ZERO_TYPE_FP16 0
#define ZERO_TYPE_BF16 1
#define ZERO_TYPE_FP32 2 /* gradients only */

/* ------------------------------------------------------------------------ */
/* AdamW over many tensors, gradient norm                                   */
/* ------------------------------------------------------------------------ */

/* One tensor of a plan.  Buffers are device memory.
 * 8-bit moments: the tensor is cut into blocks of 256 elements from its
 * first one on (the last may be shorter).  m holds OCP E4M3 codes of
 * momentum / m_scale[block], v holds E4M3 codes of sqrt(variance) /
 * v_scale[block] (the root, so that the code's range of 2^17 is one of 2^35
 * for the variance; its sign bit is 0).  All-zero codes and scales are a
 * zero state. */
typedef struct {
    const void* grad;    /* rank r's gradient at grad + r * rank_stride, type grad_type */
    int64_t rank_stride; /* elements between ranks, >= n (unused with P = 1) */
    float* master;       /* fp32 [n], read and written */
    void* m;             /* fp32 [n], or E4M3 codes [n]; read and written */
    void* v;             /* fp32 [n], or E4M3 codes [n]; read and written */
    float* m_scale;      /* 8-bit moments: fp32 [ceil(n / 256)], read and written */
    float* v_scale;      /* 8-bit moments: fp32 [ceil(n / 256)], read and written */
    void* param;         /* param_type [n], written: the rounded new weights */
    int64_t n;           /* elements; 0 is allowed (the pointers are then not looked at) */
    float weight_decay;  /* finite, >= 0 */
    float lr_scale;      /* this tensor's learning rate is lr * lr_scale; finite, >= 0 */
} zero_adamw_tensor_t;

/* What a plan holds on the host; its table is device memory. */
typedef struct {
    int32_t n_tensors;
    int32_t P;
    int32_t grad_type;
    int32_t param_type;
    int32_t state_bits; /* 32, 8, or 0: gradients only (zero_grad_norm) */
    int32_t vector_tensors; /* tensors whose streams share one 16-byte phase: whole-vector accesses */
    int32_t pipeline;       /* 1: all of them do (8-bit codes on 16 bytes), a large step may copy in bulk */
    int32_t norm_vecs;      /* size of the norm's units of work */
    int64_t elements;   /* of all tensors */
    int64_t chunks;     /* units of work of a step */
    int64_t norm_chunks;
    int64_t table_bytes;
} zero_adamw_plan_t;

/* Plan a list of tensors (host only).  Fills *plan and, when table_out is not
 * NULL, writes plan->table_bytes bytes of table there (capacity table_bytes);
 * the caller copies them to device memory aligned to 16 bytes and passes that
 * copy to the calls below, which use part of it as scratch: calls with one
 * table must not overlap on the GPU.  The table names the tensors' addresses;
 * a plan serves as long as they stay.  Two-call pattern: with table_out NULL
 * only *plan is filled.
 * state_bits 0 plans gradients alone: param_type and every buffer but grad
 * are not looked at.
 * Errors: ZERO_EINVAL (null pointer, n_tensors < 1, P outside
 * [1, ZERO_MAX_RANKS], an unknown type or state_bits, n < 0, rank_stride < n
 * with P > 1, a bad weight_decay or lr_scale, capacity too small),
 * ZERO_EALIGN (a buffer not aligned to its element size), ZERO_EOVERLAP (two
 * written buffers, or a written buffer and a gradient, share a byte),
 * ZERO_ENOMEM. */
int zero_adamw_plan(const zero_adamw_tensor_t* tensors, int32_t n_tensors, int32_t P,
                    int32_t grad_type, int32_t param_type, int32_t state_bits,
                    zero_adamw_plan_t* plan, void* table_out, int64_t table_bytes);

/* Norm of the mean gradient of all tensors together, and the factor that
 * clips it.  stats (device fp32 [3]) receives
 *   stats[0] = grad_scale * sqrt(sum over all elements of mean_r(grad)^2)
 *   stats[1] = grad_scale * min(1, max_norm / (stats[0] + 1e-6)), or
 *              grad_scale when max_norm <= 0 (no clipping), or 0 when the
 *              norm is not finite
 *   stats[2] = 1 when the norm is finite, else 0.
 * grad_scale undoes a loss scale (1 / loss scale); max_norm applies to the
 * scaled norm.  Squares are summed in fp32 with compensation, those that leave
 * its range in fp64, and joined in fp64 in a fixed order: the same gradients
 * give the same bits on one device model.  Means (fp32) of any size count; the
 * norm is not finite when one of them or stats[0] itself is not.
 * Errors: ZERO_EINVAL (null pointer, grad_scale not finite and positive,
 * max_norm NaN), ZERO_EALIGN, ZERO_ECUDA. */
int zero_grad_norm(const zero_adamw_plan_t* plan, void* table, float grad_scale, float max_norm,
                   float* stats, void* cuda_stream);

/* One AdamW step (decoupled weight decay) over every tensor of the plan, in
 * one launch.  Per element, in fp32 and in this order:
 *   g  = ((0 + g_0) + g_1) + ... + g_{P-1};  g = g / P;  g = g * stats[1]
 *   m  = b1*m + (1-b1)*g;   v = b2*v + (1-b2)*(g*g)
 *   w  = w - (lr_j*wd_j)*w;   w = w - (m*(lr_j*r1)) / (sqrt(v)*c2 + eps)
 *   param = round(w)  (nearest even)
 * with lr_j = lr * lr_scale_j, 1-b in fp32, r1 = fp32(1 / (1 - b1^t)) and
 * c2 = fp32(1 / sqrt(1 - b2^t)) (from the fp32 betas, in double).  In the
 * lines of g, m and v every operation is rounded by itself; in the line of w
 * the products are fused with the sums, and the quotient and, with 32-bit
 * moments, the square root are within 2 ulp (they enter the update, which is
 * small against the weight).
 * stats NULL: no factor.  stats (of zero_grad_norm, on the same stream):
 * g is multiplied by stats[1], and when stats[2] is 0 the step leaves
 * everything as it was (a gradient overflowed).
 * 8-bit moments are widened (m = code * m_scale, v = (code * v_scale)^2),
 * updated as above, and the weights use the updated moments before these are
 * rounded for storage.  Storage, per block of 256: with a the block's largest
 * |m|, m_scale = a * fp32(1/448) and the codes are the nearest (even) E4M3
 * values of m * (448 / a); for r = sqrt(v) likewise, but its codes are
 * rounded to a neighbour at random in proportion to the distances, so that
 * the slow average v follows its gradients in expectation although a code's
 * step is wider than one update; an r above 0 never gets the code 0 (an
 * update divides by it).  A block whose a is below 2^-96 gets scale 0.  A
 * block with a non-finite moment gets the scale NaN.
 * The random bits are those of seed (vary it per step, for instance t), the
 * tensor's index and the element's index alone: a step can be repeated.
 * Errors: ZERO_EINVAL (null pointer, plan with state_bits 0, t < 1, a
 * hyper-parameter that is not finite, beta outside [0, 1), eps neither 0 nor
 * at least 2^-126), ZERO_EALIGN, ZERO_ECUDA. */
int zero_adamw_step(const zero_adamw_plan_t* plan, void* table, const float* stats, int64_t t,
                    float lr, float beta1, float beta2, float eps, uint32_t seed,
                    void* cuda_stream);

/* ------------------------------------------------------------------------ */
/* The linear layer                                                         */
/* ------------------------------------------------------------------------ */

#define ZERO_ACT_NONE 0
#define ZERO_ACT_RELU 1 /* NaN stays NaN; the gradient passes where z > 0, and is 0 elsewhere whatever it holds */
#define ZERO_ACT_GELU 2 /* tanh's form: z / (1 + exp(-2 sqrt(2/pi) (z + 0.044715 z^3))) */
#define ZERO_ACT_SILU 3 /* z / (1 + exp(-z)) */

/* Bytes of workspace that is enough for a call of zero_linear_forward
 * (backward 0) or zero_linear_backward (backward 1) of these sizes.  aligned
 * != 0 when x, w, dy and z start on 16 bytes and have row strides that are
 * multiples of 8 elements; otherwise room for aligned copies is counted (rows
 * laid out off that boundary are copied in every call: pad a weight's rows
 * once to save it).  May be 0.  Host only.  Errors: ZERO_EINVAL. */
int zero_linear_workspace(int64_t T, int64_t K, int64_t N, int32_t act, int32_t backward,
                          int32_t aligned, int64_t* bytes);

/* y = act(x w^T + bias) + residual for T tokens, K inputs, N features:
 * x [T][ldx], w [N][ldw] (both K wide), bias [N] or NULL, residual [T][ldr]
 * or NULL, y [T][ldy], all of `type` (ZERO_TYPE_FP16 or ZERO_TYPE_BF16).
 * z [T][ldz] or NULL receives x w^T + bias, which the backward pass of a
 * layer with an activation needs.  Products are summed in fp32; y and z are
 * each rounded once, y from the unrounded z.  residual may be y itself (same
 * pointer and stride).  T may be 0.
 * workspace: device, 16-byte aligned, zero_linear_workspace bytes (may be
 * NULL when that is 0); calls that share one must not overlap on the GPU.
 * The same call gives the same bits.
 * Errors: ZERO_EINVAL (sizes above 2^31 - 513, a null pointer, a row stride
 * below its row, act or type unknown, workspace too small), ZERO_EALIGN
 * (a pointer not on its element size, workspace not on 16 bytes),
 * ZERO_EOVERLAP (y or z shares an element with an input or each other, or the
 * used workspace a byte with any of them), ZERO_ECUDA. */
int zero_linear_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                        const void* residual, int64_t ldr, void* y, int64_t ldy, void* z,
                        int64_t ldz, int64_t T, int64_t K, int64_t N, int32_t act, int32_t type,
                        void* workspace, int64_t workspace_bytes, void* cuda_stream);

/* The gradients of zero_linear_forward from dy [T][lddy], the gradient of y:
 *   dz = dy * act'(z)   (z [T][ldz] of the forward call; unused with
 *                        ZERO_ACT_NONE, may then be NULL)
 *   dx = dz w  [T][lddx];  dw = dz^T x  [N][lddw];  db = sum over tokens of dz [N]
 * The residual's gradient is dy itself.  dx, dw and db may each be NULL (not
 * computed; w is unused without dx, x without dw).  dw and db may lie
 * anywhere, for instance in a rank's gradients of the flat vector that
 * zero_adam_step takes.  dz is rounded to `type` once, before the products (in
 * fp16 above 65504 it becomes infinite, below 3e-8 zero: scale the loss), and db
 * is summed from it unrounded; sums are in fp32.  With T = 0 dw and db become 0.
 * workspace, errors: as zero_linear_forward (also ZERO_EINVAL when dx, dw and
 * db are all NULL). */
int zero_linear_backward(const void* dy, int64_t lddy, const void* z, int64_t ldz, const void* x,
                         int64_t ldx, const void* w, int64_t ldw, void* dx, int64_t lddx, void* dw,
                         int64_t lddw, void* db, int64_t T, int64_t K, int64_t N, int32_t act,
                         int32_t type, void* workspace, int64_t workspace_bytes,
                         void* cuda_stream);

/* Which kernel the products of a linear layer would take (a diagnostic like
 * zero_step_plan: nothing is launched).  products: 0 the forward product, 1 dx,
 * 2 dw, 3 both.  *launches: how many the products take; of the first one, the
 * *rows x *columns of a tile, the CTAs of a *cluster (256 rows: a pair that
 * shares a tile; 128 rows: they share a contraction) and the CTAs *per_sm.
 * Depends on the current device's SM count.
 * Errors: ZERO_EINVAL (also T < 1), ZERO_ECUDA. */
int zero_linear_plan(int64_t T, int64_t K, int64_t N, int32_t products, int32_t* launches,
                     int32_t* rows, int32_t* columns, int32_t* cluster, int32_t* per_sm);

/* Bounded waits of the kernels of this header that gave up on the current
 * device since the last reset; like zero_device_timeouts (0 in every correct
 * run, reading it synchronises). */
int zero_train_timeouts(int64_t* count, int32_t reset);

/* Diagnostic of those waits, like zero_selftest_wait_timeout: enqueues the step
 * of zero_adamw_step (without stats) through the pipeline of bulk copies, whose
 * first CTA never hands a stage of its ring back, while half of the lanes of its
 * copying warp are told that it did.  That warp's wait runs out after 2 seconds,
 * the CTA adds 1 to the count of zero_train_timeouts and returns; every other
 * CTA finishes and the context stays usable.  The first CTA's part of the
 * tensors is left partly updated.
 * Errors: as zero_adamw_step, and ZERO_EINVAL unless the plan has fp16 gradients
 * of one rank, fp16 parameters, fp32 moments, and takes the pipeline (4096
 * chunks). */
int zero_selftest_adamw_wait(const zero_adamw_plan_t* plan, void* table, int64_t t, float lr,
                             float beta1, float beta2, float eps, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_TRAIN_H */
