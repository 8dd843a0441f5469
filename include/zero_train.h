/*
 * zero_train.h -- C ABI of the training operators beside the ZeRO step
 * (zero_step.h): AdamW over many separate tensors with 32-bit or 8-bit
 * moments, the global gradient norm with its clipping factor, and the layers
 * whose gradients the steps consume: the linear layer, the gated feed-forward
 * projections, embedding, layer norm, and the loss that ends a language model.
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
#define ZERO_TYPE_FP32 2 /* gradients of AdamW and its norm, a teacher's logits */

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

/* ------------------------------------------------------------------------ */
/* Gated feed-forward projections                                           */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace that is enough for a call of zero_gated_forward (backward
 * 0) or zero_gated_backward (backward 1) of these sizes.  aligned != 0 when x,
 * wg and wu start on 16 bytes and have row strides that are multiples of 8
 * elements; otherwise room for aligned copies is counted.  May be 0 for the
 * forward call.  Host only.  Errors: ZERO_EINVAL. */
int zero_gated_workspace(int64_t T, int64_t K, int64_t N, int32_t backward, int32_t aligned,
                         int64_t* bytes);

/* h = act(g) * u with g = x wg^T + bg and u = x wu^T + bu for T tokens, K
 * inputs, N features: x [T][ldx], wg [N][ldwg] and wu [N][ldwu] (both K wide;
 * they may be halves of one matrix), bg and bu [N] or NULL, h [T][ldh], all of
 * `type` (ZERO_TYPE_FP16 or ZERO_TYPE_BF16).  g [T][ldg] and u [T][ldu], both
 * or neither NULL, receive the pre-activations, which the backward pass needs.
 * Products are summed in fp32; h, g and u are each rounded once, h from the
 * unrounded g and u.  T may be 0.  (The block's down-projection, with its
 * residual, is zero_linear_forward on h.)
 * workspace: device, 16-byte aligned, zero_gated_workspace bytes (may be NULL
 * when that is 0); calls that share one must not overlap on the GPU.  The same
 * call gives the same bits.
 * Errors: ZERO_EINVAL (T or K above 2^31 - 513, N above half of that, a null
 * pointer, one of g and u NULL, a row stride below its row, act or type
 * unknown, workspace too small), ZERO_EALIGN (a pointer not on its element
 * size, workspace not on 16 bytes), ZERO_EOVERLAP (an output shares an element
 * with an input or another output, or the used workspace a byte with any of
 * them), ZERO_ECUDA. */
int zero_gated_forward(const void* x, int64_t ldx, const void* wg, int64_t ldwg, const void* wu,
                       int64_t ldwu, const void* bg, const void* bu, void* h, int64_t ldh, void* g,
                       int64_t ldg, void* u, int64_t ldu, int64_t T, int64_t K, int64_t N,
                       int32_t act, int32_t type, void* workspace, int64_t workspace_bytes,
                       void* cuda_stream);

/* The gradients of zero_gated_forward from dh [T][lddh], the gradient of h,
 * and the forward call's g and u:
 *   du = dh * act(g);  dg = dh * u * act'(g)
 *   dx = dg wg + du wu  [T][lddx]
 *   dwg = dg^T x  [N][lddwg];  dwu = du^T x  [N][lddwu]
 *   dbg = sum over tokens of dg;  dbu = sum over tokens of du  [N]
 * Each of dx, dwg, dwu, dbg and dbu may be NULL (not computed; wg and wu are
 * unused without dx, x without dwg and dwu).  dg and du are rounded to `type`
 * once, before the products (in fp16 above 65504 they become infinite, below
 * 3e-8 zero: scale the loss), and dbg and dbu are summed from them unrounded;
 * sums are in fp32.  With ZERO_ACT_RELU dg is 0 where g is not above 0,
 * whatever dh and u hold.  With T = 0 all of dwg, dwu, dbg and dbu become 0.
 * workspace (never 0 bytes here, unless T is 0), errors: as zero_gated_forward
 * (also ZERO_EINVAL when all outputs are NULL). */
int zero_gated_backward(const void* dh, int64_t lddh, const void* g, int64_t ldg, const void* u,
                        int64_t ldu, const void* x, int64_t ldx, const void* wg, int64_t ldwg,
                        const void* wu, int64_t ldwu, void* dx, int64_t lddx, void* dwg,
                        int64_t lddwg, void* dwu, int64_t lddwu, void* dbg, void* dbu, int64_t T,
                        int64_t K, int64_t N, int32_t act, int32_t type, void* workspace,
                        int64_t workspace_bytes, void* cuda_stream);

/* Which kernel the gated projections' products would take, like
 * zero_linear_plan: products 0 the forward product, 1 dx, 2 dwg and dwu, 3 all
 * three; of the first launch the tile (of a forward product half of its
 * columns are the gate's; up to 128 tokens half of its rows), the cluster and
 * the CTAs per SM.  Errors: ZERO_EINVAL (also T < 1), ZERO_ECUDA. */
int zero_gated_plan(int64_t T, int64_t K, int64_t N, int32_t products, int32_t* launches,
                    int32_t* rows, int32_t* columns, int32_t* cluster, int32_t* per_sm);

/* ------------------------------------------------------------------------ */
/* Embedding                                                                */
/* ------------------------------------------------------------------------ */

/* y[t] = scale * table[ids[t]] for T tokens: ids int32 [T], table [V][ldt]
 * (D wide), y [T][ldy], of `type` (ZERO_TYPE_FP16 or ZERO_TYPE_BF16), rounded
 * once.  An id outside [0, V) (padding) gives a row of zeros.  T may be 0.
 * Errors: ZERO_EINVAL (a null pointer, T above 2^31 - 513, D or V above 2^30,
 * a row stride below D, scale not finite, type unknown), ZERO_EALIGN (a
 * pointer not on its element size), ZERO_EOVERLAP (y shares an element with
 * the table or the ids), ZERO_ECUDA. */
int zero_embed_forward(const int32_t* ids, const void* table, int64_t ldt, void* y, int64_t ldy,
                       int64_t T, int64_t D, int64_t V, float scale, int32_t type,
                       void* cuda_stream);

/* Bytes of workspace of zero_embed_backward, never above
 * 2 (T + 3) (D + 23) + 17408 (the parts of rows that are added up last, for few
 * tokens; for many about an eighth of that).  Host only.  Errors:
 * ZERO_EINVAL. */
int zero_embed_workspace(int64_t T, int64_t D, int64_t V, int64_t* bytes);

/* The table's gradient, dtable[v] = scale * sum of dy[t] over the tokens with
 * ids[t] = v, dtable [V][lddt], dy [T][lddy].  Sums are in fp32, over a row's
 * tokens in a fixed order (the same call gives the same bits), rounded once.
 * add 0: every row of dtable is written, those without a token with zeros.
 * add 1: the sums are added to what dtable holds (a table whose gradient the
 * output layer has written already) before the rounding, and rows without a
 * token stay as they are.  Tokens outside [0, V) are passed over, whatever
 * their rows of dy hold.  With T = 0 dtable becomes 0 (add 0) or stays.
 * workspace: device, 16-byte aligned, zero_embed_workspace bytes; calls that
 * share one must not overlap on the GPU.
 * Errors: as zero_embed_forward (also a workspace too small; dtable shares an
 * element with dy or the ids, or the workspace a byte with any of them). */
int zero_embed_backward(const int32_t* ids, const void* dy, int64_t lddy, void* dtable,
                        int64_t lddt, int64_t T, int64_t D, int64_t V, float scale, int32_t add,
                        int32_t type, void* workspace, int64_t workspace_bytes,
                        void* cuda_stream);

/* ------------------------------------------------------------------------ */
/* Layer norm                                                               */
/* ------------------------------------------------------------------------ */

/* y = (x - mean) * rstd * weight + bias over rows of D elements, with
 * rstd = 1 / sqrt(mean((x - mean)^2) + eps): x [T][ldx], y [T][ldy], weight [D]
 * or NULL (ones), bias [D] or NULL (zeros), all of `type`.  mean and rstd (fp32
 * [T], each may be NULL) receive the statistics that the backward pass needs.
 * Statistics are in fp32, the variance that of the centred values; y is
 * rounded once.  y may be x itself (same pointer and stride).  T may be 0.
 * Errors: ZERO_EINVAL (a null pointer, T above 2^31 - 513, D above 2^30, a row
 * stride below D, eps not finite or below 2^-126, type unknown), ZERO_EALIGN
 * (a pointer not on its element size), ZERO_EOVERLAP (an output shares an
 * element with an input or another output), ZERO_ECUDA. */
int zero_layernorm_forward(const void* x, int64_t ldx, const void* weight, const void* bias,
                           void* y, int64_t ldy, float* mean, float* rstd, int64_t T, int64_t D,
                           float eps, int32_t type, void* cuda_stream);

/* Bytes of workspace of zero_layernorm_backward.  Host only.  Errors:
 * ZERO_EINVAL. */
int zero_layernorm_workspace(int64_t T, int64_t D, int64_t* bytes);

/* The gradients of zero_layernorm_forward from dy [T][lddy] and the forward
 * call's mean and rstd.  With h = (x - mean) * rstd and a = dy * weight:
 *   dx = rstd * (a - mean(a) - h * mean(a * h)) + dres   [T][lddx]
 *   dweight = sum over rows of dy * h;  dbias = sum over rows of dy   [D]
 * dres [T][lddr] or NULL is the gradient that reaches x past the norm (a
 * residual's).  dx, dweight and dbias may each be NULL (not computed).  dx may
 * be dres itself, and dy itself where D is at most 16384 (same pointer and
 * stride).  Sums are in fp32 and in a fixed order; each output is rounded
 * once.  With T = 0 dweight and dbias become 0.
 * workspace: device, 16-byte aligned, zero_layernorm_workspace bytes (may be
 * NULL without dweight and dbias); calls that share one must not overlap on
 * the GPU.
 * Errors: as zero_layernorm_forward (also ZERO_EINVAL when all outputs are
 * NULL or the workspace is too small, and ZERO_EOVERLAP when the workspace
 * shares a byte with a matrix). */
int zero_layernorm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                            const void* weight, const float* mean, const float* rstd,
                            const void* dres, int64_t lddr, void* dx, int64_t lddx, void* dweight,
                            void* dbias, int64_t T, int64_t D, int32_t type, void* workspace,
                            int64_t workspace_bytes, void* cuda_stream);

/* ------------------------------------------------------------------------ */
/* Loss against targets and a teacher                                       */
/* ------------------------------------------------------------------------ */

/* The loss of T rows of logits [T][ldl] (V wide) against a target token each
 * and a teacher's K largest logits, and its gradient.  Per row, with z the
 * temperature, q = softmax(logits), q' = softmax(logits / z), p = softmax over
 * the row's K entries of teacher / z, j_k their indices and w the row's weight:
 *   loss[t] = w * ((1 - alpha) * -log q[target]
 *                  + alpha * z^2 * sum_k p_k * (log p_k - log q'[j_k]))
 *   dlogits[t][j] = grad_scale * d loss[t] / d logits[t][j]
 * alpha 0 is plain cross-entropy (K, index and teacher are not looked at),
 * alpha 1 the teacher alone (targets is not looked at).
 * targets: int32 [T]; one outside [0, V) leaves its row without the first
 * term.  index: int32 [T][ldk]; an index outside [0, V) and a teacher's logit
 * of minus infinity have no probability, a row without any (or K = 0) has no
 * second term.  An index that occurs twice counts as two entries.  teacher:
 * [T][ldk] of teacher_type (ZERO_TYPE_FP16, _BF16 or _FP32).  weights: fp32
 * [T] or NULL (ones).  A row with weight 0 or without terms gets loss 0 and a
 * gradient of zeros, whatever its logits hold.  Logits of minus infinity
 * (masked) have probability 0: a row whose target, or a teacher's entry with a
 * probability, is masked has an infinite loss (its gradient is finite), and one
 * with a term whose logits are all masked has neither a loss nor a gradient:
 * both are NaN, as they are of a row that holds NaN or plus infinity.  Give such
 * rows weight 0.
 * The second term is z^2 times a difference of fp32 logarithms, off by about
 * z^2 2^-19: where the teacher's entries are nearly all of V and z is in the
 * hundreds, that is not small beside the term (its gradient is not concerned).
 * loss: fp32 [T].  dlogits [T][lddl], of `type` like the logits, or NULL (not
 * computed); it may be logits itself (same pointer and stride).  Sums are in
 * fp32, the gradient is rounded once; the same call gives the same bits.  T
 * may be 0.
 * Errors: ZERO_EINVAL (a null pointer, T above 2^31 - 513, V above 2^30, K
 * outside [0, 1024], a row stride below its row, temperature outside [2^-10,
 * 2^10], alpha outside [0, 1], grad_scale not finite, a type unknown),
 * ZERO_EALIGN (a pointer not on its element size), ZERO_EOVERLAP (an output
 * shares an element with an input or the other output), ZERO_ECUDA. */
int zero_distill_loss(const void* logits, int64_t ldl, const int32_t* targets,
                      const int32_t* index, const void* teacher, int64_t ldk,
                      const float* weights, float* loss, void* dlogits, int64_t lddl, int64_t T,
                      int64_t V, int64_t K, float temperature, float alpha, float grad_scale,
                      int32_t type, int32_t teacher_type, void* cuda_stream);

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
