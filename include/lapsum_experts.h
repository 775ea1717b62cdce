/*
 * lapsum_experts.h -- C ABI of the operators of a layer of experts behind a
 * router, the hard counterpart of the soft top-k memberships of
 * lapsum_topk.h: the choice of k experts per token with their weights, the
 * exchange between token order and expert order, and the product of every
 * expert's rows with its own weights, each with its backward pass.
 *
 * Conventions (those of lapsum_topk.h):
 *   - All array pointers are DEVICE pointers owned by the caller, row-major,
 *     each with its own row stride in elements.  The library allocates no
 *     memory.  Outputs may not overlap inputs.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream) of the
 *     current device, on which the arrays live.  No entry point synchronises
 *     the host; every one may be captured into a CUDA graph.
 *   - Arguments are validated on the host before anything is launched; a
 *     non-zero return code (LAPSUM_* of lapsum_topk.h) means nothing was
 *     enqueued.  Index arrays (chosen experts, slots, rows, offsets) are
 *     read on the device: an index out of range is treated as "none", never
 *     followed.
 *   - Nothing is accumulated by atomics in floating point: the same call on
 *     the same inputs gives the same bits.
 *   - The first call on a device sets kernel attributes; later ones do not.
 */
#ifndef LAPSUM_EXPERTS_H
#define LAPSUM_EXPERTS_H

#include <stddef.h>
#include <stdint.h>

#include "lapsum_topk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types ------------------------------------------------------ */
#define LAPSUM_F32 0
#define LAPSUM_BF16 1
#define LAPSUM_F16 2

/* ---- limits ------------------------------------------------------------- */
#define LAPSUM_EXPERTS_MAX 1024   /* experts of a layer */
#define LAPSUM_EXPERTS_MAX_K 32   /* experts of one token */
#define LAPSUM_EXPERTS_MAX_GROUPS 32

/* ---- scores of the router ----------------------------------------------- */
#define LAPSUM_SCORE_SOFTMAX 0
#define LAPSUM_SCORE_SIGMOID 1
#define LAPSUM_SCORE_IDENTITY 2   /* scores are memberships already (for
                                     instance those of lapsum_topk_fwd) */

/*
 * Choice of experts.  For the scores l_1..l_E of one token:
 *
 *     s = softmax(l) | sigmoid(l) | l,     key_i = s_i + bias_i,
 *
 * the experts fall into `groups` groups of E/groups neighbours; a group's
 * value is the sum of its group_top (1 or 2) highest keys; the groups_kept
 * groups of highest value stay, and of their experts the k with the highest
 * keys are chosen, in descending order of the key; ties go to the lowest
 * index, of groups and of experts.  Without a bias and without sums of two keys
 * the scores themselves are compared; keys closer than fp32 can tell apart are
 * compared in fp64.  The weights leave the bias out:
 *
 *     w_j = scale * s_{e_j}                  (renormalize == 0)
 *     w_j = scale * s_{e_j} / sum_m s_{e_m}  (renormalize != 0; 0 when the sum
 *                                             is 0, softmax and sigmoid in fp64)
 *
 * An expert whose score or bias is -inf is masked: it counts as if it were
 * not there (also in the softmax's denominator).  Where fewer than k experts
 * are left, the remaining places get expert -1 and weight 0; a group with no
 * expert left is never kept before one that has some.  A token with a NaN or
 * +inf in an unmasked score or bias gets expert -1 and weight NaN in all
 * places.
 *
 *   scores      in   [tokens, row_stride] of type dtype
 *   k           in   1 <= k <= min(LAPSUM_EXPERTS_MAX_K, E/groups*groups_kept)
 *   bias        in   fp32 [E], or NULL
 *   groups      in   a divisor of E, at most LAPSUM_EXPERTS_MAX_GROUPS;
 *                    groups_kept in 1..groups
 *   scale       in   finite, > 0
 *   weights     out  fp32 [tokens, k]
 *   chosen      out  int32 [tokens, k]
 */
LAPSUM_API int lapsum_experts_route_fwd(const void* scores, int dtype, int64_t tokens, int experts,
                                        int64_t row_stride, int k, int score, const float* bias, int groups,
                                        int groups_kept, int group_top, int renormalize, float scale,
                                        float* weights, int32_t* chosen, void* stream);

/*
 * Its vector-Jacobian product at fixed choice: dL/dscores (all of [tokens, E],
 * in the type of scores) from dL/dweights.  `chosen` and `weights` are the
 * forward's.  The bias has no gradient: it moves only the choice.  Masked
 * experts get 0; a token the forward gave NaN gets NaN.
 */
LAPSUM_API int lapsum_experts_route_bwd(const void* scores, int dtype, int64_t tokens, int experts,
                                        int64_t row_stride, int k, int score, const float* bias, int renormalize,
                                        float scale, const int32_t* chosen, const float* weights,
                                        const float* grad_weights, void* grad_scores, int64_t grad_stride,
                                        void* stream);

/*
 * Plan of the exchange.  Slot s = token * k + j holds expert chosen[s]; a slot
 * whose expert is not in 0..experts-1 is dropped.  The slots are put in order
 * of their expert, those of one expert in ascending order of the slot:
 *
 *   offsets     out  int32 [experts + 1]: expert e has rows
 *                    offsets[e] .. offsets[e + 1] - 1
 *   rows        out  int32 [slots]: the row of a slot, or -1
 *   slot_of     out  int32 [slots]: the slot of a row; -1 from
 *                    offsets[experts] on
 *   workspace   in   lapsum_experts_plan_workspace_size bytes, 256-byte
 *                    aligned; contents on entry are ignored
 */
LAPSUM_API size_t lapsum_experts_plan_workspace_size(int64_t slots, int experts);
LAPSUM_API int lapsum_experts_plan(const int32_t* chosen, int64_t slots, int experts, int32_t* offsets,
                                   int32_t* rows, int32_t* slot_of, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * Token order to expert order: out[r] = x[slot_of[r] / k], a row without a
 * slot gets 0.  x [tokens, dim], out [tokens * k, dim].
 */
LAPSUM_API int lapsum_experts_dispatch(const void* x, int dtype, int64_t tokens, int k, int64_t dim,
                                       int64_t x_stride, const int32_t* slot_of, void* out, int64_t out_stride,
                                       void* stream);

/*
 * Expert order to token order: out[t] = residual[t] + sum_j w[t, j] y[rows[t, j]],
 * summed in fp32 in the order of j.  A slot without a row adds w[t, j] * 0 (so
 * that a NaN weight shows).  y [tokens * k, dim]; weights fp32 [tokens, k] or
 * NULL (all 1: the backward of lapsum_experts_dispatch); residual [tokens, dim]
 * or NULL.
 */
LAPSUM_API int lapsum_experts_combine(const void* y, int dtype, int64_t tokens, int k, int64_t dim,
                                      int64_t y_stride, const float* weights, const int32_t* rows,
                                      const void* residual, int64_t residual_stride, void* out,
                                      int64_t out_stride, void* stream);

/*
 * Backward of lapsum_experts_combine for g = dL/dout [tokens, dim]:
 * grad_y[rows[t, j]] = w[t, j] g[t] (rows without a slot get 0) and
 * grad_weights[t, j] = <g[t], y[rows[t, j]]> (0 for a slot without a row).
 * Either output may be NULL.  slot_of is the plan's: the inverse of rows, of which
 * places may have been taken away since (rows[t, j] = -1, the row then has no slot).
 */
LAPSUM_API int lapsum_experts_combine_bwd(const void* grad, int dtype, int64_t tokens, int k, int64_t dim,
                                          int64_t grad_stride, const void* y, int64_t y_stride,
                                          const float* weights, const int32_t* rows, const int32_t* slot_of,
                                          void* grad_y, int64_t grad_y_stride, float* grad_weights, void* stream);

/* ---- activations of the experts' products -------------------------------- */
#define LAPSUM_ACT_NONE 0
#define LAPSUM_ACT_RELU 1
#define LAPSUM_ACT_SILU 2
#define LAPSUM_ACT_GELU 3     /* h Phi(h), Phi the normal CDF (no tanh form); before
                                 its rounding within 3e-6 of the value for |h| <= 4
                                 and 2e-5 beyond, in the lower tail too */
#define LAPSUM_ACT_SWIGLU 4   /* silu(h_i) h_{i + out/2}: half as wide */

/* ---- asynchronous status bits of the products ----------------------------- */
#define LAPSUM_EXPERTS_TIMEOUT 0x1u  /* a bounded device wait gave up: the
                                        outputs it left undone are NaN */

/*
 * Experts' product with its epilogue:
 *
 *     y_r = act(W_e x_r + b_e) + residual_r     for offsets[e] <= r < offsets[e + 1]
 *
 * with fp32 sums on the tensor cores, bias, activation and residual in fp32,
 * and one rounding to the type.  Rows from offsets[experts] on get
 * residual_r (0 without a residual).
 *
 * x, residual, y and preact (and the gradients below) are 16-byte aligned with
 * row strides that are multiples of 8.
 *   x           in   bf16 or fp16 [rows, in]
 *   weight      in   [experts, out, in], contiguous, 16-byte aligned; in and
 *                    out multiples of 8 (out of 16 for LAPSUM_ACT_SWIGLU)
 *   offsets     in   int32 [experts + 1], ascending from 0; NULL with
 *                    experts == 1: one matrix for all rows
 *   bias        in   [experts, out] of the type, or NULL
 *   residual    in   [rows, width] or NULL; width is out, or out/2 for
 *                    LAPSUM_ACT_SWIGLU
 *   y           out  [rows, width]
 *   preact      out  [rows, out] h = W_e x_r + b_e rounded to the type (fp16: what
 *                    is finite stays so, as the type's largest value; for
 *                    LAPSUM_ACT_RELU what is positive stays positive), which
 *                    the backward pass takes (rows from offsets[experts] on
 *                    are left as they were); or NULL.  y does not depend on it.
 *                    Where a factor of LAPSUM_ACT_SWIGLU lies beyond the type's
 *                    range, its gradients are those of the largest value
 *   status      i/o  uint32 [1] or NULL: LAPSUM_EXPERTS_* bits are or'ed in
 */
LAPSUM_API int lapsum_experts_linear_fwd(const void* x, int dtype, int64_t rows, int64_t in, int64_t x_stride,
                                         const void* weight, int experts, int64_t out, const int32_t* offsets,
                                         const void* bias, int activation, const void* residual,
                                         int64_t residual_stride, void* y, int64_t y_stride, void* preact,
                                         int64_t preact_stride, uint32_t* status, void* stream);

/*
 * First step of its backward: grad_h = grad_y * act'(h) (rows from
 * offsets[experts] on are left as they were) and grad_bias [experts, out] =
 * the sums of grad_h over each expert's rows, in fp32, rounded once.  preact may
 * be NULL for LAPSUM_ACT_NONE, whose grad_h may be NULL too (it is grad_y);
 * grad_bias may be NULL.
 */
LAPSUM_API size_t lapsum_experts_linear_act_workspace_size(int64_t rows, int experts, int64_t out);
LAPSUM_API int lapsum_experts_linear_act_bwd(const void* grad_y, int dtype, int64_t rows, int64_t out,
                                             int64_t grad_y_stride, const void* preact, int64_t preact_stride,
                                             int experts, const int32_t* offsets, int activation, void* grad_h,
                                             int64_t grad_h_stride, void* grad_bias, void* workspace,
                                             size_t workspace_bytes, void* stream);

/* grad_x_r = W_e^T grad_h_r; rows from offsets[experts] on get 0. */
LAPSUM_API int lapsum_experts_linear_dx(const void* grad_h, int dtype, int64_t rows, int64_t out,
                                        int64_t grad_h_stride, const void* weight, int experts, int64_t in,
                                        const int32_t* offsets, void* grad_x, int64_t grad_x_stride,
                                        uint32_t* status, void* stream);

/* grad_weight_e = sum_r grad_h_r x_r^T over the expert's rows ([experts, out, in],
   contiguous; 0 for an expert without rows). */
LAPSUM_API int lapsum_experts_linear_dweight(const void* grad_h, int dtype, int64_t rows, int64_t out,
                                             int64_t grad_h_stride, const void* x, int64_t in, int64_t x_stride,
                                             int experts, const int32_t* offsets, void* grad_weight,
                                             uint32_t* status, void* stream);

/*
 * The whole backward in one call: the three steps above, grad_h in the
 * workspace (lapsum_experts_linear_bwd_workspace_size bytes, 256-byte aligned).
 * Any of grad_x, grad_weight and grad_bias may be NULL; preact may be NULL for
 * LAPSUM_ACT_NONE.  grad_x, preact and grad_bias are contiguous.
 */
LAPSUM_API size_t lapsum_experts_linear_bwd_workspace_size(int64_t rows, int experts, int64_t out, int activation,
                                                           int with_bias);
LAPSUM_API int lapsum_experts_linear_bwd(const void* grad_y, int dtype, int64_t rows, int64_t out,
                                         int64_t grad_y_stride, const void* preact, const void* x, int64_t in,
                                         int64_t x_stride, const void* weight, int experts, const int32_t* offsets,
                                         int activation, void* grad_x, void* grad_weight, void* grad_bias,
                                         uint32_t* status, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The layer in one call: plan, dispatch, product with bias and activation,
 * product with bias, weighted sum with residual, each as above, for x [tokens,
 * dim] (bf16 or fp16), chosen and weights [tokens, k], w_in [experts, up, dim]
 * (up = hidden, or 2 hidden for LAPSUM_ACT_SWIGLU), w_out [experts, dim_out,
 * hidden] and out [tokens, dim_out].  What lies between is in the workspace
 * (lapsum_experts_mlp_workspace_size bytes, 256-byte aligned); with keep != 0 it
 * holds what lapsum_experts_mlp_bwd takes and must be left as it is until then.
 * x, residual and out have any row stride; the rest is contiguous.
 */
LAPSUM_API size_t lapsum_experts_mlp_workspace_size(int64_t tokens, int k, int experts, int64_t dim, int64_t up,
                                                    int activation, int64_t dim_out, int keep);
LAPSUM_API int lapsum_experts_mlp_fwd(const void* x, int dtype, int64_t tokens, int64_t dim, int64_t x_stride,
                                      const float* weights, const int32_t* chosen, int k, const void* w_in,
                                      const void* b_in, int experts, int64_t up, int activation, const void* w_out,
                                      const void* b_out, int64_t dim_out, const void* residual,
                                      int64_t residual_stride, void* out, int64_t out_stride, int keep,
                                      uint32_t* status, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Its backward for grad [tokens, dim_out] (any row stride): the gradients of x,
 * of the weights of the choice, of w_in, b_in, w_out and b_out, contiguous, any of
 * them NULL.  kept is the forward's workspace.  The residual's gradient is grad;
 * residual_is_x != 0 adds it to grad_x (dim == dim_out).
 */
LAPSUM_API size_t lapsum_experts_mlp_bwd_workspace_size(int64_t tokens, int k, int experts, int64_t dim, int64_t up,
                                                        int activation, int64_t dim_out);
LAPSUM_API int lapsum_experts_mlp_bwd(const void* grad, int dtype, int64_t tokens, int64_t dim, int64_t grad_stride,
                                      const float* weights, int k, const void* w_in, int experts, int64_t up,
                                      int activation, const void* w_out, int64_t dim_out, const void* kept,
                                      int residual_is_x, void* grad_x, float* grad_weights, void* grad_w_in,
                                      void* grad_b_in, void* grad_w_out, void* grad_b_out, uint32_t* status,
                                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Test knob of the calling host thread: with polls > 0 the products it launches
 * from now on copy nothing and their waits give up after that many polls, so that they end
 * with LAPSUM_EXPERTS_TIMEOUT and NaN in every row that an expert owns (a weight
 * gradient: in every expert that has rows).  Nothing waits forever and no fault
 * is raised.  0: as usual again.
 */
LAPSUM_API void lapsum_experts_test_timeout(uint32_t polls);

/* Text of the CUDA error behind the last LAPSUM_ECUDA that this library
   returned on the calling host thread. */
LAPSUM_API const char* lapsum_experts_last_cuda_error(void);

/* Counterparts of lapsum_launch_count, lapsum_trace_enable and
   lapsum_trace_collect for this library's kernels. */
LAPSUM_API uint64_t lapsum_experts_launch_count(void);
LAPSUM_API void lapsum_experts_trace_enable(int on);
LAPSUM_API int lapsum_experts_trace_collect(char* buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* LAPSUM_EXPERTS_H */
