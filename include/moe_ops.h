/*
 * moe_ops.h — C ABI of the operators around the expert pass: tokens sorted by
 * expert and back with their weights, the router's gradient, and the norms
 * between one block and the next; each with its gradient.
 *
 *   moe_permute              tokens copied into rows grouped by expert: every
 *                            (token, rank) pair, or only the pairs that
 *                            moe_expert_forward misses (slot_table given)
 *   moe_unpermute            the rows' weighted sum per token; with an fp32
 *                            output, moe_combine's miss_partial
 *   moe_permute_backward, moe_unpermute_backward
 *                            their gradients (rows, tokens and weights)
 *   moe_route_backward       gradient of moe_route_topk's gates with respect to
 *                            the logits, x, Wr and bias
 *   moe_block_norm           norm after a block, its gate, the scaled residual
 *                            and the norm before the next block, in one pass
 *   moe_block_norm_backward  its gradients
 *
 * The pages name 512 routed experts of which 10 per token are computed, hot
 * ones on the GPU and the misses elsewhere (wiselychen RTX 5090 report, "30
 * 秒定位" and §2); they give neither a layout for the missed tokens nor any
 * norm or gradient: the formulas below are this library's.
 *
 * Conventions are those of moe.h (device pointers owned by the caller, calls
 * asynchronous on `stream`, argument errors returned synchronously with nothing
 * launched, no allocation, no float atomics: identical calls give identical
 * bits).  In addition:
 *  - Matrices are row-major and contiguous.  Elements are of type `dtype`
 *    (moe_dtype); every pointer is aligned to its element.  Rows whose length
 *    in bytes is a multiple of 16, in 16-byte aligned buffers, take wider loads.
 *  - Sums, norms and softmax terms are formed in fp32 and rounded to `dtype`
 *    once, when they are stored.
 *  - Outputs alias neither inputs nor one another unless stated.
 *  - Workspaces need no initialisation and hold nothing between calls; calls
 *    sharing one must not overlap on the device.  Their sizes never fall as T
 *    grows: one for the most tokens serves every smaller batch of the same D, E
 *    and k.
 *  - Limits (MOE_ERR_UNSUPPORTED beyond): 1 <= D <= 8192, 1 <= k <= 16,
 *    1 <= E <= 1024, 0 <= T <= 65536.  T == 0 is valid.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_dtype { MOE_BF16 = 0, MOE_F16 = 1, MOE_F32 = 2 } moe_dtype;

/*
 * Tokens sorted by expert.  Pair p = t*k + r is taken if its expert ids[t][r]
 * is in [0, E) and, with slot_table, that expert's entry is outside [0,
 * n_slots): a pair moe_expert_forward reports as a miss.  The N taken pairs get
 * rows 0..N-1 by expert, then by p.  A token may name one expert twice: those
 * are two pairs.
 *   ids        int32 [T][k];  slot_table int32 [E] or NULL (every pair with an
 *              expert in range is taken; n_slots is then ignored)
 *   x          [T][D], or NULL together with rows: only the plan is made
 *   rows       [T*k][D] out: row i is x of row i's token; rows N.. are left as
 *              they were
 *   offsets    int32 [E+1] out: expert e has rows offsets[e]..offsets[e+1]-1;
 *              offsets[E] = N
 *   pair_row   int32 [T][k] out: the pair's row, -1 if it is not taken
 *   row_pair   int32 [T*k] out: the row's pair p (its token is p / k); entries
 *              N.. are left as they were
 * T == 0 zeroes offsets.
 */
moe_status moe_permute(const int32_t* ids, int T, int k, int E, const int32_t* slot_table, int n_slots, const void* x,
                       int D, int dtype, void* rows, int32_t* offsets, int32_t* pair_row, int32_t* row_pair,
                       moe_stream_t stream);

/*
 * Test hook: moe_permute's plan (no slot_table, no rows) by the kernel of large
 * batches, in one cluster of `blocks` = 16, or of 8, which moe_permute takes where
 * the device (a partition of one) has no room for 16.  T >= 1.
 */
moe_status moe_debug_permute_plan(const int32_t* ids, int T, int k, int E, int blocks, int32_t* offsets,
                                  int32_t* pair_row, int32_t* row_pair, moe_stream_t stream);

/*
 * Gradient of moe_permute's rows with respect to x:
 *   dx[t] = sum over r of drows[pair_row[t][r]], r ascending; 0 for a token
 *   without rows.
 *   drows      [n_rows][D];  pair_row int32 [T][k]: entries outside [0, n_rows)
 *              have no row;  dx [T][D] out
 */
moe_status moe_permute_backward(const void* drows, int n_rows, const int32_t* pair_row, int T, int k, int D, int dtype,
                                void* dx, moe_stream_t stream);

/*
 * Rows back to their tokens:
 *   out[t] = sum over r of weights[t][r] * rows[pair_row[t][r]], r ascending; 0
 *   for a token without rows.
 *   rows       [n_rows][D] of type dtype;  pair_row int32 [T][k]: entries
 *              outside [0, n_rows) have no row (their weight is not used)
 *   weights    fp32 [T][k] (the router's gates), or NULL: all 1
 *   out        [T][D] of type out_dtype, which is dtype or MOE_F32 (a
 *              miss_partial for moe_combine)
 */
moe_status moe_unpermute(const void* rows, int n_rows, const int32_t* pair_row, const float* weights, int T, int k,
                         int D, int dtype, void* out, int out_dtype, moe_stream_t stream);

/*
 * Gradients of moe_unpermute:
 *   drows[pair_row[t][r]] = weights[t][r] * dout[t]     (rows of no pair are left
 *                                                        as they were)
 *   dweights[t][r] = <dout[t], rows[pair_row[t][r]]>    (0 for a pair without row)
 *   dout       [T][D] of type out_dtype (dtype or MOE_F32)
 *   rows       [n_rows][D], may be NULL if dweights is
 *   drows      [n_rows][D] out;  dweights fp32 [T][k] out; either may be NULL,
 *              not both
 *   A row named by two pairs gets one of their gradients (moe_permute names
 *   each row once).
 */
moe_status moe_unpermute_backward(const void* dout, int out_dtype, const void* rows, int n_rows,
                                  const int32_t* pair_row, const float* weights, int T, int k, int D, int dtype,
                                  void* drows, float* dweights, moe_stream_t stream);

/*
 * Gradient of moe_route_topk, through the gates it returned (the selection of
 * the experts is held fixed, as it is piecewise constant):
 *   dlogits[t][r] = gates[t][r] * (dgates[t][r] - sum_j gates[t][j] dgates[t][j])
 *   dx[t]  = sum_r dlogits[t][r] * Wr[ids[t][r]]  (+ dx_add[t])
 *   dWr[e] = sum of dlogits[t][r] * x[t] over the pairs with ids[t][r] = e
 *   dbias[e] = the same sum of dlogits[t][r]
 * A pair whose id is outside [0, E) counts as gate 0.
 *   dgates, gates fp32 [T][k];  ids int32 [T][k];  x bf16 [T][D];  Wr bf16 [E][D]
 *   offsets, row_pair   moe_permute's, of these ids and E with slot_table NULL
 *   dlogits    fp32 [T][k] out (the selected logits; every other one's is 0)
 *   dx         bf16 [T][D] out or NULL;  dx_add bf16 [T][D] or NULL (dx may
 *              alias it)
 *   dWr        fp32 [E][D] out or NULL;  dbias fp32 [E] out or NULL
 *   ws         moe_route_backward_workspace_size bytes, 256-byte aligned
 * D % 256 == 0 and k <= E as in moe_route_topk; x, Wr, dx, dx_add and dWr are
 * 16-byte aligned.  T == 0 zeroes dWr and dbias.
 */
size_t moe_route_backward_workspace_size(int T, int D, int E, int k);
moe_status moe_route_backward(const float* dgates, const float* gates, const int32_t* ids, const uint16_t* x,
                              const uint16_t* Wr, const int32_t* offsets, const int32_t* row_pair, int T, int D, int E,
                              int k, const uint16_t* dx_add, float* dlogits, uint16_t* dx, float* dWr, float* dbias,
                              void* ws, size_t ws_bytes, moe_stream_t stream);

/* What moe_block_norm's gate is: absent, one value per channel or per token. */
typedef enum moe_gate_mode { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2 } moe_gate_mode;

/*
 * From one block's output to the next block's input, RMS norms:
 *   z      = y * rsqrt(mean(y^2) + eps) * w_post     (z = y if w_post is NULL)
 *   x_out  = alpha * residual + gate * z             (residual NULL: 0; no gate: 1)
 *   normed = x_out * rsqrt(mean(x_out^2) + eps) * w_next
 * per token (the means run over D).  The second norm reads x_out as it is
 * stored, rounded to dtype, so that one call gives what two calls give.
 *   y          [T][D], e.g. moe_combine's out;  residual [T][D] or NULL, the
 *              residual stream
 *   gate       fp32 [D] (MOE_GATE_CHANNEL) or [T] (MOE_GATE_TOKEN), NULL with
 *              MOE_GATE_NONE;  alpha finite
 *   w_post, w_next   fp32 [D] or NULL;  eps >= 0
 *   x_out      [T][D] out, or NULL (then only normed is written; may alias
 *              residual or y)
 *   normed     [T][D] out, given if and only if w_next is
 *   rstd_post, rstd_next   fp32 [T] out or NULL: the norms' rsqrt(...), which
 *              the gradient reads
 */
moe_status moe_block_norm(const void* y, const void* residual, const float* gate, int gate_mode, float alpha,
                          const float* w_post, const float* w_next, float eps, int T, int D, int dtype, void* x_out,
                          void* normed, float* rstd_post, float* rstd_next, moe_stream_t stream);

/*
 * Gradients of moe_block_norm (alpha and eps are constants).  With
 * xh = x_out * rstd_next, yh = y * rstd_post (y without w_post) and u = dnormed * w_next:
 *   G         = dx_out + rstd_next * (u - xh * mean(xh u))
 *   dresidual = alpha * G
 *   dgate     = sum of G * z over the tokens (channel) or channels (token)
 *   v         = gate * G * w_post,  dy = rstd_post * (v - yh * mean(yh v))
 *               (dy = gate * G if w_post is NULL)
 *   dw_post   = sum over tokens of gate * G * yh;  dw_next = sum of dnormed * xh
 *   dx_out     [T][D] or NULL (0);  dnormed [T][D], given if and only if w_next is
 *   x_out, rstd_next   the forward pass's, needed with w_next
 *   y, rstd_post       the forward pass's: rstd_post with w_post; y with
 *              w_post or dgate
 *   dy         [T][D] out;  dresidual [T][D] out or NULL (may alias dx_out)
 *   dgate, dw_post, dw_next   fp32 out or NULL, only with what they belong to
 *   ws         moe_block_norm_backward_workspace_size bytes, 256-byte aligned
 * At least one of dx_out and dnormed is given.  T == 0 zeroes dw_post, dw_next
 * and a channel gate's dgate.
 */
size_t moe_block_norm_backward_workspace_size(int T, int D);
moe_status moe_block_norm_backward(const void* dx_out, const void* dnormed, const void* x_out, const void* y,
                                   const float* gate, int gate_mode, float alpha, const float* w_post,
                                   const float* rstd_post, const float* w_next, const float* rstd_next, int T, int D,
                                   int dtype, void* dy, void* dresidual, float* dgate, float* dw_post, float* dw_next,
                                   void* ws, size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
