/*
 * moe_step_ops.h — C ABI of further operators of a MoE layer's step
 * (libmfr.so, GB300 / sm_103a), next to those of moe_layer_ops.h:
 *
 *   moe_gate_*          router logits to the k experts of each token and their
 *                       weights (what moe_route_run and the finalize take), and
 *                       the gradient of the weights
 *   moe_small_layer_*   a whole MoE layer for a few tokens: the gated experts of
 *                       every token and their weighted sum
 *   moe_qk_norm_rope_*  RMSNorm of every query and key head with the position
 *                       rotation in the same pass, and its gradient
 *   moe_grad_clip_*     the L2 norm of many gradient tensors together, and the
 *                       tensors scaled to a largest norm
 *
 * Conventions are those of moe_layer_ops.h: plans are moe_op_t (moe_op_destroy,
 * moe_op_get_status, moe_op_workspace_bytes), every input is read after waiting on
 * the preceding kernel in the stream, outputs repeat bit for bit for the same
 * plan and inputs, T == 0 is a no-op unless the function says otherwise.
 */
#ifndef MOE_STEP_OPS_H
#define MOE_STEP_OPS_H

#include <stdint.h>

#include "moe_layer_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- gate: experts and weights from router logits --------------------------------
 *   p  = softmax(logits[t, :])  (MFR_SCORE_SOFTMAX)  or  sigmoid(logits[t, e])  (MFR_SCORE_SIGMOID)
 *   expert_ids[t, :]    the k experts with the largest keys, in falling order; among
 *                       equal keys the lower index first.  The key is the logit, or
 *                       with a bias sigmoid(logit) + bias[e]
 *   topk_weights[t, j]  = scale * p_j / (renormalize ? p_1 + .. + p_k : 1)   (p of the chosen;
 *                       quotients below 2^-126 may be 0)
 * An expert whose logit is -infinity or NaN (or whose key is) is never chosen and
 * does not count for the softmax.  A token with fewer than k others gets id -1 and
 * weight 0 in its last slots; moe_route_plan and the finalize take those with
 * sentinel_skip.  +infinity counts as the largest FP32 value.  The choice is that
 * of exact keys: FP32 ones that lie too close are compared in 64 bits.
 *  bf16_logits   0: logits FP32 [T, E]; 1: bf16
 *  bias          FP32 [E], MFR_SCORE_SIGMOID only; or NULL
 *  expert_ids    int32 [T, k];  topk_weights FP32 [T, k]
 * Needs 1 <= k <= 16, k <= E <= 1024, scale finite and > 0.  logits 16-byte aligned,
 * the others 4-byte.  Outputs overlap nothing. */
#define MFR_SCORE_SOFTMAX 0
#define MFR_SCORE_SIGMOID 1
int moe_gate_plan(moe_op_t* op, int64_t T, int E, int k, int score, int renormalize, float scale, int bf16_logits,
                  const mfr_options* opt);
int moe_gate_run(moe_op_t op, const void* logits, const float* bias, int32_t* expert_ids, float* topk_weights,
                 void* stream);

/* Its gradient, with the choice held fixed: d_logits [T, E] (type of the logits,
 * written whole) from d_topk_weights FP32 [T, k], the logits and the expert_ids of
 * moe_gate_run.  With q_j = p_j / (p_1 + .. + p_k) and g = scale * d_topk_weights:
 *   softmax, renormalised   d_l = q_j (g_j - <g, q>) for the chosen, else 0
 *   softmax                 d_l = p_e (g_j [e chosen] - <g, p>)
 *   sigmoid, renormalised   d_l = p_j (1 - p_j) (g_j - <g, q>) / (p_1 + .. + p_k)
 *   sigmoid                 d_l = p_j (1 - p_j) g_j
 * A slot with id -1 takes no part; an id outside [-1, E) neither, and sets
 * MFR_STATUS_BAD_INDEX.  An expert in several slots gets the sum.  The
 * biases get no gradient.  Quotients below 2^-126 may be 0.  d_logits 16-byte aligned. */
int moe_gate_grad_run(moe_op_t op, const float* d_topk_weights, const void* logits, const int32_t* expert_ids,
                      void* d_logits, void* stream);

/* ---- a MoE layer for a few tokens --------------------------------------------
 * With e = expert_ids[t, j]:
 *   h[t, j] = silu(G_e x[t]) * (U_e x[t])       silu(g) = g / (1 + exp(-g))
 *   out[t]  = bf16( sum_j topk_weights[t, j] * (D_e h[t, j]) )
 * in slot order, in FP32, for T * k <= 4096 pairs.  Larger calls are moe_route_run,
 * moe_dispatch_run, a grouped GEMM of the caller's and a finalize.  The output is an x
 * of moe_residual_rmsnorm_run.
 *  x             [T, H]
 *  expert_ids    int32 [T, k], repeats allowed.  A pair whose id lies outside [0, E)
 *                adds nothing and raises MFR_STATUS_BAD_INDEX, unless it is
 *                negative and sentinel_skip is 1; a token without pairs gets zeros
 *  topk_weights  FP32 [T, k]
 *  w13           [E, 2 I, H]: the rows of G_e, then those of U_e
 *  w2            [E, H, I]: D_e
 *  out           bf16 [T, H]
 *  workspace     moe_op_workspace_bytes(op) bytes
 * e4m3 = 0: x, w13 and w2 are bf16, and h is held as the sum of two bf16 values, off by
 *  2^-16 of itself at most (an infinity in w2 therefore gives NaN where the lower one
 *  is 0 or of the other sign).  Needs H % 8 == 0 and I % 8 == 0; x_sf, w13_sf and w2_sf
 *  NULL.
 * e4m3 = 1: x, w13 and w2 are E4M3 codes.  x_sf FP32 [T, ceil(H/128)] holds x's
 *  scales as moe_residual_rmsnorm_run writes them with MFR_QUANT_GROUP128; w13_sf
 *  FP32 [E, 2 I / 128, ceil(H/128)] and w2_sf FP32 [E, ceil(H/128), I / 128] a scale
 *  for every 128 x 128 weights; h is quantised with MFR_QUANT_GROUP128's rule.
 *  Needs H % 16 == 0 and I % 128 == 0.
 * 8 <= H, I <= 16384, 1 <= E <= 1024, 1 <= k <= 16.  x, w13, w2, out and the
 * workspace 16-byte aligned, the others 4-byte.  Outputs overlap nothing. */
int moe_small_layer_plan(moe_op_t* op, int64_t T, int64_t H, int64_t I, int E, int k, int e4m3, const mfr_options* opt);
/* Failure-path self test.  The kernels' warps hand each other stages of a ring in shared
 * memory; their waits give up after about 2 s with MFR_STATUS_TIMEOUT.  This sets
 * another limit for the plan's later runs, in SM cycles from 0 (every wait gives up at
 * once) to 4000000000 (the limit a plan begins with), else MFR_ERR_INVALID_ARG. */
int moe_small_layer_set_wait_limit(moe_op_t op, int64_t limit_cycles);
int moe_small_layer_run(moe_op_t op, const void* x, const float* x_sf, const int32_t* expert_ids,
                        const float* topk_weights, const void* w13, const float* w13_sf, const void* w2,
                        const float* w2_sf, void* out, void* workspace, int64_t workspace_bytes, void* stream);

/* ---- RMSNorm of query and key heads with the rotation ------------------------------
 * For every token t and every head x of D elements of q (and of k, with gamma_k):
 *   n = x * rsqrt(mean(x^2) + eps) * gamma_q                        (FP32)
 *   (n_a, n_b) -> (n_a cos - n_b sin, n_a sin + n_b cos)             for rotary / 2 pairs
 * pair i: elements i and i + rotary / 2, or with interleaved = 1 elements 2 i and
 * 2 i + 1; elements from `rotary` on are not rotated.  cos = cos_sin[p, i] and
 * sin = cos_sin[p, rotary / 2 + i] at p = positions[t].
 *  q, k, q_out, k_out  bf16 (fp16 = 1: fp16) [T, heads, D] with strides in elements
 *                      (moe_heads_t), multiples of 8; the D elements of a head lie
 *                      together.  Parts of one packed tensor are fine: [T, heads_q +
 *                      heads_k + .., D], or [T, heads, 3, D] with a head's parts side by
 *                      side.  q_out may be q and k_out k, with the same strides; other
 *                      overlaps are refused
 *  gamma_q, gamma_k    [D], of the same type
 *  cos_sin             FP32 [max_positions, rotary]
 *  positions           int32 [T].  A token whose position lies outside [0,
 *                      max_positions) sets MFR_STATUS_BAD_INDEX and its heads are
 *                      left as they were
 * Needs D % 8 == 0, 8 <= D <= 512, rotary % 16 == 0, 0 <= rotary <= D, 1 <= heads_q
 * and heads_k <= 1024, max_positions >= 1 (cos_sin may be NULL when rotary is 0).
 * Heads, gammas and cos_sin 16-byte aligned, positions 4-byte. */
typedef struct {
    void* data;
    int64_t token_stride;
    int64_t head_stride;
} moe_heads_t;
int moe_qk_norm_rope_plan(moe_op_t* op, int64_t T, int heads_q, int heads_k, int D, int rotary, int interleaved, int fp16,
                          int max_positions, const mfr_options* opt);
int moe_qk_norm_rope_run(moe_op_t op, const moe_heads_t* q, const moe_heads_t* k, const void* gamma_q, const void* gamma_k,
                         float eps, const float* cos_sin, const int32_t* positions, const moe_heads_t* q_out,
                         const moe_heads_t* k_out, void* stream);

/* Its gradient: with d = d_q_out turned back, unit = x * inv, inv = rsqrt(mean(x^2) + eps):
 *   d_q = inv * (gamma_q d - unit * mean(gamma_q d unit)),   d_gamma_q = sum of d * unit
 * over all tokens and heads (FP32 [D], overwritten; zeros when T == 0), and the
 * same for k.  q and k are the forward's inputs.  d_q may be d_q_out or q, d_k
 * d_k_out or k, with the same strides.  A token whose position is out of range adds
 * nothing and its d_q and d_k are left as they were.  workspace: moe_op_workspace_bytes(op). */
int moe_qk_norm_rope_grad_run(moe_op_t op, const moe_heads_t* d_q_out, const moe_heads_t* d_k_out, const moe_heads_t* q,
                              const moe_heads_t* k, const void* gamma_q, const void* gamma_k, float eps,
                              const float* cos_sin, const int32_t* positions, const moe_heads_t* d_q,
                              const moe_heads_t* d_k, float* d_gamma_q, float* d_gamma_k, void* workspace,
                              int64_t workspace_bytes, void* stream);

/* ---- gradient norm and clipping ----------------------------------------------------
 * For n tensors of numel[i] elements of types[i] (MFR_GRAD_*):
 *   norm = sqrt( sum of the squares of all elements )               -> norm[0], FP32
 *   out[i] = in[i] * min(1, max_norm / (norm + eps))                  rounded to the type
 * out[i] may be in[i].  A norm that is not finite (NaN or infinity in a tensor, or
 * squares beyond FP32: magnitudes from 1.8e19 on) scales nothing: out[i] = in[i].
 * Magnitudes below 1e-19 lose bits of their squares.
 *  in, out    host arrays of n device pointers, read during the call; each aligned
 *             to its element, fastest where in[i] and out[i] lie alike towards 16
 *             bytes; NULL where numel[i] is 0
 *  workspace  moe_op_workspace_bytes(op) bytes, 16-byte aligned
 * 0 <= n <= 65536, numel[i] < 2^40.  Outputs overlap nothing but their own input, which
 * is then the same tensor: the same tensor twice in place is refused.  A call has two
 * launches for every 512 tensors, and each second one adds all launches' sums: beyond
 * some thousands of tensors their number decides its time (8192 of 16384 FP32 elements
 * 0.56 ms, 65536 of 4096 17 ms). */
#define MFR_GRAD_F32  0
#define MFR_GRAD_BF16 1
#define MFR_GRAD_F16  2
int moe_grad_clip_plan(moe_op_t* op, int n, const int64_t* numel, const int* types, const mfr_options* opt);
int moe_grad_clip_run(moe_op_t op, const void* const* in, void* const* out, float max_norm, float eps, float* norm,
                      void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_STEP_OPS_H */
