/*
 * moe_step_ops.h — C ABI of further operators of a MoE layer's step
 * (libmfr.so, GB300 / sm_103a), next to those of moe_layer_ops.h:
 *
 *   moe_small_layer_*   a whole MoE layer for a few tokens: the gated experts of
 *                       every token and their weighted sum
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

/* ---- a MoE layer for a few tokens --------------------------------------------
 * With e = expert_ids[t, j]:
 *   h[t, j] = silu(G_e x[t]) * (U_e x[t])       silu(g) = g / (1 + exp(-g))
 *   out[t]  = bf16( sum_j topk_weights[t, j] * (D_e h[t, j]) )
 * in slot order, in FP32, for T * k <= 4096 pairs.  Larger calls are moe_route_run,
 * moe_dispatch_run, a grouped GEMM and a finalize.  The output is an x of
 * moe_residual_rmsnorm_run.
 *  x             [T, H]
 *  expert_ids    int32 [T, k], repeats allowed.  A pair whose id lies outside [0, E)
 *                adds nothing and raises MFR_STATUS_BAD_INDEX, unless it is
 *                negative and sentinel_skip is 1; a token without pairs gets zeros
 *  topk_weights  FP32 [T, k]
 *  w13           [E, 2 I, H]: the rows of G_e, then those of U_e
 *  w2            [E, H, I]: D_e
 *  out           bf16 [T, H]
 *  workspace     moe_op_workspace_bytes(op) bytes
 * e4m3 = 0: x, w13 and w2 are bf16 and h is rounded to bf16.  Needs H % 8 == 0 and
 *  I % 8 == 0; x_sf, w13_sf and w2_sf NULL.
 * e4m3 = 1: x, w13 and w2 are E4M3 codes.  x_sf FP32 [T, ceil(H/128)] holds x's
 *  scales as moe_residual_rmsnorm_run writes them with MFR_QUANT_GROUP128; w13_sf
 *  FP32 [E, 2 I / 128, ceil(H/128)] and w2_sf FP32 [E, ceil(H/128), I / 128] a scale
 *  for every 128 x 128 weights; h is quantised with MFR_QUANT_GROUP128's rule.
 *  Needs H % 16 == 0 and I % 128 == 0.
 * 8 <= H, I <= 16384, 1 <= E <= 1024, 1 <= k <= 16.  x, w13, w2, out and the
 * workspace 16-byte aligned, the others 4-byte.  Outputs overlap nothing. */
int moe_small_layer_plan(moe_op_t* op, int64_t T, int64_t H, int64_t I, int E, int k, int e4m3, const mfr_options* opt);
int moe_small_layer_run(moe_op_t op, const void* x, const float* x_sf, const int32_t* expert_ids,
                        const float* topk_weights, const void* w13, const float* w13_sf, const void* w2,
                        const float* w2_sf, void* out, void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_STEP_OPS_H */
