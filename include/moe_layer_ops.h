/*
 * moe_layer_ops.h — C ABI of the operators that stand around the MoE finalize
 * in one MoE block (libmfr.so, GB300 / sm_103a):
 *
 *   moe_route_*               (token, slot) pairs sorted by expert: the index
 *                             maps every other call here and the finalize read
 *   moe_dispatch_*            token rows copied into expert order, and the
 *                             gradient of that copy
 *   moe_finalize_grad_*       gradient of the finalize's weighted sum
 *   moe_residual_rmsnorm_*    residual addition + RMSNorm, written in 8 bits
 *                             (E4M3) with scales and / or in bf16
 *   moe_residual_rmsnorm_grad_*  gradient of residual addition + RMSNorm
 *
 * The gradient of the fused finalize (moe_finalize_rmsnorm_run: weighted sum
 * + residual + RMSNorm) is moe_residual_rmsnorm_grad_run on its residual_out,
 * then moe_finalize_grad_run with d_out = that call's d_residual_in.
 *
 * Conventions are those of moe_finalize_rmsnorm.h (device pointers owned by
 * the caller, dense row-major layouts, `stream` a cudaStream_t as void*, every
 * function returns MFR_OK or an MFR_ERR_* code with its reason in
 * moe_finalize_rmsnorm_last_error(), no run allocates), and:
 *  - Plans (moe_op_t) are made for the current device and belong to one
 *    operator; each run function refuses another operator's plan.  A plan holds
 *    its status word on the device (8 bytes) and nothing else there.
 *  - mfr_options: enable_pdl, debug_checks and sentinel_skip have the meaning
 *    they have for the finalize, except that these kernels read EVERY input
 *    after waiting on the preceding kernel in the stream, so any input may
 *    come from it.  force_variant must be MFR_VARIANT_AUTO; cluster_size 0
 *    except where a plan says otherwise.
 *  - A kernel that a plan launched may be followed by a finalize plan with
 *    enable_pdl = 1, which reads permuted_row_of, topk_weights and gamma
 *    before its own wait: those must not be outputs of the call directly
 *    before it in the stream.
 *  - A plan may be run concurrently on several streams; calls that are given
 *    the same workspace, graphs that captured it included, must not overlap.
 *    The status word belongs to the plan: its bits are those of all its calls
 *    since the last reading, whatever their streams.  With debug_checks a
 *    plan's calls take turns, each from its launch to its check, so that a
 *    call reports its own bits.
 *    MFR_STATUS_TIMEOUT: every output of that call, its workspace included, is
 *    invalid.
 *  - Runs may be captured into a graph, which must not outlive its plans.  Make
 *    plans before the capture.  debug_checks and moe_op_get_status wait for
 *    their stream: on a stream that is being captured they are refused with
 *    MFR_ERR_INVALID_ARG and the capture goes on; on another stream they work
 *    while it does.
 *  - Sums are FP32, in an order that the plan fixes: the same plan and inputs
 *    give the same bits.  A plan of another T may add a token's terms in
 *    another order, so a token's last bits can change with the size of its batch.
 *  - T == 0 is a no-op returning MFR_OK unless the function says otherwise.
 *
 * The pair of index maps.  A pair s = t * k + j (token t, slot j) has the row
 * permuted_row_of[s] of the [R, H] matrices in expert order, and row r has the
 * pair slot_of_row[r].  They are inverse to each other:
 *   permuted_row_of[s]  in [0, R), or negative: the pair's expert is not local
 *                       (allowed with sentinel_skip = 1)
 *   slot_of_row[r]      >= 0: the row's pair; MFR_ROW_PADDING: the row only
 *                       fills its expert's block up; MFR_ROW_UNUSED: the row
 *                       lies behind the last block
 * moe_dispatch_run and moe_finalize_grad_run read both and write row r for
 * pair s only where permuted_row_of[s] == r and slot_of_row[r] == s.  Any
 * disagreement (an index out of range, two pairs with the same row, a row
 * whose pair points elsewhere) sets MFR_STATUS_BAD_INDEX; the row is left as it
 * was, and the pair's weight gradient is 0.  Padding rows are written with
 * zeros, unused rows are left as they were.
 */
#ifndef MOE_LAYER_OPS_H
#define MOE_LAYER_OPS_H

#include <stdint.h>

#include "moe_finalize_rmsnorm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MFR_ROW_PADDING (-1)
#define MFR_ROW_UNUSED  (-2)

typedef struct moe_op_s* moe_op_t;

/* Frees a plan (NULL is allowed), also while a graph that does not use it is
 * being captured.  No call with it may be in flight. */
void moe_op_destroy(moe_op_t op);

/* Waits for `stream`, then reads the plan's status word (MFR_STATUS_* bits) into
 * *device_status and clears it in one step: a bit that a call on another
 * stream raises meanwhile is in this reading or in the next. */
int moe_op_get_status(moe_op_t op, void* stream, int* device_status);

/* Bytes of the device workspace the operator's run function takes (0: none
 * needed, NULL accepted); -1 for a NULL plan. */
int64_t moe_op_workspace_bytes(moe_op_t op);

/* ---- route: pairs sorted by expert ---------------------------------------
 * A stable counting sort of the T * k pairs by expert id.  With c_e the pairs
 * of expert e and p_e = c_e rounded up to a multiple of `align`:
 *   expert_offsets[e]  = p_0 + ... + p_{e-1}     (e = 0 .. E: E + 1 values)
 *   expert_counts[e]   = c_e
 *   permuted_row_of[s] = expert_offsets[e] + (pairs of expert e before s)
 * and slot_of_row as above.  align > 1 gives every expert's block the row
 * granularity of a grouped GEMM's tile.
 * Needs 1 <= k <= 16, 1 <= E <= 1024, 1 <= align <= 4096 and
 * moe_route_rows <= 2^31 - 1.
 * expert_ids: int32 [T, k], in any order, repeats allowed.  An id outside
 * [0, E) gets permuted_row_of -1; it raises MFR_STATUS_BAD_INDEX unless it is
 * negative and sentinel_skip is 1.
 * The outputs are written whole.  All pointers 4-byte aligned; no two overlap.
 * cluster_size (0 = automatic, else 1, 2, 4, 8 or 16): CTAs of the one-launch
 * form, for up to 4096 pairs a CTA; larger calls take two launches and a
 * workspace (16-byte aligned).  T == 0 writes expert_offsets and expert_counts
 * (zeros). */
int moe_route_plan(moe_op_t* op, int64_t T, int k, int E, int align, const mfr_options* opt);
/* Rows R that always hold every block: T*k + min(E, T*k) * (align - 1); -1
 * for a plan of another kind. */
int64_t moe_route_rows(moe_op_t op);
int moe_route_run(moe_op_t op, const int32_t* expert_ids, int32_t* permuted_row_of, int32_t* slot_of_row,
                  int32_t* expert_offsets, int32_t* expert_counts, void* workspace, int64_t workspace_bytes,
                  void* stream);

/* ---- dispatch: token rows into expert order --------------------------------
 * rows_out[permuted_row_of[t, j], :] = x[t, :] for every pair, and the same for
 * the rows of scales, sf_out[permuted_row_of[t, j], :] = sf[t, :].
 *  elem_bytes  size of an element of x and rows_out: 1, 2 or 4 (the values are
 *              copied, not read); H * elem_bytes a multiple of 16, H <= 16384
 *  sf_bytes    bytes of one row of scales, up to 65536; 0: none, sf and sf_out
 *              NULL
 *  x, rows_out 16-byte aligned, sf and sf_out 4-byte where sf_bytes is a
 *              multiple of 4; R up to 2^31 - 1
 * Outputs overlap nothing. */
int moe_dispatch_plan(moe_op_t* op, int64_t T, int64_t H, int k, int64_t R, int elem_bytes, int sf_bytes,
                      const mfr_options* opt);
int moe_dispatch_run(moe_op_t op, const void* x, const void* sf, const int32_t* permuted_row_of,
                     const int32_t* slot_of_row, void* rows_out, void* sf_out, void* stream);

/* Its gradient, for bf16 rows (plans with elem_bytes = 2 and sf_bytes = 0):
 *   d_x[t, :] = bf16( sum_j d_rows[permuted_row_of[t, j], :] )
 * summed in FP32 in slot order.  A pair whose entry lies outside [0, R) adds
 * nothing and sets MFR_STATUS_BAD_INDEX, unless it is negative and
 * sentinel_skip is 1.  d_rows and d_x bf16, 16-byte aligned; d_x overlaps no
 * input. */
int moe_dispatch_grad_run(moe_op_t op, const void* d_rows, const int32_t* permuted_row_of, void* d_x, void* stream);

/* ---- gradient of the finalize's weighted sum --------------------------------
 * For out[t] = sum_j w[t, j] * E[permuted_row_of[t, j]] (moe_finalize_run):
 *   d_expert_out[permuted_row_of[t, j], h] = bf16( w[t, j] * d_out[t, h] )
 *   d_topk_weights[t, j] = sum_h d_out[t, h] * E[permuted_row_of[t, j], h]   (FP32)
 * d_topk_weights of a pair without a row is 0.
 *  grad_fp32   0: d_out is bf16 [T, H]; 1: FP32 [T, H]
 *  expert_out, d_out, d_expert_out 16-byte aligned; the others 4-byte
 * Shapes as for moe_finalize_plan.  Outputs overlap nothing. */
int moe_finalize_grad_plan(moe_op_t* op, int64_t T, int64_t H, int k, int64_t R, int grad_fp32,
                           const mfr_options* opt);
int moe_finalize_grad_run(moe_op_t op, const void* d_out, const void* expert_out, const int32_t* permuted_row_of,
                          const int32_t* slot_of_row, const float* topk_weights, void* d_expert_out,
                          float* d_topk_weights, void* stream);

/* ---- residual addition + RMSNorm, 8-bit output ---------------------------------
 *   r = residual_in + x                                      (FP32) -> residual_out
 *   y = (r * rsqrt(mean_h(r^2) + eps)) * gamma                (FP32)
 * y is written in bf16 (out, when not NULL) and / or, by `quant`, as E4M3
 * codes with scales (out_q, out_sf): for each group of columns of a token,
 *   amax = min(max(max |y|, 2^-100), FLT_MAX)
 *   MFR_QUANT_TOKEN     one group of H columns   \  scale = amax / 448 (FP32),
 *   MFR_QUANT_GROUP128  groups of 128 columns    /  q = E4M3(y * (448 / amax))
 *   MFR_QUANT_MX32      groups of 32 columns: scale = the smallest power of two
 *                       with amax / scale <= 448, stored as E8M0 (its exponent
 *                       + 127, one byte), q = E4M3(y / scale)
 *   MFR_QUANT_NONE      no 8-bit output (out_q and out_sf NULL, out required)
 * so that y ~ value(q) * scale.  E4M3 rounds to nearest even and saturates at
 * 448; a NaN in y is the code 0x7F and does not count for amax.  The last
 * group of a row may be shorter.
 *  x       bf16 [T, H];  residual_in / residual_out FP32 [T, H], may be equal
 *  out     bf16 [T, H];  out_q uint8 [T, H];  gamma bf16 [H]
 *  out_sf  FP32 [T] / FP32 [T, ceil(H/128)] / uint8 [T, ceil(H/32)] row-major,
 *          or for MFR_QUANT_MX32 with MFR_SF_TILED_128x4 the tiled layout of
 *          moe_finalize_rmsnorm_nvfp4_plan_ex (padding bytes are not written)
 *  x, residuals, gamma, out 16-byte aligned; out_q 8-byte; out_sf 4-byte
 *          (1-byte for MX32)
 * Needs H % 8 == 0, 8 <= H <= 16384.  sf_layout other than MFR_SF_ROW_MAJOR
 * only with MFR_QUANT_MX32. */
#define MFR_QUANT_NONE     0
#define MFR_QUANT_TOKEN    1
#define MFR_QUANT_GROUP128 2
#define MFR_QUANT_MX32     3
int moe_residual_rmsnorm_plan(moe_op_t* op, int64_t T, int64_t H, int quant, int sf_layout, const mfr_options* opt);
/* Bytes of out_sf (0 for MFR_QUANT_NONE); -1 for a plan of another kind. */
int64_t moe_residual_rmsnorm_sf_bytes(moe_op_t op);
int moe_residual_rmsnorm_run(moe_op_t op, const void* x, const float* residual_in, float* residual_out,
                             const void* gamma, float eps, void* out, void* out_q, void* out_sf, void* stream);

/* ---- gradient of residual addition + RMSNorm -------------------------------------
 * For r = residual_in + x, y = r * inv * gamma, inv = (mean(r^2) + eps)^-1/2,
 * with d_out the gradient of y and d_residual_out that of r from elsewhere:
 *   d_r = d_residual_out + inv * (gamma * d_out) - r * inv^3 * mean_h(gamma * d_out * r)
 *   d_residual_in = d_r (FP32);   d_x = bf16(d_r)
 *   d_gamma[h] = sum_t d_out[t, h] * r[t, h] * inv[t]           (FP32)
 *  d_out           bf16 [T, H]
 *  d_residual_out  FP32 [T, H], or NULL for zeros
 *  residual        FP32 [T, H]: r, the forward's residual_out
 *  d_residual_in   FP32 [T, H]; may equal d_residual_out
 *  d_x             bf16 [T, H], or NULL
 *  d_gamma         FP32 [H], overwritten (zeros when T == 0)
 *  workspace       moe_op_workspace_bytes(op) bytes, 16-byte aligned
 * Matrices and gamma 16-byte aligned, d_gamma 4-byte.  Needs H % 8 == 0, 8 <= H <= 16384. */
int moe_residual_rmsnorm_grad_plan(moe_op_t* op, int64_t T, int64_t H, const mfr_options* opt);
/* Failure-path self test.  Rows of more than 512 columns pass through a ring in
 * shared memory, whose waits give up after about 2 s with MFR_STATUS_TIMEOUT.  This
 * sets another limit for the plan's later runs, in SM cycles from 0 (every
 * wait gives up at once) to 4000000000 (the limit a plan begins with), else
 * MFR_ERR_INVALID_ARG.  The next run is not affected by one that gave up. */
int moe_residual_rmsnorm_grad_set_wait_limit(moe_op_t op, int64_t limit_cycles);
int moe_residual_rmsnorm_grad_run(moe_op_t op, const void* d_out, const float* d_residual_out, const float* residual,
                                  const void* gamma, float eps, float* d_residual_in, void* d_x, float* d_gamma,
                                  void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_OPS_H */
