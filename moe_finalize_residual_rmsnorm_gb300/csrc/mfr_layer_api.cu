// Host side of the C ABI declared in include/moe_layer_ops.h: argument checks,
// launch geometry, the plan's status word.
#include <cstdlib>

#include "mfr_op.h"

namespace {

using namespace mfr;

mfr::MapParams map_params(moe_op_t op, const int32_t* row_of, const int32_t* slot_of) {
    mfr::MapParams m{};
    m.row_of = row_of;
    m.slot_of = slot_of;
    m.status = op->status.words;
    m.T = op->T;
    m.R = op->R;
    m.k = op->k;
    m.sentinel = op->opt.sentinel_skip ? 1 : 0;
    return m;
}

}  // namespace

extern "C" {

void moe_op_destroy(moe_op_t op) {
    if (!op) return;
    mfr::status_free(op->status);
    std::free(op->host);
    delete op;
}

int moe_op_get_status(moe_op_t op, void* stream, int* device_status) {
    mfr::set_last_error("%s", "");
    if (!op || !device_status) return MFR_FAIL(MFR_ERR_INVALID_ARG, "the plan and device_status must not be NULL");
    if (mfr::being_captured(static_cast<cudaStream_t>(stream)))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "the stream to wait for is being captured");
    const std::lock_guard<std::mutex> turn(op->status.turn);
    return take(op, stream, device_status);
}

int64_t moe_op_workspace_bytes(moe_op_t op) { return op ? op->workspace : -1; }

// ---- route ---------------------------------------------------------------------------

int moe_route_plan(moe_op_t* op, int64_t T, int k, int E, int align, const mfr_options* opt) {
    int rc = begin_plan(op, T, 0);
    if (rc != MFR_OK) return rc;
    if (k < 1 || k > mfr::kMaxK || E < 1 || E > mfr::kMaxExperts || align < 1 || align > mfr::kMaxAlign)
        return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "unsupported k=%d E=%d align=%d (need 1 <= k <= %d, 1 <= E <= %d, 1 <= align <= %d)",
                        k, E, align, mfr::kMaxK, mfr::kMaxExperts, mfr::kMaxAlign);
    const int64_t N = T * k;
    const int64_t R = T > 0 ? N + (E < N ? E : N) * (align - 1) : 0;
    if (R > INT32_MAX) return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "%lld rows do not fit an int32 index", (long long)R);
    rc = make_op(op, kRoute, T, opt);
    if (rc != MFR_OK) return rc;
    moe_op_s* p = *op;
    p->k = k;
    p->E = E;
    p->align = align;
    p->R = R;
    p->route = mfr::route_choose(N, R, E, p->opt.cluster_size, p->sms);
    cudaError_t e = mfr::route_prepare(p->route);
    if (e == cudaSuccess && !mfr::route_resident(p->route, E)) {
        if (p->opt.cluster_size) {
            moe_op_destroy(p);
            *op = nullptr;
            return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "a cluster of %d CTAs cannot be resident", opt->cluster_size);
        }
        p->route = mfr::route_choose(N, R, E, -1, p->sms);
        e = mfr::route_prepare(p->route);
    }
    p->workspace = N > 0 ? mfr::route_workspace(p->route, E) : 0;
    return prepared(op, e);
}

int64_t moe_route_rows(moe_op_t op) { return op && op->kind == kRoute ? op->R : -1; }

int moe_route_run(moe_op_t op, const int32_t* expert_ids, int32_t* permuted_row_of, int32_t* slot_of_row,
                  int32_t* expert_offsets, int32_t* expert_counts, void* workspace, int64_t workspace_bytes,
                  void* stream) {
    int rc = check_op(op, kRoute);
    if (rc != MFR_OK) return rc;
    const int64_t N = op->T * op->k;
    if (!expert_offsets || !expert_counts || (N > 0 && (!expert_ids || !permuted_row_of || !slot_of_row)))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(expert_ids, 4) || !aligned(permuted_row_of, 4) || !aligned(slot_of_row, 4) ||
        !aligned(expert_offsets, 4) || !aligned(expert_counts, 4))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "ids, maps, offsets and counts must be 4-byte aligned");
    if ((rc = check_workspace(op, workspace, workspace_bytes)) != MFR_OK) return rc;
    const Span in[] = {{expert_ids, N * 4}};
    const Span out[] = {{permuted_row_of, N * 4}, {slot_of_row, op->R * 4}, {expert_offsets, (op->E + 1) * int64_t(4)},
                        {expert_counts, op->E * int64_t(4)}, {workspace, op->workspace}};
    if (outputs_meet(out, in)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "two arguments overlap");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    mfr::RouteParams p{};
    p.ids = expert_ids;
    p.row_of = permuted_row_of;
    p.slot_of = slot_of_row;
    p.offsets = expert_offsets;
    p.counts = expert_counts;
    p.block_counts = static_cast<int32_t*>(workspace);
    p.status = op->status.words;
    p.N = N;
    p.R = op->R;
    p.E = op->E;
    p.align = op->align;
    p.sentinel = op->opt.sentinel_skip ? 1 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int pdl = op->opt.enable_pdl ? 1 : 0;
    const mfr::DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, N > 0 ? mfr::route_launch(p, op->route, pdl, s) : mfr::route_empty_launch(p, pdl, s), stream);
}

// ---- dispatch ------------------------------------------------------------------------

int moe_dispatch_plan(moe_op_t* op, int64_t T, int64_t H, int k, int64_t R, int elem_bytes, int sf_bytes,
                      const mfr_options* opt) {
    int rc = begin_plan(op, T, R);
    if (rc != MFR_OK) return rc;
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "elem_bytes must be 1, 2 or 4 (got %d)", elem_bytes);
    if (sf_bytes < 0 || sf_bytes > 65536) return MFR_FAIL(MFR_ERR_INVALID_ARG, "sf_bytes must be in [0, 65536] (got %d)", sf_bytes);
    if (H < 1 || H > mfr::kMaxH || H * elem_bytes % 16 != 0 || k < 1 || k > mfr::kMaxK)
        return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE,
                        "unsupported shape H=%lld k=%d (need H * elem_bytes %% 16 == 0, 1 <= H <= %d, 1 <= k <= %d)",
                        (long long)H, k, mfr::kMaxH, mfr::kMaxK);
    if (T * k > INT32_MAX) return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "T * k must fit an int32 index");
    rc = make_op(op, kDispatch, T, opt);
    if (rc != MFR_OK) return rc;
    moe_op_s* p = *op;
    p->H = H;
    p->k = k;
    p->R = R;
    p->elem_bytes = elem_bytes;
    p->sf_bytes = sf_bytes;
    return prepared(op, mfr::dispatch_prepare());
}

int moe_dispatch_run(moe_op_t op, const void* x, const void* sf, const int32_t* permuted_row_of,
                     const int32_t* slot_of_row, void* rows_out, void* sf_out, void* stream) {
    int rc = check_op(op, kDispatch);
    if (rc != MFR_OK) return rc;
    if (op->T == 0) return MFR_OK;
    const int64_t T = op->T, R = op->R, row = op->H * op->elem_bytes;
    if (!x || !permuted_row_of || (R > 0 && (!slot_of_row || !rows_out)) ||
        (op->sf_bytes > 0 && (!sf || (R > 0 && !sf_out))))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(x, 16) || !aligned(rows_out, 16)) return MFR_FAIL(MFR_ERR_MISALIGNED, "x and rows_out must be 16-byte aligned");
    if (!aligned(permuted_row_of, 4) || !aligned(slot_of_row, 4) ||
        (op->sf_bytes % 4 == 0 && op->sf_bytes > 0 && (!aligned(sf, 4) || !aligned(sf_out, 4))))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "the maps, sf and sf_out must be 4-byte aligned");
    const int64_t N = T * op->k;
    const Span in[] = {{x, T * row}, {sf, T * op->sf_bytes}, {permuted_row_of, N * 4}, {slot_of_row, R * 4}};
    const Span out[] = {{rows_out, R * row}, {sf_out, R * op->sf_bytes}};
    if (outputs_meet(out, in)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "an output overlaps another argument");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    mfr::DispatchParams p{};
    p.m = map_params(op, permuted_row_of, slot_of_row);
    p.x = static_cast<const uint8_t*>(x);
    p.sf = static_cast<const uint8_t*>(sf);
    p.out = static_cast<uint8_t*>(rows_out);
    p.sf_out = static_cast<uint8_t*>(sf_out);
    p.row_bytes = static_cast<int>(row);
    p.sf_bytes = op->sf_bytes;
    const mfr::DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, mfr::dispatch_launch(p, op->sms, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

int moe_dispatch_grad_run(moe_op_t op, const void* d_rows, const int32_t* permuted_row_of, void* d_x, void* stream) {
    int rc = check_op(op, kDispatch);
    if (rc != MFR_OK) return rc;
    if (op->elem_bytes != 2 || op->sf_bytes != 0)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "the gradient needs a plan for 16-bit rows without scales");
    if (op->T == 0) return MFR_OK;
    const int64_t T = op->T, H = op->H, R = op->R, N = T * op->k;
    if (!permuted_row_of || !d_x || (R > 0 && !d_rows)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(d_rows, 16) || !aligned(d_x, 16)) return MFR_FAIL(MFR_ERR_MISALIGNED, "d_rows and d_x must be 16-byte aligned");
    if (!aligned(permuted_row_of, 4)) return MFR_FAIL(MFR_ERR_MISALIGNED, "permuted_row_of must be 4-byte aligned");
    const Span in[] = {{d_rows, R * H * 2}, {permuted_row_of, N * 4}};
    const Span out[] = {{d_x, T * H * 2}};
    if (outputs_meet(out, in)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "d_x overlaps an input");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    mfr::DispatchGradParams p{};
    p.m = map_params(op, permuted_row_of, nullptr);
    p.d_rows = static_cast<const uint16_t*>(d_rows);
    p.d_x = static_cast<uint16_t*>(d_x);
    p.H = static_cast<int>(H);
    const mfr::DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, mfr::dispatch_grad_launch(p, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

// ---- gradient of the weighted sum -------------------------------------------------------

int moe_finalize_grad_plan(moe_op_t* op, int64_t T, int64_t H, int k, int64_t R, int grad_fp32, const mfr_options* opt) {
    int rc = begin_plan(op, T, R);
    if (rc != MFR_OK) return rc;
    if (grad_fp32 != 0 && grad_fp32 != 1) return MFR_FAIL(MFR_ERR_INVALID_ARG, "grad_fp32 must be 0 or 1 (got %d)", grad_fp32);
    if (!moe_finalize_rmsnorm_supports(H, k) || T * k > INT32_MAX)
        return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE,
                        "unsupported shape T=%lld H=%lld k=%d (need H %% 8 == 0, 8 <= H <= %d, 1 <= k <= %d, T * k < 2^31)",
                        (long long)T, (long long)H, k, mfr::kMaxH, mfr::kMaxK);
    rc = make_op(op, kFinalizeGrad, T, opt);
    if (rc != MFR_OK) return rc;
    moe_op_s* p = *op;
    p->H = H;
    p->k = k;
    p->R = R;
    p->grad_fp32 = grad_fp32;
    return prepared(op, mfr::finalize_grad_prepare(k, grad_fp32));
}

int moe_finalize_grad_run(moe_op_t op, const void* d_out, const void* expert_out, const int32_t* permuted_row_of,
                          const int32_t* slot_of_row, const float* topk_weights, void* d_expert_out,
                          float* d_topk_weights, void* stream) {
    int rc = check_op(op, kFinalizeGrad);
    if (rc != MFR_OK) return rc;
    if (op->T == 0) return MFR_OK;
    const int64_t T = op->T, R = op->R, H = op->H, N = T * op->k;
    if (!d_out || !permuted_row_of || !topk_weights || !d_topk_weights ||
        (R > 0 && (!expert_out || !slot_of_row || !d_expert_out)))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(d_out, 16) || !aligned(expert_out, 16) || !aligned(d_expert_out, 16))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "d_out, expert_out and d_expert_out must be 16-byte aligned");
    if (!aligned(permuted_row_of, 4) || !aligned(slot_of_row, 4) || !aligned(topk_weights, 4) || !aligned(d_topk_weights, 4))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "the maps and weights must be 4-byte aligned");
    const Span in[] = {{d_out, T * H * (op->grad_fp32 ? 4 : 2)}, {expert_out, R * H * 2}, {permuted_row_of, N * 4},
                       {slot_of_row, R * 4}, {topk_weights, N * 4}};
    const Span out[] = {{d_expert_out, R * H * 2}, {d_topk_weights, N * 4}};
    if (outputs_meet(out, in)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "an output overlaps another argument");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    mfr::FinalizeGradParams p{};
    p.m = map_params(op, permuted_row_of, slot_of_row);
    p.d_out = d_out;
    p.expert_out = static_cast<const uint16_t*>(expert_out);
    p.w = topk_weights;
    p.d_expert_out = static_cast<uint16_t*>(d_expert_out);
    p.d_w = d_topk_weights;
    p.H = static_cast<int>(H);
    p.fp32 = op->grad_fp32;
    const mfr::DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, mfr::finalize_grad_launch(p, op->sms, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

// ---- residual addition + RMSNorm --------------------------------------------------------

int moe_residual_rmsnorm_plan(moe_op_t* op, int64_t T, int64_t H, int quant, int sf_layout, const mfr_options* opt) {
    int rc = begin_plan(op, T, 0);
    if (rc != MFR_OK) return rc;
    if (quant < MFR_QUANT_NONE || quant > MFR_QUANT_MX32)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "quant %d is not one of MFR_QUANT_*", quant);
    if (sf_layout != MFR_SF_ROW_MAJOR && !(sf_layout == MFR_SF_TILED_128x4 && quant == MFR_QUANT_MX32))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "sf_layout %d is not available with quant %d", sf_layout, quant);
    if (!moe_finalize_rmsnorm_supports(H, 1))
        return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "unsupported H=%lld (need H %% 8 == 0, 8 <= H <= %d)", (long long)H, mfr::kMaxH);
    rc = make_op(op, kResNorm, T, opt);
    if (rc != MFR_OK) return rc;
    moe_op_s* p = *op;
    p->H = H;
    p->quant = quant;
    p->sf_tiled = sf_layout == MFR_SF_TILED_128x4 ? 1 : 0;
    return prepared(op, mfr::resnorm_prepare(T, static_cast<int>(H), quant, p->sms));
}

int64_t moe_residual_rmsnorm_sf_bytes(moe_op_t op) {
    if (!op || op->kind != kResNorm) return -1;
    const int64_t S = (op->H + 31) / 32;
    switch (op->quant) {
        case MFR_QUANT_TOKEN: return op->T * 4;
        case MFR_QUANT_GROUP128: return op->T * ((op->H + 127) / 128) * 4;
        case MFR_QUANT_MX32: return op->sf_tiled ? (op->T + 127) / 128 * 128 * ((S + 3) / 4 * 4) : op->T * S;
        default: return 0;
    }
}

int moe_residual_rmsnorm_run(moe_op_t op, const void* x, const float* residual_in, float* residual_out,
                             const void* gamma, float eps, void* out, void* out_q, void* out_sf, void* stream) {
    int rc = check_op(op, kResNorm);
    if (rc != MFR_OK) return rc;
    if (op->T == 0) return MFR_OK;
    const bool quant = op->quant != MFR_QUANT_NONE;
    if (!x || !residual_in || !residual_out || !gamma || (quant ? (!out_q || !out_sf) : !out))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!quant && (out_q || out_sf)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "a plan with MFR_QUANT_NONE writes no out_q and out_sf");
    if (!std::isfinite(eps) || eps < 0.f) return MFR_FAIL(MFR_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!aligned(x, 16) || !aligned(residual_in, 16) || !aligned(residual_out, 16) || !aligned(gamma, 16) ||
        !aligned(out, 16))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "x, residual_in, residual_out, gamma and out must be 16-byte aligned");
    if (!aligned(out_q, 8) || (op->quant != MFR_QUANT_MX32 && !aligned(out_sf, 4)))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "out_q must be 8-byte aligned and FP32 scales 4-byte aligned");
    const int64_t n = op->T * op->H;
    const Span in[] = {{x, n * 2}, {residual_in == residual_out ? nullptr : residual_in, n * 4}, {gamma, op->H * 2}};
    const Span outs[] = {{residual_out, n * 4}, {out, n * 2}, {out_q, n}, {out_sf, moe_residual_rmsnorm_sf_bytes(op)}};
    if (outputs_meet(outs, in)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "an output overlaps another argument");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    mfr::ResNormParams p{};
    p.x = static_cast<const uint16_t*>(x);
    p.residual_in = residual_in;
    p.residual_out = residual_out;
    p.gamma = static_cast<const uint16_t*>(gamma);
    p.out = static_cast<uint16_t*>(out);
    p.q = static_cast<uint8_t*>(out_q);
    p.sf = out_sf;
    p.T = op->T;
    p.H = static_cast<int>(op->H);
    p.eps = eps;
    p.quant = op->quant;
    p.sf_tiled = op->sf_tiled;
    const mfr::DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, mfr::resnorm_launch(p, op->sms, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

int moe_residual_rmsnorm_grad_plan(moe_op_t* op, int64_t T, int64_t H, const mfr_options* opt) {
    int rc = begin_plan(op, T, 0);
    if (rc != MFR_OK) return rc;
    if (!moe_finalize_rmsnorm_supports(H, 1))
        return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "unsupported H=%lld (need H %% 8 == 0, 8 <= H <= %d)", (long long)H, mfr::kMaxH);
    rc = make_op(op, kResNormGrad, T, opt);
    if (rc != MFR_OK) return rc;
    moe_op_s* p = *op;
    p->H = H;
    p->wait_limit = mfr::kWaitCycles;
    p->workspace = mfr::resnorm_grad_partials(T, static_cast<int>(H), p->sms) * H * 4;
    return prepared(op, mfr::resnorm_grad_prepare(static_cast<int>(H), false));
}

int moe_residual_rmsnorm_grad_set_wait_limit(moe_op_t op, int64_t limit_cycles) {
    int rc = check_op(op, kResNormGrad);
    if (rc != MFR_OK) return rc;
    if (limit_cycles < 0 || limit_cycles > mfr::kWaitCycles)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "limit_cycles must be in [0, %lld] (got %lld)", mfr::kWaitCycles, (long long)limit_cycles);
    if ((rc = check_device(op)) != MFR_OK) return rc;
    if (limit_cycles != mfr::kWaitCycles) {
        const cudaError_t e = mfr::resnorm_grad_prepare(static_cast<int>(op->H), true);
        if (e != cudaSuccess) return fail_cuda(MFR_ERR_CUDA, "kernel setup", e);
    }
    op->wait_limit = limit_cycles;
    return MFR_OK;
}

int moe_residual_rmsnorm_grad_run(moe_op_t op, const void* d_out, const float* d_residual_out, const float* residual,
                                  const void* gamma, float eps, float* d_residual_in, void* d_x, float* d_gamma,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
    int rc = check_op(op, kResNormGrad);
    if (rc != MFR_OK) return rc;
    const int64_t n = op->T * op->H;
    if (!d_gamma || (n > 0 && (!d_out || !residual || !gamma || !d_residual_in)))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!std::isfinite(eps) || eps < 0.f) return MFR_FAIL(MFR_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!aligned(d_out, 16) || !aligned(d_residual_out, 16) || !aligned(residual, 16) || !aligned(gamma, 16) ||
        !aligned(d_residual_in, 16) || !aligned(d_x, 16) || !aligned(d_gamma, 4))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "the matrices and gamma must be 16-byte aligned, d_gamma 4-byte");
    if ((rc = check_workspace(op, workspace, workspace_bytes)) != MFR_OK) return rc;
    const Span in[] = {{d_out, n * 2}, {d_residual_out == d_residual_in ? nullptr : d_residual_out, n * 4},
                       {residual, n * 4}, {gamma, op->H * 2}};
    const Span outs[] = {{d_residual_in, n * 4}, {d_x, n * 2}, {d_gamma, op->H * 4}, {workspace, op->workspace}};
    if (outputs_meet(outs, in)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "an output overlaps another argument");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    mfr::ResNormGradParams p{};
    p.d_out = static_cast<const uint16_t*>(d_out);
    p.d_res = d_residual_out;
    p.r = residual;
    p.gamma = static_cast<const uint16_t*>(gamma);
    p.d_in = d_residual_in;
    p.d_x = static_cast<uint16_t*>(d_x);
    p.d_gamma = d_gamma;
    p.partial = static_cast<float*>(workspace);
    p.wait_limit = op->wait_limit;
    p.status = op->status.words;
    p.T = op->T;
    p.H = static_cast<int>(op->H);
    p.eps = eps;
    const mfr::DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, mfr::resnorm_grad_launch(p, op->sms, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

}  // extern "C"
