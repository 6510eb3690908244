// Host side of the C ABI declared in include/moe_step_ops.h: argument checks,
// launch geometry.
#include "moe_step_ops.h"
#include "mfr_op.h"

namespace {

using namespace mfr;

int64_t blocks128(int64_t n) { return (n + 127) / 128; }

}  // namespace

extern "C" {

// ---- a MoE layer for a few tokens ------------------------------------------------------

int moe_small_layer_plan(moe_op_t* op, int64_t T, int64_t H, int64_t I, int E, int k, int e4m3, const mfr_options* opt) {
    int rc = begin_plan(op, T, 0);
    if (rc != MFR_OK) return rc;
    if (e4m3 != 0 && e4m3 != 1) return MFR_FAIL(MFR_ERR_INVALID_ARG, "e4m3 must be 0 or 1 (got %d)", e4m3);
    const int64_t h = e4m3 ? 16 : 8, i = e4m3 ? 128 : 8;
    if (H < h || H > kMaxH || H % h != 0 || I < i || I > kMaxH || I % i != 0 || E < 1 || E > kMaxExperts || k < 1 || k > kMaxK)
        return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE,
                        "unsupported shape H=%lld I=%lld E=%d k=%d (need H %% %lld == 0, I %% %lld == 0, H, I <= %d, 1 <= E <= %d, 1 <= k <= %d)",
                        (long long)H, (long long)I, E, k, (long long)h, (long long)i, kMaxH, kMaxExperts, kMaxK);
    if (T * k > kMoeMaxPairs)
        return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "T * k = %lld exceeds the %d pairs of a call", (long long)(T * k), kMoeMaxPairs);
    rc = make_op(op, kMoeLayer, T, opt);
    if (rc != MFR_OK) return rc;
    moe_op_s* p = *op;
    p->H = H;
    p->k = k;
    p->E = E;
    if (T == 0) return MFR_OK;
    MoeLayerShape& s = p->layer;
    s.T = static_cast<int>(T);
    s.H = static_cast<int>(H);
    s.I = static_cast<int>(I);
    s.E = E;
    s.k = k;
    s.fp8 = e4m3;
    moe_layer_choose(s, p->sms);
    p->workspace = s.bytes;
    return prepared(op, moe_layer_encoder() ? moe_layer_prepare(s) : cudaErrorNotSupported);
}

int moe_small_layer_run(moe_op_t op, const void* x, const float* x_sf, const int32_t* expert_ids,
                        const float* topk_weights, const void* w13, const float* w13_sf, const void* w2,
                        const float* w2_sf, void* out, void* workspace, int64_t workspace_bytes, void* stream) {
    int rc = check_op(op, kMoeLayer);
    if (rc != MFR_OK) return rc;
    if (op->T == 0) return MFR_OK;
    const MoeLayerShape& s = op->layer;
    if (!x || !expert_ids || !topk_weights || !w13 || !w2 || !out || (s.fp8 && (!x_sf || !w13_sf || !w2_sf)))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!s.fp8 && (x_sf || w13_sf || w2_sf)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "a plan for bf16 takes no scales");
    if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(out, 16))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "x, w13, w2 and out must be 16-byte aligned");
    if (!aligned(expert_ids, 4) || !aligned(topk_weights, 4) || !aligned(x_sf, 4) || !aligned(w13_sf, 4) || !aligned(w2_sf, 4))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "ids, weights and scales must be 4-byte aligned");
    if ((rc = check_workspace(op, workspace, workspace_bytes)) != MFR_OK) return rc;
    const int64_t T = s.T, H = s.H, I = s.I, E = s.E, P = T * s.k, b = s.fp8 ? 1 : 2, hb = blocks128(H), ib = I / 128;
    const Span in[] = {{x, T * H * b}, {x_sf, T * hb * 4}, {expert_ids, P * 4}, {topk_weights, P * 4},
                       {w13, E * 2 * I * H * b}, {w13_sf, E * 2 * ib * hb * 4}, {w2, E * H * I * b}, {w2_sf, E * hb * ib * 4}};
    const Span outs[] = {{out, T * H * 2}, {workspace, op->workspace}};
    if (outputs_meet(outs, in)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "an output overlaps another argument");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    MoeParams p{};
    p.ids = expert_ids;
    p.w = topk_weights;
    p.x_sf = x_sf;
    p.w13_sf = w13_sf;
    p.w2_sf = w2_sf;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.act = ws + s.act;
    p.act_sf = reinterpret_cast<float*>(ws + s.act_sf);
    p.y = reinterpret_cast<float*>(ws + s.y);
    p.counters = reinterpret_cast<int*>(ws + s.counters);
    p.out = static_cast<uint16_t*>(out);
    p.status = op->status.words;
    p.T = s.T;
    p.H = s.H;
    p.I = s.I;
    p.E = s.E;
    p.k = s.k;
    p.entries = s.entries;
    p.stages = s.stages;
    p.sentinel = op->opt.sentinel_skip ? 1 : 0;
    const DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, moe_layer_launch(s, p, x, w13, w2, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

}  // extern "C"
