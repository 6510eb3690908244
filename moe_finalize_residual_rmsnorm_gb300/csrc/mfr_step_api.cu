// Host side of the C ABI declared in include/moe_step_ops.h: argument checks,
// launch geometry.
#include <algorithm>
#include <cstdlib>
#include <numeric>

#include "moe_step_ops.h"
#include "mfr_op.h"

namespace {

using namespace mfr;

int64_t blocks128(int64_t n) { return (n + 127) / 128; }

// [T, heads, D] with strides, 16-bit elements.
struct Heads {
    const char* name;
    const moe_heads_t* h;
    int heads;
};

int64_t row_extent(const Heads& a, int D) { return (a.heads - 1) * a.h->head_stride + D; }      // elements of a token
int64_t extent_bytes(const Heads& a, int64_t T, int D) { return ((T - 1) * a.h->token_stride + row_extent(a, D)) * 2; }

bool same_heads(const moe_heads_t* a, const moe_heads_t* b) {
    return a->data == b->data && a->token_stride == b->token_stride && a->head_stride == b->head_stride;
}

// The heads' first elements lie a multiple of this apart; 0: there is one head.
int64_t head_pitch(const Heads& a, int64_t T) {
    return std::gcd(T > 1 ? a.h->token_stride : 0, a.heads > 1 ? a.h->head_stride : 0);
}

// Where b lies within a's period of `pitch` bytes.
int64_t offset_within(const Heads& a, const Heads& b, int64_t pitch) {
    const int64_t d = (reinterpret_cast<intptr_t>(b.h->data) - reinterpret_cast<intptr_t>(a.h->data)) % pitch;
    return d < 0 ? d + pitch : d;
}

// Whether two may share a byte.  Parts of one packed tensor are told apart by their
// places within a token (a's heads, then b's), or where heads of both lie between each
// other, by their places within the pitch that all of them keep.
bool heads_meet(const Heads& a, const Heads& b, int64_t T, int D) {
    if (!meet({a.h->data, extent_bytes(a, T, D)}, {b.h->data, extent_bytes(b, T, D)})) return false;
    const int64_t token = a.h->token_stride * 2, ra = row_extent(a, D) * 2, rb = row_extent(b, D) * 2, head = int64_t(2) * D;
    if (T > 1 && a.h->token_stride == b.h->token_stride && ra <= token && rb <= token) {
        const int64_t d = offset_within(a, b, token);
        if (d >= ra && d + rb <= token) return false;
    }
    const int64_t pitch = std::gcd(head_pitch(a, T), head_pitch(b, T)) * 2;
    if (pitch == 0) return true;
    const int64_t d = offset_within(a, b, pitch);
    return d < head || d + head > pitch;
}

// `output`: no two heads may share a byte.
int check_heads(const Heads& a, int64_t T, int D, bool output) {
    if (!a.h || !a.h->data) return MFR_FAIL(MFR_ERR_INVALID_ARG, "%s must not be NULL", a.name);
    if (!aligned(a.h->data, 16) || a.h->token_stride % 8 != 0 || a.h->head_stride % 8 != 0)
        return MFR_FAIL(MFR_ERR_MISALIGNED, "%s must be 16-byte aligned with strides that are multiples of 8", a.name);
    const int64_t most = int64_t(1) << 40;
    if (a.h->token_stride < 0 || a.h->head_stride < 0 || a.h->token_stride > most || a.h->head_stride > most)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40]", a.name);
    // no address space holds more, and the extents below stay within 64 bits
    if (T > 1 && a.h->token_stride > (int64_t(1) << 56) / T)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "%s: its tokens span more than 2^56 elements", a.name);
    // heads within a token, or tokens within a head's row
    const bool apart = (a.heads == 1 || a.h->head_stride >= D) && (T == 1 || a.h->token_stride >= row_extent(a, D));
    const bool across = (T == 1 || a.h->token_stride >= D) && (a.heads == 1 || a.h->head_stride >= (T - 1) * a.h->token_stride + D);
    if (output && !apart && !across) return MFR_FAIL(MFR_ERR_INVALID_ARG, "%s: its heads overlap", a.name);
    return MFR_OK;
}

QkSide qk_side(const moe_heads_t* x, const moe_heads_t* d, const moe_heads_t* out, const void* gamma, float* d_gamma, int heads) {
    QkSide s{};
    s.x = static_cast<const uint16_t*>(x->data);
    s.x_token = x->token_stride;
    s.x_head = x->head_stride;
    if (d) {
        s.d_out = static_cast<const uint16_t*>(d->data);
        s.d_token = d->token_stride;
        s.d_head = d->head_stride;
    }
    s.out = static_cast<uint16_t*>(out->data);
    s.out_token = out->token_stride;
    s.out_head = out->head_stride;
    s.gamma = static_cast<const uint16_t*>(gamma);
    s.d_gamma = d_gamma;
    s.heads = heads;
    return s;
}

QkParams qk_params(moe_op_t op, float eps, const float* table, const int32_t* positions) {
    QkParams p{};
    p.table = table;
    p.positions = positions;
    p.status = op->status.words;
    p.T = op->T;
    p.D = op->qk.D;
    p.rotary = op->qk.rotary;
    p.max_positions = op->qk.max_positions;
    p.eps = eps;
    return p;
}

// The inputs that both directions have.
int check_qk(const QkShape& s, const void* gamma_q, const void* gamma_k, float eps, const float* cos_sin, const int32_t* positions) {
    if (!gamma_q || !gamma_k || !positions || (s.rotary > 0 && !cos_sin)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!std::isfinite(eps) || eps < 0.f) return MFR_FAIL(MFR_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!aligned(gamma_q, 16) || !aligned(gamma_k, 16) || !aligned(cos_sin, 16) || !aligned(positions, 4))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "gammas and cos_sin must be 16-byte aligned, positions 4-byte");
    return MFR_OK;
}

// The bytes of a tensor of moe_grad_clip_run.
struct Extent {
    uintptr_t from, to;
    bool written;
};

// Whether a written one shares a byte with any other; sorts them.
bool written_meet(Extent* e, int n) {
    const auto before = [](const Extent& a, const Extent& b) { return a.from < b.from; };
    if (!std::is_sorted(e, e + n, before)) std::sort(e, e + n, before);
    uintptr_t read = 0, written = 0;          // how far those before reach
    for (int i = 0; i < n; ++i) {
        if (e[i].from < written || (e[i].written && e[i].from < read)) return true;
        uintptr_t& end = e[i].written ? written : read;
        end = std::max(end, e[i].to);
    }
    return false;
}

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
    p->wait_limit = kWaitCycles;
    if (T == 0) return MFR_OK;
    MoeLayerShape& s = p->layer;
    s.T = static_cast<int>(T);
    s.H = static_cast<int>(H);
    s.I = static_cast<int>(I);
    s.E = E;
    s.k = k;
    s.fp8 = e4m3;
    moe_layer_choose(s);
    rc = prepared(op, moe_layer_encoder() ? moe_layer_prepare(s, p->sms) : cudaErrorNotSupported);
    if (rc == MFR_OK) p->workspace = s.bytes;
    return rc;
}

int moe_small_layer_set_wait_limit(moe_op_t op, int64_t limit_cycles) {
    const int rc = check_op(op, kMoeLayer);
    if (rc != MFR_OK) return rc;
    if (limit_cycles < 0 || limit_cycles > kWaitCycles)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "limit_cycles must be in [0, %lld] (got %lld)", kWaitCycles, (long long)limit_cycles);
    op->wait_limit = limit_cycles;
    return MFR_OK;
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
    p.rows = ws + s.rows;
    p.parts = reinterpret_cast<float*>(ws + s.parts);
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
    p.wait_limit = op->wait_limit;
    const DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, moe_layer_launch(s, p, x, w13, w2, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

// ---- gate --------------------------------------------------------------------------------

int moe_gate_plan(moe_op_t* op, int64_t T, int E, int k, int score, int renormalize, float scale, int bf16_logits,
                  const mfr_options* opt) {
    int rc = begin_plan(op, T, 0);
    if (rc != MFR_OK) return rc;
    if (score != MFR_SCORE_SOFTMAX && score != MFR_SCORE_SIGMOID)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "score %d is not one of MFR_SCORE_*", score);
    if ((renormalize != 0 && renormalize != 1) || (bf16_logits != 0 && bf16_logits != 1))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "renormalize and bf16_logits must be 0 or 1");
    if (!std::isfinite(scale) || scale <= 0.f) return MFR_FAIL(MFR_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (k < 1 || k > kMaxK || E < k || E > kMaxExperts)
        return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "unsupported E=%d k=%d (need 1 <= k <= %d, k <= E <= %d)", E, k, kMaxK, kMaxExperts);
    rc = make_op(op, kGate, T, opt);
    if (rc != MFR_OK) return rc;
    moe_op_s* p = *op;
    p->E = E;
    p->k = k;
    p->gate = {score == MFR_SCORE_SIGMOID ? 1 : 0, renormalize, bf16_logits, scale};
    return prepared(op, gate_prepare(E, bf16_logits));
}

static GateParams gate_params(moe_op_t op) {
    GateParams p{};
    p.status = op->status.words;
    p.T = op->T;
    p.E = op->E;
    p.k = op->k;
    p.sigmoid = op->gate.sigmoid;
    p.renormalize = op->gate.renormalize;
    p.scale = op->gate.scale;
    return p;
}

int moe_gate_run(moe_op_t op, const void* logits, const float* bias, int32_t* expert_ids, float* topk_weights, void* stream) {
    int rc = check_op(op, kGate);
    if (rc != MFR_OK) return rc;
    if (bias && !op->gate.sigmoid) return MFR_FAIL(MFR_ERR_INVALID_ARG, "a bias needs MFR_SCORE_SIGMOID");
    if (op->T == 0) return MFR_OK;
    if (!logits || !expert_ids || !topk_weights) return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(logits, 16)) return MFR_FAIL(MFR_ERR_MISALIGNED, "logits must be 16-byte aligned");
    if (!aligned(bias, 4) || !aligned(expert_ids, 4) || !aligned(topk_weights, 4))
        return MFR_FAIL(MFR_ERR_MISALIGNED, "bias, ids and weights must be 4-byte aligned");
    const int64_t N = op->T * op->k, n = op->T * op->E;
    const Span in[] = {{logits, n * (op->gate.b16 ? 2 : 4)}, {bias, op->E * int64_t(4)}};
    const Span outs[] = {{expert_ids, N * 4}, {topk_weights, N * 4}};
    if (outputs_meet(outs, in)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "an output overlaps another argument");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    GateParams p = gate_params(op);
    p.logits = logits;
    p.bias = bias;
    p.ids = expert_ids;
    p.w = topk_weights;
    const DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, gate_launch(p, op->gate.b16, false, op->sms, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

int moe_gate_grad_run(moe_op_t op, const float* d_topk_weights, const void* logits, const int32_t* expert_ids, void* d_logits,
                      void* stream) {
    int rc = check_op(op, kGate);
    if (rc != MFR_OK) return rc;
    if (op->T == 0) return MFR_OK;
    if (!d_topk_weights || !logits || !expert_ids || !d_logits) return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(logits, 16) || !aligned(d_logits, 16)) return MFR_FAIL(MFR_ERR_MISALIGNED, "logits and d_logits must be 16-byte aligned");
    if (!aligned(expert_ids, 4) || !aligned(d_topk_weights, 4)) return MFR_FAIL(MFR_ERR_MISALIGNED, "ids and weights must be 4-byte aligned");
    const int64_t N = op->T * op->k, bytes = op->T * op->E * (op->gate.b16 ? 2 : 4);
    const Span in[] = {{d_topk_weights, N * 4}, {logits, bytes}, {expert_ids, N * 4}};
    const Span outs[] = {{d_logits, bytes}};
    if (outputs_meet(outs, in)) return MFR_FAIL(MFR_ERR_INVALID_ARG, "d_logits overlaps an input");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    GateParams p = gate_params(op);
    p.logits = logits;
    p.ids_in = expert_ids;
    p.d_w = d_topk_weights;
    p.d_logits = d_logits;
    const DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, gate_launch(p, op->gate.b16, true, op->sms, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

// ---- norms of query and key heads with the rotation -----------------------------------------

int moe_qk_norm_rope_plan(moe_op_t* op, int64_t T, int heads_q, int heads_k, int D, int rotary, int interleaved, int fp16,
                          int max_positions, const mfr_options* opt) {
    int rc = begin_plan(op, T, 0);
    if (rc != MFR_OK) return rc;
    if ((interleaved != 0 && interleaved != 1) || (fp16 != 0 && fp16 != 1))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "interleaved and fp16 must be 0 or 1");
    if (heads_q < 1 || heads_q > 1024 || heads_k < 1 || heads_k > 1024 || D < 8 || D > 512 || D % 8 != 0 || rotary < 0 ||
        rotary > D || rotary % 16 != 0 || max_positions < 1)
        return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE,
                        "unsupported shape heads %d and %d, D=%d rotary=%d max_positions=%d (need 1 to 1024 heads, D %% 8 == 0, "
                        "8 <= D <= 512, rotary %% 16 == 0, 0 <= rotary <= D, max_positions >= 1)",
                        heads_q, heads_k, D, rotary, max_positions);
    rc = make_op(op, kQkNorm, T, opt);
    if (rc != MFR_OK) return rc;
    moe_op_s* p = *op;
    p->qk = {heads_q, heads_k, D, rotary, interleaved, fp16, max_positions};
    p->workspace = static_cast<int64_t>(qk_grad_partials(p->qk, T, p->sms)) * D * 4;
    return prepared(op, qk_prepare(p->qk));
}

int moe_qk_norm_rope_run(moe_op_t op, const moe_heads_t* q, const moe_heads_t* k, const void* gamma_q, const void* gamma_k,
                         float eps, const float* cos_sin, const int32_t* positions, const moe_heads_t* q_out,
                         const moe_heads_t* k_out, void* stream) {
    int rc = check_op(op, kQkNorm);
    if (rc != MFR_OK) return rc;
    if (op->T == 0) return MFR_OK;
    const QkShape& s = op->qk;
    const int64_t T = op->T;
    const int D = s.D;
    const Heads in[] = {{"q", q, s.heads_q}, {"k", k, s.heads_k}}, out[] = {{"q_out", q_out, s.heads_q}, {"k_out", k_out, s.heads_k}};
    for (int i = 0; i < 2; ++i)
        if ((rc = check_heads(in[i], T, D, false)) != MFR_OK || (rc = check_heads(out[i], T, D, true)) != MFR_OK) return rc;
    if ((rc = check_qk(s, gamma_q, gamma_k, eps, cos_sin, positions)) != MFR_OK) return rc;
    bool clash = heads_meet(out[0], out[1], T, D);
    const Span others[] = {{gamma_q, D * 2}, {gamma_k, D * 2}, {cos_sin, int64_t(4) * s.max_positions * s.rotary}, {positions, T * 4}};
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < 2; ++j)
            if (!(i == j && same_heads(in[j].h, out[i].h))) clash = clash || heads_meet(out[i], in[j], T, D);
        for (const Span& o : others) clash = clash || meet({out[i].h->data, extent_bytes(out[i], T, D)}, o);
    }
    if (clash) return MFR_FAIL(MFR_ERR_INVALID_ARG, "an output overlaps another argument");
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    QkParams p = qk_params(op, eps, cos_sin, positions);
    p.side[0] = qk_side(q, nullptr, q_out, gamma_q, nullptr, s.heads_q);
    p.side[1] = qk_side(k, nullptr, k_out, gamma_k, nullptr, s.heads_k);
    const DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, qk_launch(s, p, false, op->sms, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

int moe_qk_norm_rope_grad_run(moe_op_t op, const moe_heads_t* d_q_out, const moe_heads_t* d_k_out, const moe_heads_t* q,
                              const moe_heads_t* k, const void* gamma_q, const void* gamma_k, float eps,
                              const float* cos_sin, const int32_t* positions, const moe_heads_t* d_q,
                              const moe_heads_t* d_k, float* d_gamma_q, float* d_gamma_k, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    int rc = check_op(op, kQkNorm);
    if (rc != MFR_OK) return rc;
    const QkShape& s = op->qk;
    const int64_t T = op->T;
    const int D = s.D;
    if (!d_gamma_q || !d_gamma_k) return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(d_gamma_q, 4) || !aligned(d_gamma_k, 4)) return MFR_FAIL(MFR_ERR_MISALIGNED, "d_gamma_q and d_gamma_k must be 4-byte aligned");
    const Span sums[] = {{d_gamma_q, D * 4}, {d_gamma_k, D * 4}, {workspace, op->workspace}};
    QkParams p{};
    if (T > 0) {
        const Heads in[] = {{"d_q_out", d_q_out, s.heads_q}, {"d_k_out", d_k_out, s.heads_k}, {"q", q, s.heads_q}, {"k", k, s.heads_k}};
        const Heads out[] = {{"d_q", d_q, s.heads_q}, {"d_k", d_k, s.heads_k}};
        for (const Heads& h : in)
            if ((rc = check_heads(h, T, D, false)) != MFR_OK) return rc;
        for (const Heads& h : out)
            if ((rc = check_heads(h, T, D, true)) != MFR_OK) return rc;
        if ((rc = check_qk(s, gamma_q, gamma_k, eps, cos_sin, positions)) != MFR_OK) return rc;
        if ((rc = check_workspace(op, workspace, workspace_bytes)) != MFR_OK) return rc;
        bool clash = heads_meet(out[0], out[1], T, D);
        const Span others[] = {{gamma_q, D * 2}, {gamma_k, D * 2}, {cos_sin, int64_t(4) * s.max_positions * s.rotary}, {positions, T * 4}};
        for (int i = 0; i < 2; ++i) {
            const Span whole{out[i].h->data, extent_bytes(out[i], T, D)};
            for (int j = 0; j < 4; ++j)
                if (!(j % 2 == i && same_heads(in[j].h, out[i].h))) clash = clash || heads_meet(out[i], in[j], T, D);
            for (const Span& o : others) clash = clash || meet(whole, o);
            for (const Span& o : sums) clash = clash || meet(whole, o);
        }
        for (const Span& o : sums)
            for (const Heads& h : in) clash = clash || meet(o, {h.h->data, extent_bytes(h, T, D)});
        if (outputs_meet(sums, others) || clash) return MFR_FAIL(MFR_ERR_INVALID_ARG, "an output overlaps another argument");
        p = qk_params(op, eps, cos_sin, positions);
        p.side[0] = qk_side(q, d_q_out, d_q, gamma_q, d_gamma_q, s.heads_q);
        p.side[1] = qk_side(k, d_k_out, d_k, gamma_k, d_gamma_k, s.heads_k);
        p.partial = static_cast<float*>(workspace);
    } else {
        if (meet(sums[0], sums[1])) return MFR_FAIL(MFR_ERR_INVALID_ARG, "an output overlaps another argument");
        p = qk_params(op, eps, cos_sin, positions);
        p.side[0].d_gamma = d_gamma_q;
        p.side[1].d_gamma = d_gamma_k;
    }
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    const DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, qk_launch(s, p, true, op->sms, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

// ---- gradient norm and clipping -----------------------------------------------------------

int moe_grad_clip_plan(moe_op_t* op, int n, const int64_t* numel, const int* types, const mfr_options* opt) {
    int rc = begin_plan(op, 0, 0);
    if (rc != MFR_OK) return rc;
    if (n < 0 || (n > 0 && (!numel || !types))) return MFR_FAIL(MFR_ERR_INVALID_ARG, "n must be >= 0 and numel and types given");
    if (n > kClipMaxTensors) return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "n=%d exceeds %d tensors", n, kClipMaxTensors);
    int64_t pieces = 0;        // of 64 KB: their numbers fit 32 bits
    for (int i = 0; i < n; ++i) {
        if (types[i] < MFR_GRAD_F32 || types[i] > MFR_GRAD_F16)
            return MFR_FAIL(MFR_ERR_INVALID_ARG, "types[%d]=%d is not one of MFR_GRAD_*", i, types[i]);
        if (numel[i] < 0) return MFR_FAIL(MFR_ERR_INVALID_ARG, "numel[%d] must be >= 0", i);
        if (numel[i] >= int64_t(1) << 40) return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "numel[%d]=%lld exceeds 2^40", i, (long long)numel[i]);
        pieces += numel[i] / (kClipMaxVectors * 4) + 1;
    }
    if (pieces >= int64_t(1) << 31) return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "too many elements in all");
    rc = make_op(op, kGradClip, 0, opt);
    if (rc != MFR_OK) return rc;
    moe_op_s* p = *op;
    p->host = std::malloc(static_cast<size_t>(n + 1) * (sizeof(int64_t) + sizeof(uint32_t) + 1));
    if (!p->host) {
        moe_op_destroy(p);
        *op = nullptr;
        return MFR_FAIL(MFR_ERR_CUDA, "out of host memory");
    }
    ClipShape& s = p->clip;
    s.n = n;
    s.numel = static_cast<int64_t*>(p->host);
    s.pieces = reinterpret_cast<uint32_t*>(s.numel + n);
    s.type = reinterpret_cast<uint8_t*>(s.pieces + n);
    for (int i = 0; i < n; ++i) {
        s.numel[i] = numel[i];
        s.type[i] = static_cast<uint8_t>(types[i]);
    }
    clip_choose(s, p->sms);
    p->workspace = static_cast<int64_t>(s.groups) * s.grid * 8;
    return prepared(op, clip_prepare());
}

int moe_grad_clip_run(moe_op_t op, const void* const* in, void* const* out, float max_norm, float eps, float* norm,
                      void* workspace, int64_t workspace_bytes, void* stream) {
    int rc = check_op(op, kGradClip);
    if (rc != MFR_OK) return rc;
    const ClipShape& s = op->clip;
    if (!norm || (s.n > 0 && (!in || !out))) return MFR_FAIL(MFR_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!std::isfinite(max_norm) || max_norm < 0.f || !std::isfinite(eps) || eps < 0.f)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "max_norm and eps must be finite and >= 0");
    if (!aligned(norm, 4)) return MFR_FAIL(MFR_ERR_MISALIGNED, "norm must be 4-byte aligned");
    if ((rc = check_workspace(op, workspace, workspace_bytes)) != MFR_OK) return rc;
    const Span mine[] = {{norm, 4}, {workspace, op->workspace}};
    // room for a few on the stack
    Extent few[2 * kClipFew + 2], *e = few;
    if (s.n > kClipFew && !(e = static_cast<Extent*>(std::malloc(sizeof(Extent) * (2 * static_cast<size_t>(s.n) + 2)))))
        return MFR_FAIL(MFR_ERR_CUDA, "out of host memory");
    int count = 0;
    const auto add = [&](const void* p, int64_t bytes, bool written) {
        const uintptr_t from = reinterpret_cast<uintptr_t>(p);
        e[count++] = {from, from + static_cast<uintptr_t>(bytes), written};
    };
    rc = MFR_OK;
    for (int i = 0; i < s.n && rc == MFR_OK; ++i) {
        if (s.numel[i] == 0) continue;
        const int size = s.type[i] == MFR_GRAD_F32 ? 4 : 2;
        if (!in[i] || !out[i]) {
            rc = MFR_FAIL(MFR_ERR_INVALID_ARG, "tensor %d is NULL", i);
        } else if (!aligned(in[i], size) || !aligned(out[i], size)) {
            rc = MFR_FAIL(MFR_ERR_MISALIGNED, "tensor %d is not aligned to its element", i);
        } else {
            add(out[i], s.numel[i] * size, true);
            if (in[i] != out[i]) add(in[i], s.numel[i] * size, false);
        }
    }
    for (const Span& m : mine) add(m.p, m.bytes, true);
    if (rc == MFR_OK && written_meet(e, count))
        rc = MFR_FAIL(MFR_ERR_INVALID_ARG, "an output, norm or the workspace overlaps another argument");
    if (e != few) std::free(e);
    if (rc != MFR_OK) return rc;
    if ((rc = check_place(op, stream)) != MFR_OK) return rc;
    ClipParams p{};
    p.partial = static_cast<double*>(workspace);
    p.norm = norm;
    p.max_norm = max_norm;
    p.eps = eps;
    p.partials = s.groups * s.grid;
    p.vectors = s.vectors;
    const DebugTurn turn(op->status, op->opt.debug_checks != 0);
    return finish(op, clip_launch(s, p, in, out, op->opt.enable_pdl ? 1 : 0, static_cast<cudaStream_t>(stream)), stream);
}

}  // extern "C"
