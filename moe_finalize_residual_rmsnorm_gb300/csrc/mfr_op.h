// What the host sides of moe_layer_ops.h (mfr_layer_api.cu) and moe_step_ops.h
// (mfr_step_api.cu) share: the plan, the checks of its options and arguments, the
// end of a run.
#pragma once

#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_runtime.h>

#include "moe_layer_ops.h"
#include "mfr_internal.h"
#include "mfr_layer.h"
#include "mfr_status.h"
#include "mfr_step.h"

namespace mfr {

enum Kind { kRoute = 1, kDispatch, kFinalizeGrad, kResNorm, kResNormGrad, kMoeLayer, kGate, kQkNorm, kGradClip };

inline const char* kind_name(Kind kind) {
    switch (kind) {
        case kRoute: return "moe_route_plan";
        case kDispatch: return "moe_dispatch_plan";
        case kFinalizeGrad: return "moe_finalize_grad_plan";
        case kResNorm: return "moe_residual_rmsnorm_plan";
        case kResNormGrad: return "moe_residual_rmsnorm_grad_plan";
        case kMoeLayer: return "moe_small_layer_plan";
        case kGate: return "moe_gate_plan";
        case kQkNorm: return "moe_qk_norm_rope_plan";
        default: return "moe_grad_clip_plan";
    }
}

}  // namespace mfr

struct moe_op_s {
    mfr::Kind kind;
    int64_t T;
    int64_t H;
    int64_t R;
    int64_t workspace;
    int64_t wait_limit;
    int k;
    int E;
    int align;
    int elem_bytes;
    int sf_bytes;
    int grad_fp32;
    int quant;
    int sf_tiled;
    int device;
    int sms;
    mfr_options opt;
    mfr::RouteLaunch route;
    mfr::MoeLayerShape layer;
    mfr::GateShape gate;
    mfr::QkShape qk;
    mfr::ClipShape clip;
    void* host;          // owned: the clip shape's arrays
    mfr::StatusWord status;
};

namespace mfr {

#define MFR_FAIL(code, ...) (mfr::set_last_error(__VA_ARGS__), (code))

inline int fail_cuda(int code, const char* what, cudaError_t e) {
    cudaGetLastError();
    return MFR_FAIL(code, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
    const void* p;
    int64_t bytes;
};

inline bool meet(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// Whether an output shares a byte with an input or with another output.
template <int NO, int NI>
bool outputs_meet(const Span (&out)[NO], const Span (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (meet(out[i], in[j])) return true;
        for (int j = i + 1; j < NO; ++j)
            if (meet(out[i], out[j])) return true;
    }
    return false;
}

// What every plan checks first; clears *op.
inline int begin_plan(moe_op_t* op, int64_t T, int64_t R) {
    set_last_error("%s", "");
    if (!op) return MFR_FAIL(MFR_ERR_INVALID_ARG, "the plan must not be NULL");
    *op = nullptr;
    if (T < 0 || R < 0)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "T and R must be >= 0 (T=%lld R=%lld)", (long long)T, (long long)R);
    if (T > (int64_t(1) << 26)) return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "T=%lld exceeds 2^26 tokens per call", (long long)T);
    if (R > INT32_MAX) return MFR_FAIL(MFR_ERR_UNSUPPORTED_SHAPE, "R must fit an int32 index");
    return MFR_OK;
}

// Checks the options, finds the device and makes a plan without its operator's own fields.
inline int make_op(moe_op_t* op, Kind kind, int64_t T, const mfr_options* opt) {
    mfr_options o;
    moe_finalize_rmsnorm_default_options(&o);
    if (opt) o = *opt;
    if (o.force_variant != MFR_VARIANT_AUTO)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "force_variant %d: this operator has no variants", o.force_variant);
    const bool pow2 = o.cluster_size == 1 || o.cluster_size == 2 || o.cluster_size == 4 || o.cluster_size == 8 ||
                      o.cluster_size == 16;
    if (o.cluster_size != 0 && !(kind == kRoute && pow2))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "cluster_size %d is not available here", o.cluster_size);
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(MFR_ERR_BAD_DEVICE, "cudaGetDevice", e);
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return fail_cuda(MFR_ERR_BAD_DEVICE, "cudaDeviceGetAttribute", e);
    if (major != 10 || minor != 3)
        return MFR_FAIL(MFR_ERR_BAD_DEVICE, "device %d is sm_%d%d; this library is built for sm_103a only", dev, major, minor);
    moe_op_s* p = new (std::nothrow) moe_op_s{};
    if (!p) return MFR_FAIL(MFR_ERR_CUDA, "out of host memory");
    p->kind = kind;
    p->T = T;
    p->device = dev;
    p->sms = sms;
    p->opt = o;
    if ((e = mfr::status_make(p->status)) != cudaSuccess) {
        moe_op_destroy(p);
        return fail_cuda(MFR_ERR_CUDA, "the plan's status word", e);
    }
    *op = p;
    return MFR_OK;
}

// The end of a plan: its kernels are loaded and set up, or there is none.
inline int prepared(moe_op_t* op, cudaError_t e) {
    if (e == cudaSuccess) return MFR_OK;
    moe_op_destroy(*op);
    *op = nullptr;
    return fail_cuda(MFR_ERR_CUDA, "kernel setup", e);
}

// What every run checks first.
inline int check_op(moe_op_t op, Kind kind) {
    set_last_error("%s", "");
    if (!op) return MFR_FAIL(MFR_ERR_INVALID_ARG, "the plan must not be NULL");
    if (op->kind != kind) return MFR_FAIL(MFR_ERR_INVALID_ARG, "this plan was not made by %s", kind_name(kind));
    return MFR_OK;
}

inline int check_device(moe_op_t op) {
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(MFR_ERR_CUDA, "cudaGetDevice", e);
    if (dev != op->device)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "current device %d is not the plan's device %d", dev, op->device);
    return MFR_OK;
}

// What every run checks last.
inline int check_place(moe_op_t op, void* stream) {
    const int rc = check_device(op);
    if (rc != MFR_OK) return rc;
    if (op->opt.debug_checks && mfr::being_captured(static_cast<cudaStream_t>(stream)))
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "a call with debug_checks waits for its stream, which is being captured");
    return MFR_OK;
}

inline int check_workspace(moe_op_t op, const void* workspace, int64_t bytes) {
    if (op->workspace == 0) return MFR_OK;
    if (!workspace || bytes < op->workspace)
        return MFR_FAIL(MFR_ERR_INVALID_ARG, "workspace of %lld bytes is smaller than the %lld the plan needs",
                        (long long)(workspace ? bytes : 0), (long long)op->workspace);
    if (!aligned(workspace, 16)) return MFR_FAIL(MFR_ERR_MISALIGNED, "the workspace must be 16-byte aligned");
    return MFR_OK;
}

inline int take(moe_op_t op, void* stream, int* bits) {
    const cudaError_t e = mfr::status_take(op->status, static_cast<cudaStream_t>(stream), bits);
    return e == cudaSuccess ? MFR_OK : fail_cuda(MFR_ERR_CUDA, "reading the status word", e);
}

// The end of a run, whose DebugTurn the caller holds.
inline int finish(moe_op_t op, cudaError_t e, void* stream) {
    if (e != cudaSuccess) return fail_cuda(MFR_ERR_LAUNCH, "kernel launch", e);
    if (op->opt.debug_checks) {
        int st = 0;
        const int rc = take(op, stream, &st);
        if (rc != MFR_OK) return rc;
        if (st & MFR_STATUS_TIMEOUT)
            return MFR_FAIL(MFR_ERR_CUDA, "an on-chip wait timed out; the outputs are not valid");
        if (st & MFR_STATUS_BAD_INDEX) return MFR_FAIL(MFR_ERR_BAD_INDEX, "an expert id, an index map entry or a position was out of range");
    }
    return MFR_OK;
}

}  // namespace mfr
