// Declarations shared by the host side of moe_layer_ops.h (mfr_layer_api.cu)
// and its kernel files.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mfr_policy.h"

namespace mfr {

constexpr int kMaxExperts = 1024;
constexpr int kMaxAlign = 4096;

// ---- route (mfr_route.cu) -----------------------------------------------------
constexpr int kRouteThreads = 1024;
constexpr int kRouteMaxItems = 4;                      // one launch: pairs per thread
constexpr int64_t kRouteOneLaunchPairs = 32 * 1024;    // calls up to here are one launch

struct RouteParams {
    const int32_t* ids;      // [N]
    int32_t* row_of;         // [N]
    int32_t* slot_of;        // [R]
    int32_t* offsets;        // [E + 1]
    int32_t* counts;         // [E]
    int32_t* block_counts;   // [blocks, block_pitch(E)]: the two-launch form's workspace
    int* status;
    int64_t N;
    int64_t R;
    int E;
    int align;
    int sentinel;
};

struct RouteLaunch {
    int cluster;   // CTAs of the one-launch form; 0: the two-launch form
    int threads;   // per CTA, at least E
    int items;     // pairs per thread
    int blocks;    // two-launch form: CTAs of each launch
    int rounds;    // two-launch form: turns of a CTA
};

// Launch geometry for N pairs and R rows; forced: CTAs of the one-launch form,
// 0: automatic, -1: the two-launch form.
RouteLaunch route_choose(int64_t N, int64_t R, int E, int forced, int sms);
int64_t route_workspace(const RouteLaunch& l, int E);
cudaError_t route_prepare(const RouteLaunch& l);
// Whether the device holds the one-launch form's cluster.
bool route_resident(const RouteLaunch& l, int E);
cudaError_t route_launch(const RouteParams& p, const RouteLaunch& l, int pdl, cudaStream_t s);
// The outputs of a call without pairs.
cudaError_t route_empty_launch(const RouteParams& p, int pdl, cudaStream_t s);

// ---- dispatch and the finalize's gradient (mfr_dispatch.cu, mfr_finalize_grad.cu) ----
struct MapParams {
    const int32_t* row_of;    // [T, k]
    const int32_t* slot_of;   // [R]
    int* status;
    int64_t T;
    int64_t R;
    int k;
    int sentinel;
};

// Whether `chunks` 16-byte pieces of tokens are 2048 an SM or more: enough for
// several waves of work, so that bytes count and latency does not.
inline bool fills_gpu(int64_t chunks, int sms) { return chunks > int64_t(2048) * sms; }

// Rows whose padding one warp looks after: half as many as there are tokens an
// SM, more where rows outnumber them by far, 1 to 32.  The warps that do come
// first in the grid, so that the zeros they write, row after row, are not the
// call's tail (measured, dispatch of 16384 x 4096 to 8 slots, blocks of 128:
// 208 us with them last, 190 first), and a small call has many of them (1024 x
// 2048, blocks of 16: 12.7 us with 32 rows, 7.3 with 8, 6.7 with 4 and with the
// rule's 3; 16384 x 4096: 190 us with 32, 192 with 8, 194 with 4).
inline int rows_per_warp(int64_t T, int64_t R, int sms) {
    const int64_t by_tokens = T / (2 * static_cast<int64_t>(sms)), by_rows = R / (64 * static_cast<int64_t>(sms));
    const int64_t rows = by_tokens > by_rows ? by_tokens : by_rows;
    return rows < 1 ? 1 : rows > 32 ? 32 : static_cast<int>(rows);
}

struct DispatchParams {
    MapParams m;
    const uint8_t* x;         // [T, row_bytes]
    const uint8_t* sf;        // [T, sf_bytes]
    uint8_t* out;             // [R, row_bytes]
    uint8_t* sf_out;          // [R, sf_bytes]
    int row_bytes;            // a multiple of 16
    int sf_bytes;
};

struct DispatchGradParams {
    MapParams m;              // slot_of: not read
    const uint16_t* d_rows;   // [R, H]
    uint16_t* d_x;            // [T, H]
    int H;
};

// Each prepare loads the kernels that the plan's calls launch and sets their attributes.
cudaError_t dispatch_prepare();
cudaError_t dispatch_launch(const DispatchParams& p, int sms, int pdl, cudaStream_t s);
cudaError_t dispatch_grad_launch(const DispatchGradParams& p, int pdl, cudaStream_t s);

struct FinalizeGradParams {
    MapParams m;
    const void* d_out;          // [T, H] bf16 or fp32
    const uint16_t* expert_out; // [R, H]
    const float* w;             // [T, k]
    uint16_t* d_expert_out;     // [R, H]
    float* d_w;                 // [T, k]
    int H;
    int fp32;
};

cudaError_t finalize_grad_prepare(int k, int fp32);
cudaError_t finalize_grad_launch(const FinalizeGradParams& p, int sms, int pdl, cudaStream_t s);

// ---- residual addition + RMSNorm (mfr_resnorm.cu) --------------------------------
struct ResNormParams {
    const uint16_t* x;
    const float* residual_in;
    float* residual_out;
    const uint16_t* gamma;
    uint16_t* out;       // NULL: none
    uint8_t* q;
    void* sf;            // FP32, or E8M0 bytes
    int64_t T;
    int H;
    float eps;
    int quant;           // MFR_QUANT_*
    int sf_tiled;
};

cudaError_t resnorm_prepare(int64_t T, int H, int quant, int sms);
cudaError_t resnorm_launch(const ResNormParams& p, int sms, int pdl, cudaStream_t s);

struct ResNormGradParams {
    const uint16_t* d_out;
    const float* d_res;   // NULL: zeros
    const float* r;
    const uint16_t* gamma;
    float* d_in;
    uint16_t* d_x;        // NULL: none
    float* d_gamma;
    float* partial;       // [resnorm_grad_partials, H]
    int* status;
    int64_t T;
    int H;
    float eps;
    long long wait_limit; // cycles after which a wait of the ring gives up: kWaitCycles, or less to test that
};

// Rows of the workspace of partial gamma gradients: resnorm_grad_partials.
cudaError_t resnorm_grad_prepare(int H, bool limited);
int resnorm_grad_partials(int64_t T, int H, int sms);
cudaError_t resnorm_grad_launch(const ResNormGradParams& p, int sms, int pdl, cudaStream_t s);

// Loads a kernel when its plan is made, so that its first launch may be a captured one.
template <typename Kernel>
cudaError_t preload(Kernel* kernel) {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(kernel));
}

// A kernel launch with programmatic stream serialization and a cluster along x, where asked for.
template <typename... Params, typename... Args>
cudaError_t layer_launch(void (*kernel)(Params...), int64_t grid, int block, int smem, int cluster, int pdl,
                         cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(block), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(n);
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace mfr
