// Declarations shared by the host side of moe_step_ops.h (mfr_step_api.cu) and
// its kernel files.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mfr {

// ---- a MoE layer for a few tokens (mfr_moe_layer.cu) ---------------------------------
constexpr int kMoeMaxPairs = 4096;
constexpr int kMoeRows = 128;      // weight rows of one accumulator; a tile of weights has two
constexpr int kMoeThreads = 320;   // a warp that loads, one that multiplies, eight that finish

struct MoeLayerShape {
    int T;
    int H;
    int I;
    int E;
    int k;
    int fp8;
    int columns;      // NB: pairs that one accumulator holds, 16 .. 128
    int stages;
    int smem;
    int entries;      // most (expert, chunk of pairs) entries
    int grid;
    // workspace: byte offsets
    int64_t act;      // [pairs, I] bf16 or E4M3
    int64_t act_sf;   // [pairs, I / 128] FP32 (E4M3)
    int64_t y;        // [pairs, H] FP32
    int64_t counters; // [tiles of H] int
    int64_t bytes;
};

struct MoeParams {
    const int32_t* ids;       // [T, k]
    const float* w;           // [T, k]
    const float* x_sf;        // E4M3: [T, ceil(H / 128)]
    const float* w13_sf;      // E4M3: [E, 2 I / 128, ceil(H / 128)]
    const float* w2_sf;       // E4M3: [E, ceil(H / 128), I / 128]
    uint8_t* act;
    float* act_sf;
    float* y;
    int* counters;
    uint16_t* out;            // [T, H]
    int* status;
    int T;
    int H;
    int I;
    int E;
    int k;
    int entries;
    int stages;
    int sentinel;
};

// Fills the launch geometry and the workspace's layout from T .. fp8.
void moe_layer_choose(MoeLayerShape& s, int sms);
cudaError_t moe_layer_prepare(const MoeLayerShape& s);
// The encoder of tensor maps that the driver has; NULL: it has none.
void* moe_layer_encoder();
cudaError_t moe_layer_launch(const MoeLayerShape& s, const MoeParams& p, const void* x, const void* w13, const void* w2,
                             int pdl, cudaStream_t st);

}  // namespace mfr
