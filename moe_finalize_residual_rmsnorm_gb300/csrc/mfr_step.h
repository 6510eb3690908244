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
constexpr int kMoeThreads = 352;   // two warps that load, one that multiplies, eight that finish

struct MoeLayerShape {
    int T;
    int H;
    int I;
    int E;
    int k;
    int fp8;
    int columns;      // NB: pairs that one accumulator holds, 16 .. 128
    int stages;       // of the ring
    int smem;
    int entries;      // most (expert, chunk of pairs) entries
    int cluster[2];   // CTAs of a cluster and of the grid, by launch
    int grid[2];
    // workspace: byte offsets
    int64_t act;      // [pairs, I] E4M3, or [2, pairs, I] bf16: upper and lower parts; pairs sorted by expert
    int64_t act_sf;   // [pairs, I / 128] FP32 (E4M3)
    int64_t y;        // [pairs, H] FP32
    int64_t rows;     // [pairs, H] bf16: x in the sorted order, where that is a launch of its own; or nothing
    int64_t parts;    // FP32 sums of units that are divided along K, a CTA's in a row; or nothing
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
    uint8_t* rows;
    float* parts;
    uint16_t* out;            // [T, H]
    int* status;
    int T;
    int H;
    int I;
    int E;
    int k;
    int entries;
    int stages;
    int cluster;              // CTAs of a cluster of this launch
    int sentinel;
    long long wait_limit;     // cycles after which a wait gives up: kWaitCycles, or less to test that
};

// Fills the shared memory's and the workspace's layout from T .. fp8.
void moe_layer_choose(MoeLayerShape& s);
// Sets the kernels up and fills the launch geometry and the workspace's size.
cudaError_t moe_layer_prepare(MoeLayerShape& s, int sms);
// The encoder of tensor maps that the driver has; NULL: it has none.
void* moe_layer_encoder();
cudaError_t moe_layer_launch(const MoeLayerShape& s, const MoeParams& p, const void* x, const void* w13, const void* w2,
                             int pdl, cudaStream_t st);

// ---- gate (mfr_gate.cu) ----------------------------------------------------------------
struct GateShape {
    int sigmoid;
    int renormalize;
    int b16;
    float scale;
};

struct GateParams {
    const void* logits;      // [T, E] FP32 or bf16
    const float* bias;       // [E], or NULL
    int32_t* ids;            // [T, k]
    float* w;                // [T, k]
    const int32_t* ids_in;   // the gradient's
    const float* d_w;
    void* d_logits;
    int* status;
    int64_t T;
    int E;
    int k;
    int sigmoid;
    int renormalize;
    float scale;
};

cudaError_t gate_prepare(int E, int b16);
cudaError_t gate_launch(const GateParams& p, int b16, bool grad, int sms, int pdl, cudaStream_t s);

// ---- norms of query and key heads with the rotation (mfr_qk_norm.cu) -----------------------
struct QkShape {
    int heads_q;
    int heads_k;
    int D;
    int rotary;
    int interleaved;
    int fp16;
    int max_positions;
};

// One side: queries or keys.  Strides in elements.
struct QkSide {
    const uint16_t* x;       // [T, heads, D]
    const uint16_t* d_out;   // the gradient's
    uint16_t* out;           // the output, or d_x
    const uint16_t* gamma;   // [D]
    float* d_gamma;          // [D]
    int64_t x_token, x_head, d_token, d_head, out_token, out_head;
    int heads;
};

struct QkParams {
    QkSide side[2];
    const float* table;      // [max_positions, rotary]: cosines, then sines
    const int32_t* positions;
    float* partial;          // the gradient's: [blocks, D]
    int* status;
    int64_t T;
    int D;
    int rotary;
    int max_positions;
    float eps;
};

cudaError_t qk_prepare(const QkShape& s);
// Rows of partial gamma gradients.
int qk_grad_partials(const QkShape& s, int64_t T, int sms);
cudaError_t qk_launch(const QkShape& s, const QkParams& p, bool grad, int sms, int pdl, cudaStream_t st);

// ---- gradient norm and clipping (mfr_clip.cu) ------------------------------------------------
constexpr int kClipGroup = 512;           // tensors of one launch
constexpr int kClipFew = 64;
constexpr int kClipMaxVectors = 4096;     // 16-byte vectors of a piece
constexpr int kClipMaxTensors = 65536;

struct ClipShape {
    int n;
    int groups;
    int grid;
    int vectors;
    int64_t* numel;          // [n], owned, as are the others
    uint32_t* pieces;
    uint8_t* type;
};

template <int N>
struct ClipList {
    const void* in[N];
    void* out[N];
    int64_t numel[N];
    uint32_t first[N + 1];   // piece
    int n;
    uint8_t type[N];         // MFR_GRAD_*
};

struct ClipParams {
    double* partial;
    float* norm;
    float max_norm;
    float eps;
    int partials;
    int partial_at;
    int vectors;
};

void clip_choose(ClipShape& s, int sms);
cudaError_t clip_prepare();
cudaError_t clip_launch(const ClipShape& s, const ClipParams& p, const void* const* in, void* const* out, int pdl, cudaStream_t st);

}  // namespace mfr
