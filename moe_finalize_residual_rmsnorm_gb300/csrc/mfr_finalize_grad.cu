// Gradient of the finalize's weighted sum, for the pairs (t, j) that have a row r:
//
//   d_expert_out[r, h]   = bf16( w[t, j] * d_out[t, h] )
//   d_topk_weights[t, j] = sum_h d_out[t, h] * expert_out[r, h]
//
// Both come from one pass: a token's gradient is read once and, chunk by chunk
// in registers, multiplied into its k rows, while the k rows' dot products
// run beside.  It reads a row and writes a row per pair (2.35 GB at 16384 x
// 4096, k = 8), so bytes bound it, and what counts is that enough of them are
// in flight: eight 16-byte row loads a thread, three CTAs of 256 threads an SM
// (measured at that size: 345 us, 1.01 of the copy rate; two CTAs with more
// registers 430 to 630 us, four with fewer 380 us; 512 threads a CTA 432 us).
// Rows are written past L1.  The dot products are summed per thread in column
// order, over the lanes by a reduce-scatter butterfly and over the warps in
// order, all in FP32, so a call gives the same bits every time; a row's
// gradient is rounded once, from the FP32 product to bf16, the type of the rows
// that the experts' GEMMs take their gradients in.
#include "mfr_maps.cuh"

namespace mfr {
namespace {

constexpr int kThreads = 256;

template <bool F32>
__device__ __forceinline__ void load_grad(const void* d_out, int64_t at, float (&g)[8]) {
    if constexpr (F32) {
        const float* f = static_cast<const float*>(d_out) + at;
        const float4 a = ld_once_f4(f), b = ld_once_f4(f + 4);
        g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
        g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
    } else {
        unpack8(ld_stream_u4(static_cast<const uint16_t*>(d_out) + at), g);
    }
}

// A token has `wpt` warps of its CTA; thread i of them owns the chunks i, i +
// 32 wpt, ...  The CTAs before the tokens' look after the rows' side of
// the maps.
template <bool F32>
__global__ void __launch_bounds__(kThreads, 3) finalize_grad_kernel(const FinalizeGradParams p, const int wpt,
                                                                    const int row_ctas, const int rpw) {
    constexpr int kMaxTokens = kThreads / 32;
    __shared__ int s_row[kMaxTokens][kMaxK];      // -1: the pair has no row
    __shared__ float s_part[kThreads / 32][8];
    const MapParams& m = p.m;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int nck = p.H >> 3;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x < row_ctas) {
        const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * warps + warp) * rpw;
        const bool pad = lane < rpw && r0 + lane < m.R && row_is_padding(m, r0 + lane);
        for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, pad); todo; todo &= todo - 1) {
            uint16_t* row = p.d_expert_out + (r0 + __ffs(todo) - 1) * p.H;
            for (int c = lane; c < nck; c += 32) st_stream_u4(row + c * 8, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    const int mine = warp / wpt, i0 = tid - mine * wpt * 32, nt = wpt * 32;   // this thread's token of the CTA; its place there
    const int64_t t = static_cast<int64_t>(blockIdx.x - row_ctas) * (warps / wpt) + mine;
    const bool live = t < m.T;
    if (live && i0 < m.k) s_row[mine][i0] = pair_row(m, t, i0, true);
    __syncthreads();
    for (int j0 = 0; j0 < m.k; j0 += 8) {
        int row[8];
        float w[8], dot[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            row[j] = live && j0 + j < m.k ? s_row[mine][j0 + j] : -1;
            w[j] = live && j0 + j < m.k ? p.w[t * m.k + j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int c = i0; live && c < nck; c += nt) {
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = row[j] >= 0 ? ld_stream_u4(p.expert_out + static_cast<int64_t>(row[j]) * p.H + c * 8)
                                         : make_uint4(0, 0, 0, 0);
            float g[8];
            load_grad<F32>(p.d_out, t * p.H + c * 8, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (row[j] < 0) continue;
                float e[8];
                unpack8(v[j], e);
#pragma unroll
                for (int q = 0; q < 8; ++q) dot[j] = fmaf(g[q], e[q], dot[j]);
                st_stream_u4(p.d_expert_out + static_cast<int64_t>(row[j]) * p.H + c * 8,
                       make_uint4(pack_bf16x2(w[j] * g[0], w[j] * g[1]), pack_bf16x2(w[j] * g[2], w[j] * g[3]),
                                  pack_bf16x2(w[j] * g[4], w[j] * g[5]), pack_bf16x2(w[j] * g[6], w[j] * g[7])));
            }
        }
        const float sum = warp_reduce_scatter8(dot, lane);
        if ((lane & 3) == 0) s_part[warp][lane >> 2] = sum;
        __syncthreads();
        if (live && i0 < 8 && j0 + i0 < m.k) {
            float total = 0.f;
            for (int i = 0; i < wpt; ++i) total += s_part[mine * wpt + i][i0];
            p.d_w[t * m.k + j0 + i0] = total;
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t finalize_grad_launch(const FinalizeGradParams& p, int sms, int pdl, cudaStream_t s) {
    const int nck = p.H / 8;
    // One token a CTA, whose threads divide its chunks evenly (333 x 2056,
    // 257 chunks: 160 threads twice, 5.2 us; 256 threads, of which one has a
    // second chunk, 6.3 us); narrow rows share a CTA.
    const int rpw = rows_per_warp(p.m.T * nck, sms);
    int block = kThreads, wpt = 1;
    if (nck > 64) {
        const int turns = (nck + kThreads - 1) / kThreads;
        block = ((nck + turns - 1) / turns + 31) / 32 * 32;
        wpt = block / 32;
    } else if (nck > 32) {
        wpt = 2;
    }
    const int64_t tokens = block / 32 / wpt, per = static_cast<int64_t>(block / 32) * rpw;
    const int row_ctas = static_cast<int>((p.m.R + per - 1) / per);
    const int64_t grid = row_ctas + (p.m.T + tokens - 1) / tokens;
    return p.fp32 ? layer_launch(finalize_grad_kernel<true>, grid, block, 0, 1, pdl, s, p, wpt, row_ctas, rpw)
                  : layer_launch(finalize_grad_kernel<false>, grid, block, 0, 1, pdl, s, p, wpt, row_ctas, rpw);
}

}  // namespace mfr
