// Gradient of the finalize's weighted sum.
#include "mfr_maps.cuh"

namespace mfr {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kRowsPerWarp = 32;

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

// CTA b < T: token b.  CTAs behind: the rows' side of the maps.
template <bool F32>
__global__ void __launch_bounds__(kMaxThreads) finalize_grad_kernel(const FinalizeGradParams p) {
    __shared__ int s_row[kMaxK];
    __shared__ float s_w[kMaxK];
    __shared__ float s_part[kMaxThreads / 32][8];
    const MapParams& m = p.m;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int nck = p.H >> 3;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x >= m.T) {
        const int64_t r0 = ((blockIdx.x - m.T) * warps + warp) * kRowsPerWarp;
        if (r0 >= m.R) return;
        const bool pad = r0 + lane < m.R && row_is_padding(m, r0 + lane);
        for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, pad); todo; todo &= todo - 1) {
            uint16_t* row = p.d_expert_out + (r0 + __ffs(todo) - 1) * p.H;
            for (int c = lane; c < nck; c += 32) st_u4(row + c * 8, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    const int64_t t = blockIdx.x;
    if (tid < m.k) {
        s_row[tid] = pair_row(m, t, tid, true);
        s_w[tid] = p.w[t * m.k + tid];
    }
    __syncthreads();
    for (int j0 = 0; j0 < m.k; j0 += 8) {
        int row[8];
        float w[8], dot[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            row[j] = j0 + j < m.k ? s_row[j0 + j] : -1;
            w[j] = j0 + j < m.k ? s_w[j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int c = tid; c < nck; c += blockDim.x) {
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
                const uint4 o = make_uint4(pack_bf16x2(w[j] * g[0], w[j] * g[1]), pack_bf16x2(w[j] * g[2], w[j] * g[3]),
                                           pack_bf16x2(w[j] * g[4], w[j] * g[5]), pack_bf16x2(w[j] * g[6], w[j] * g[7]));
                st_u4(p.d_expert_out + static_cast<int64_t>(row[j]) * p.H + c * 8, o);
            }
        }
        const float sum = warp_reduce_scatter8(dot, lane);
        if ((lane & 3) == 0) s_part[warp][lane >> 2] = sum;
        __syncthreads();
        if (tid < 8 && j0 + tid < m.k) {
            float total = 0.f;
            for (int i = 0; i < warps; ++i) total += s_part[i][tid];
            p.d_w[t * m.k + j0 + tid] = total;
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t finalize_grad_launch(const FinalizeGradParams& p, int sms, int pdl, cudaStream_t s) {
    (void)sms;
    const int nck = p.H / 8;
    int block = (nck + 31) / 32 * 32;
    if (block > 256) block = 256;
    const int64_t per = static_cast<int64_t>(block / 32) * kRowsPerWarp;
    const int64_t grid = p.m.T + (p.m.R + per - 1) / per;
    return p.fp32 ? layer_launch(finalize_grad_kernel<true>, grid, block, 0, 1, pdl, s, p)
                  : layer_launch(finalize_grad_kernel<false>, grid, block, 0, 1, pdl, s, p);
}

}  // namespace mfr
